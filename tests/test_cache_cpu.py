"""The paged cache without a GPU: what the C entry points and the binding
refuse before anything is launched, workspace sizes, and the plain models the
GPU tests go by."""
import ctypes
import math

import paged_model as pm
import pytest
import torch

from top_token_selection_b200 import build as pbuild
from top_token_selection_b200 import pivot as pv

FAKE = 0x10000   # never dereferenced: every call below fails validation first, or has nothing to do
WS = (FAKE, 1 << 40)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    pv.load()


def cache(**kw):
    base = dict(dtype=pv.BF16, B=4, Hkv=2, D=64, page_size=16, num_pages=32, max_pages=8, k=FAKE,
                v=FAKE, k_scale=None, v_scale=None, table=FAKE, len=FAKE, refs=FAKE)
    base.update(kw)
    return pv.PivotCache(*base.values())


def call(**kw):
    base = dict(Hq=4, total=9, max_new=3, q=FAKE, cu_new=FAKE, scale=0.1, window=0, idx=None,
                topk=0, o=FAKE, lse=None)
    base.update(kw)
    return pv.PivotAttend(*base.values())


BAD_CACHE = [
    (dict(dtype=3), 1), (dict(dtype=pv.F32), 2), (dict(B=0), 1), (dict(Hkv=0), 1), (dict(D=0), 1),
    (dict(page_size=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(table=None), 1), (dict(len=None), 1), (dict(refs=None), 1), (dict(k=FAKE + 8), 1),
    (dict(k_scale=FAKE, v_scale=FAKE), 1), (dict(dtype=pv.E4M3), 1),
    (dict(dtype=pv.E4M3, k_scale=FAKE), 1), (dict(D=12), 2), (dict(B=65537), 2),
    (dict(num_pages=1 << 28), 2), (dict(max_pages=1 << 28), 2),
]


@pytest.mark.parametrize("bad,want", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(bad, want):
    c = cache(**bad)
    assert pv.pivot_cache_append(c, FAKE, FAKE, FAKE, 4, 4, FAKE, *WS, None) == want
    assert pv.pivot_pages_fork(c, FAKE, FAKE, 2, *WS, None) == want
    assert pv.pivot_pages_free(c, FAKE, FAKE, 2, None) == want
    assert pv.pivot_pages_compact(c, None, None, *WS, None) == want
    assert pv.pivot_paged_attention(c, call(), *WS, None) == want
    assert pv.pivot_selected_attention(c, call(idx=FAKE, topk=4), *WS, None) == want
    assert pv.pivot_cache_append_workspace_size(c, 4) == 0
    assert pv.pivot_pages_fork_workspace_size(c, 2) == 0
    assert pv.pivot_pages_compact_workspace_size(c) == 0
    assert pv.pivot_paged_attention_workspace_size(c, call()) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(Hq=0), 1), (dict(Hq=5), 1), (dict(total=-1), 1), (dict(max_new=0), 1), (dict(q=None), 1),
    (dict(cu_new=None), 1), (dict(o=None), 1), (dict(q=FAKE + 2), 1), (dict(o=FAKE + 8), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(window=-1), 1), (dict(total=1 << 30, Hq=8), 2),
])
def test_attention_refuses(bad, want):
    assert pv.pivot_paged_attention(cache(), call(**bad), *WS, None) == want
    sel = dict(idx=FAKE, topk=8)
    assert pv.pivot_selected_attention(cache(), call(**{**sel, **bad}), *WS, None) == want


def test_attention_refuses_more():
    c = cache()
    assert pv.pivot_paged_attention(c, call(idx=FAKE), *WS, None) == 1            # paged takes no idx
    assert pv.pivot_paged_attention(c, call(topk=4), *WS, None) == 1
    assert pv.pivot_selected_attention(c, call(), *WS, None) == 1                  # idx and topk
    assert pv.pivot_selected_attention(c, call(idx=FAKE), *WS, None) == 1
    assert pv.pivot_selected_attention(c, call(topk=4), *WS, None) == 1
    assert pv.pivot_selected_attention(c, call(idx=FAKE, topk=4, window=3), *WS, None) == 1
    assert pv.pivot_selected_attention(c, call(idx=FAKE, topk=65537), *WS, None) == 2
    assert pv.pivot_paged_attention(cache(D=32), call(), *WS, None) == 2
    assert pv.pivot_paged_attention(c, call(scale=2e30), *WS, None) == 1
    assert pv.pivot_paged_attention(cache(max_pages=(1 << 22) + 1), call(), *WS, None) == 2
    assert pv.pivot_paged_attention(cache(D=256), call(), *WS, None) == 2
    assert pv.pivot_paged_attention(c, call(), None, 1 << 40, None) == 1
    assert pv.pivot_paged_attention(c, call(), FAKE + 16, 1 << 40, None) == 1
    need = pv.pivot_paged_attention_workspace_size(c, call())
    assert need > 0 and need % 256 == 0
    assert pv.pivot_paged_attention(c, call(), FAKE, need - 1, None) == 3
    need = pv.pivot_selected_attention_workspace_size(c, call(idx=FAKE, topk=4))
    assert pv.pivot_selected_attention(c, call(idx=FAKE, topk=4), FAKE, need - 1, None) == 3
    # no rows: nothing to do, whatever the pointers
    assert pv.pivot_paged_attention(c, call(total=0, q=None, o=None, cu_new=None), *WS, None) == 0


def test_workspace_holds_the_plan_and_grows_with_the_batch():
    small = pv.pivot_paged_attention_workspace_size(cache(), call())
    big = pv.pivot_paged_attention_workspace_size(cache(), call(total=1 << 20, max_new=1 << 20))
    assert small < big < 1 << 30


def test_page_calls_refuse():
    c = cache()
    app = lambda *a: pv.pivot_cache_append(c, *a)          # noqa: E731
    assert app(None, FAKE, FAKE, 4, 4, FAKE, *WS, None) == 1
    assert app(FAKE, None, FAKE, 4, 4, FAKE, *WS, None) == 1
    assert app(FAKE, FAKE, None, 4, 4, FAKE, *WS, None) == 1
    assert app(FAKE, FAKE, FAKE, -1, 4, FAKE, *WS, None) == 1
    assert app(FAKE, FAKE, FAKE, 4, 0, FAKE, *WS, None) == 1
    assert app(FAKE, FAKE, FAKE, 4, 4, None, *WS, None) == 1
    assert app(FAKE + 8, FAKE, FAKE, 4, 4, FAKE, *WS, None) == 1
    assert app(FAKE, FAKE, FAKE, 4, 4, FAKE, FAKE + 4, 1 << 30, None) == 1
    assert app(FAKE, FAKE, FAKE, 4, 4, FAKE, FAKE, 64, None) == 3
    assert app(FAKE, FAKE, FAKE, (1 << 30) + 1, 4, FAKE, *WS, None) == 2
    assert pv.pivot_pages_fork(c, None, FAKE, 2, *WS, None) == 1
    assert pv.pivot_pages_fork(c, FAKE, FAKE, 5, *WS, None) == 1                   # more pairs than sequences
    assert pv.pivot_pages_fork(c, FAKE, FAKE, -1, *WS, None) == 1
    assert pv.pivot_pages_fork(c, FAKE, FAKE, 2, FAKE, 16, None) == 3
    assert pv.pivot_pages_fork(c, None, None, 0, *WS, None) == 0
    assert pv.pivot_pages_free(c, FAKE, None, 2, None) == 1
    assert pv.pivot_pages_free(c, FAKE, FAKE, 5, None) == 1
    assert pv.pivot_pages_free(c, None, None, 0, None) == 0
    assert pv.pivot_pages_compact(c, None, None, FAKE, 16, None) == 3
    cp = pv.pivot_pages_copy
    assert cp(None, 4, FAKE, 4, 64, FAKE, FAKE, 1, None) == 1
    assert cp(FAKE, 0, FAKE, 4, 64, FAKE, FAKE, 1, None) == 1
    assert cp(FAKE, 4, FAKE, 4, 24, FAKE, FAKE, 1, None) == 1                      # 16 bytes at a time
    assert cp(FAKE, 4, FAKE, 4, 0, FAKE, FAKE, 1, None) == 1
    assert cp(FAKE + 4, 4, FAKE, 4, 64, FAKE, FAKE, 1, None) == 1
    assert cp(FAKE, 4, FAKE, 4, 64, None, FAKE, 1, None) == 1
    assert cp(FAKE, 4, FAKE, 4, 64, FAKE, FAKE, -1, None) == 1
    assert cp(FAKE, 4, FAKE, 4, 64, None, None, 0, None) == 0


def test_binding_refuses_tensors_of_the_wrong_kind():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)    # noqa: E731
    with pytest.raises(ValueError):                        # not on a GPU
        pv.make_cache(k, k, i32(2, 3), i32(2), i32(4))
    dev = torch.device("cpu")
    with pytest.raises(TypeError):
        pv._arg(i32(2).long(), "x", torch.int32, (2,), dev)
    with pytest.raises(ValueError):
        pv._arg(i32(2), "x", torch.int32, (3,), dev)
    with pytest.raises(ValueError):
        pv._arg(i32(4, 4).t()[:, :2], "x", torch.int32, (4, 2), dev)
    with pytest.raises(TypeError):
        pv._arg([1, 2], "x", torch.int32, (2,), dev)
    assert pv._arg(i32(2), "x", torch.int32, (2,), dev) > 0


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(pv.PivotCache) == 7 * 4 + 4 + 7 * 8
    assert ctypes.sizeof(pv.PivotAttend) == 3 * 4 + 4 + 2 * 8 + 2 * 4 + 8 + 4 + 4 + 2 * 8


def test_plain_pages_copy_a_shared_last_page_once_a_sequence():
    m = pm.Pages(3, 4, 8, 16)
    assert m.append([20, 0, 0]) == (0, [])
    m.fork([0, 0], [1, 2])
    assert m.refs[:2] == [3, 3] and m.len == [20, 20, 20]
    lack, copies = m.append([1, 0, 12])
    assert lack == 0 and copies == [(1, 2, 4), (1, 3, 4)]
    assert m.rows == [[0, 2], [0, 1], [0, 3]] and m.refs[:5] == [3, 1, 1, 1, 0]
    m.free([1], [0])
    assert m.refs[:5] == [2, 0, 1, 1, 0] and m.compact() == ([0, -1, 2, 1, -1, -1, -1, -1], 3)


def test_plain_attention_of_nothing_and_of_a_position_named_twice():
    q, k, v = torch.randn(2, 2, 8), torch.randn(3, 1, 8), torch.randn(3, 1, 8)
    o, lse, _ = pm.attention(q, k.double(), v.double(), None, torch.tensor([[0, 0, 0], [0, 2, 1]]), 0.5)
    assert not o[0].any() and bool((lse[0] == -math.inf).all())
    s = (q[1].double() @ k[:, 0].double().T) * 0.5
    w = torch.stack([2 * s[:, 1].exp(), s[:, 2].exp()], 1)
    assert torch.allclose(o[1], (w @ v[1:, 0].double()) / w.sum(1, keepdim=True))
    assert torch.allclose(lse[1], w.sum(1).log())
