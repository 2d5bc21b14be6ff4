"""Data that attention over the paged cache cannot know before it reads it:
what it then leaves alone."""
import pytest
import torch

from test_gpu_cache import DEV, agree, expected, fill, i32
from top_token_selection_b200 import pivot as pv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,Hq,topk", [(2, 4, 0), (30, 8, 0), (300, 8, 0), (3, 4, 40), (3, 80, 40)])
@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_that_descend(fp8, n, Hq, topk):
    # the same rows claimed by every other sequence, many times what the
    # workspace counts on: nothing is written past it, and (paged) no row
    B, length = 65, 320
    c, gen = fill([length] * B, 16, 1, 64, fp8, seed=17)
    q = torch.randn(n, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
    cu = i32([n * (b % 2) for b in range(B + 1)])
    assert int(cu[B]) == n
    idx = torch.randint(0, 300, (n, max(topk, 1)), generator=gen, dtype=torch.int32).to(DEV)
    o = torch.full_like(q, 3.5)
    call = pv.PivotAttend(Hq, n, n, q.data_ptr(), cu.data_ptr(), 0.125, 0, idx.data_ptr() if topk else None,
                          topk, o.data_ptr(), None)
    size = (pv.pivot_selected_attention_workspace_size if topk else
            pv.pivot_paged_attention_workspace_size)(c.c, call)
    ws = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    if topk:
        pv.selected_attention(c.c, q, cu, n, idx, o=o, ws=ws[:size])
    else:
        pv.paged_attention(c.c, q, cu, n, o=o, ws=ws[:size])
    # a selected row goes by the sequence that the search for it ends at
    assert pv.device_error() == (0 if topk else 6)
    assert bool((ws[size:] == 0x5A).all())
    if not topk:
        assert bool((o == 3.5).all())
    # the next call is as ever
    agree(pv.paged_attention(c.c, q[:2], i32([0] + [2] * B), 2, with_lse=True),
          expected(c, q[:2], [2] + [0] * (B - 1), [length] * B))
