"""The bounds-checking build (libpivot_debug.so) over the paged cache's calls:
its checks hold, and what it returns is what the normal build returns."""
import random

import pytest
import torch

from test_gpu_cache import DEV, fill, i32, offsets
from top_token_selection_b200 import build as libbuild
from top_token_selection_b200 import pivot as pv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def builds():
    """The normal library and the checking one, as the binding loads them."""
    normal = pv.load()
    path = libbuild.build(debug=True)
    pv._lib = None
    checking = pv.load(path)
    pv._lib = normal
    yield normal, checking
    pv._lib = normal


def steps(fp8, seed):
    """State and outputs of a run of page calls and both kinds of attention."""
    r = random.Random(seed)
    c, gen = fill([700, 0, 64, 333], 16, 2, 64, fp8, seed=seed, spare=60)
    table = torch.full((4, 80), -1, dtype=torch.int32, device=DEV)
    table[:, : c.table.shape[1]] = c.table
    refs = torch.zeros_like(c.refs)
    refs[table[table >= 0].long()] = 1
    cache = pv.make_cache(c.k, c.v, table, c.len, refs, c.ks, c.vs)
    out = []
    pv.pages_fork(cache, i32([0, 3]), i32([1, 2]))
    for n, Hq, topk in ((1, 8, 0), (40, 8, 0), (90, 12, 0), (2, 8, 50), (2, 80, 300)):
        counts = [n, n, 0, r.randrange(1, n + 1)]
        new = torch.randn(sum(counts), 2, 64, generator=gen).to(torch.bfloat16).to(DEV)
        lack = pv.cache_append(cache, new, new, offsets(counts), n)
        q = torch.randn(sum(counts), Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
        if topk:
            idx = torch.randint(-1, 300, (sum(counts), topk), generator=gen, dtype=torch.int32).to(DEV)
            out += pv.selected_attention(cache, q, offsets(counts), n, idx, with_lse=True)
        else:
            out += pv.paged_attention(cache, q, offsets(counts), n, window=r.choice([0, 100]), with_lse=True)
        out.append(lack)
        pv.pages_free(cache, i32([3]), i32([200]))
        out += pv.pages_compact(cache)
    assert pv.device_error() == 0
    live = refs > 0
    return out + [table, c.len, refs, c.k.view(torch.uint8)[live], c.v.view(torch.uint8)[live]]


@pytest.mark.parametrize("fp8", [False, True])
def test_the_checking_build_gives_the_same_bits(builds, fp8):
    want = steps(fp8, 40)
    pv._lib = builds[1]
    try:
        got = steps(fp8, 40)
    finally:
        pv._lib = builds[0]
    assert len(want) == len(got)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
