"""Attention over the paged cache where the size of a value, a scale or a score
is out of the ordinary: on both kernels, against 64 bits."""
import pytest
import torch

from test_gpu_cache import DEV, Cache, agree, expected, fill, i32, offsets
from top_token_selection_b200 import pivot as pv

pytestmark = pytest.mark.gpu

# sequences (over the same pages, with the same queries), new tokens, query
# heads (of one key head), selected positions (0: paged): the rows kernel with
# 16 and 32 rows a key, then the tensor-memory kernel with blocks of 128 rows,
# of 256 and selected.  One sequence's tiles are spread over all SMs; of many
# sequences one block runs whole rows.
FORMS = [(1, 1, 4, 0), (300, 1, 4, 0), (1, 3, 10, 0), (300, 3, 10, 0), (300, 1, 4, 1), (1, 2, 4, 1),
         (1, 40, 2, 0), (150, 40, 2, 0), (1, 70, 8, 0), (150, 100, 2, 0), (1, 2, 40, 1), (150, 1, 40, 1)]


def attend(c, q, B, length, picked, scale=None):
    """The call's result and what it is in 64 bits, for B sequences alike."""
    n, idx = q.shape[0], None
    table = c.table.repeat(B, 1)
    many = pv.make_cache(c.k, c.v, table, c.len.repeat(B), c.refs, c.ks, c.vs)
    qs = q.repeat(B, 1, 1)
    if picked is None:
        got = pv.paged_attention(many, qs, offsets([n] * B), n, scale=scale, with_lse=True)
    else:
        idx = picked.to(torch.int32).to(DEV).repeat(n, 1).contiguous()
        got = pv.selected_attention(many, qs, offsets([n] * B), n, idx.repeat(B, 1), scale=scale, with_lse=True)
    torch.cuda.synchronize()
    want = expected(c, q, [n], [length], idx=idx, scale=scale)
    return got, tuple(x.repeat(B, *[1] * (x.dim() - 1)) for x in want)


# A token without values that holds most of the weight, as an attention sink
# or a padded token does: the append stores scale 1 for it.  The others' sum is
# held to the same part of sum p |v| as ever (its own |v| is 0).
@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length,empty,zero_key,size", [
    (3000, [0], False, 1.0), (3000, [0], True, 0.1), (3000, [1500], False, 1e-3),
    (2600, list(range(300)), True, 1e-2), (900, [0, 5, 899 - 80], False, 1e-4), (30000, [0], False, 1.0)])
def test_a_heavy_token_without_values(D, B, n, Hq, topk, length, empty, zero_key, size):
    gen = torch.Generator().manual_seed(length + D)
    c = Cache(1, -(-length // 64), -(-length // 64), 64, 1, D, True)
    u = torch.randn(D, generator=gen)
    u /= u.norm()
    k = torch.randn(length, 1, D, generator=gen)
    v = torch.randn(length, 1, D, generator=gen) * size
    # the empty tokens' scores lie `lift` above the others', so that each holds
    # about 0.9 / len(empty) of the weight
    lift = float(torch.tensor(10.0 * length / len(empty)).log()) * D ** 0.5 / 8
    q = (8 * u + 0.3 * torch.randn(n, Hq, D, generator=gen)).to(torch.bfloat16).to(DEV)
    along = (k @ u)[..., None] * u
    k = k - along + 0.02 * along / D ** 0.5
    if zero_key:
        k = k - lift * u
    k[empty] = 0.0 if zero_key else lift * u
    v[empty] = 0.0
    k, v = (x.to(torch.bfloat16).to(DEV) for x in (k, v))
    assert int(pv.cache_append(c.c, k, v, i32([0, length]), length)) == 0
    assert float(c.vs[c.table[0, empty[0] // 64], empty[0] % 64]) == 1.0
    picked = torch.randperm(length - n, generator=gen)[: length * 3 // 4] if topk else None
    if topk:
        picked = torch.unique(torch.cat([picked, torch.tensor(empty)]))
        picked = picked[torch.randperm(len(picked), generator=gen)]
    got, want = attend(c, q, B, length, picked)
    # most of the weight is the empty tokens': the others' sum is small
    assert float((want[2].mean() / (v.float().abs().mean()))) < 0.4
    agree(got, want)


@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_very_different_tokens(D, B, n, Hq, topk):
    # one token's values are 2^10 of the others', and its weight small: neither
    # takes bits from the other
    gen = torch.Generator().manual_seed(20)
    c, _ = fill([4000], 32, 1, D, True, seed=20)
    page, slot = int(c.table[0, 60]), 7
    c.vs[page, slot] *= 1024.0
    c.ks[page, slot] *= 2.0 ** -6
    q = torch.randn(n, Hq, D, generator=gen).to(torch.bfloat16).to(DEV)
    picked = torch.randperm(4000 - n, generator=gen)[:3000] if topk else None
    agree(*attend(c, q, B, 4000, picked))


# Scores that are all (nearly) 0: a mean of the values.
@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["queries", "keys", "scale", "all"])
def test_scores_of_nothing_beside_masked_keys(what, fp8, B, n, Hq, topk):
    c, gen = fill([700], 16, 1, 128, fp8, seed=21)
    q = torch.randn(n, Hq, 128, generator=gen).to(torch.bfloat16).to(DEV)
    if what in ("queries", "all"):
        q[:, 1::2] = 0.0
        q[0] = 0.0
    if fp8 and what in ("keys", "all"):
        c.ks *= 2.0 ** -30
    picked = None
    if topk:
        picked = torch.cat([torch.arange(300), torch.full((50,), -1), torch.tensor([699, 2 ** 31 - 1])])
    agree(*attend(c, q, B, 700, picked, scale={"scale": 1e-8, "all": 1e-30}.get(what)))


@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [20, -20, 60])
def test_large_scores_beside_large_value_scales(power, D, B, n, Hq, topk):
    # scores of 1e28 choose one key: the output is its values, to the bf16
    # rounding of o (2^-9) and one of a weight of 1 in f16 with the scale's (2^-11 twice)
    c, gen = fill([400], 32, 1, D, True, seed=22)
    q = torch.randn(n, Hq, D, generator=gen)
    q[:, 1::2] *= 1e28
    q = q.to(torch.bfloat16).to(DEV)
    c.vs *= 2.0 ** power
    picked = torch.randperm(400 - n, generator=gen)[:300] if topk else None
    got, want = attend(c, q, B, 400, picked)
    assert pv.device_error() == 0
    assert bool(torch.isfinite(got[0].float()).all()) and bool(torch.isfinite(got[1]).all())
    big = (got[0].double() - want[0]).abs()[:, 1::2] / want[2][:, 1::2]
    assert float(big.max()) < 2 ** -8 + 2 ** -10
    assert float((got[1].double() / want[1] - 1).abs()[:, 1::2].max()) < 2 ** -16
    agree(tuple(x[:, ::2] for x in got), tuple(x[:, ::2] for x in want))


@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
@pytest.mark.parametrize("lift", [20.0, 43.5, 100.0])
@pytest.mark.parametrize("size", [1e20, 1e34, 1e-30])
def test_large_values_under_a_late_large_score(size, lift, B, n, Hq, topk):
    # bf16 values far up and down the type's range; the keys at the end
    # outweigh the first ones by e^lift
    length, D = 1500, 64
    c, gen = fill([length], 64, 1, D, False, seed=23)
    u = torch.randn(D, generator=gen)
    u /= u.norm()
    q = (8 * u).repeat(n, Hq, 1).to(torch.bfloat16).to(DEV)
    k = 0.05 * torch.randn(length, D, generator=gen)
    k[1300:length - n] += lift * u
    v = torch.randn(length, D, generator=gen) * size
    t = torch.arange(length, device=DEV)
    page, slot = c.table[0].long()[t // 64], t % 64
    c.k[page, slot, 0], c.v[page, slot, 0] = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    picked = torch.arange(length - n) if topk else None
    got, want = attend(c, q, B, length, picked)
    assert bool(torch.isfinite(got[0].float()).all())
    # a score's fp32 error is up to D * 2^-24 of its size, 100: 2^-11; weights and
    # outputs round to bf16, off by at most 2^-8 each
    assert float(((got[0].double() - want[0]).abs() / want[2]).max()) < 2 * 2.0 ** -8 + 2.0 ** -10
    assert float((got[1].double() - want[1]).abs().max()) < 5e-4
    assert pv.device_error() == 0


@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
def test_one_scale_for_all_tokens(B, n, Hq, topk):
    # a cache with scale 1 throughout, some of its tokens zero
    gen = torch.Generator().manual_seed(24)
    c, _ = fill([3000], 64, 1, 128, True, seed=24)
    c.ks.fill_(0.25)
    for plane in (c.k, c.v):
        plane.copy_((2 * torch.randn(plane.shape, generator=gen)).to(plane.dtype))
    empty = torch.randperm(3000, generator=gen)[:200].to(DEV)
    page, slot = c.table[0].long()[empty // 64], empty % 64
    c.v.view(torch.uint8)[page, slot] = 0
    c.vs.fill_(1.0)
    q = torch.randn(n, Hq, 128, generator=gen).to(torch.bfloat16).to(DEV)
    picked = torch.randperm(3000 - n, generator=gen)[:2000] if topk else None
    agree(*attend(c, q, B, 3000, picked))


@pytest.mark.parametrize("B,n,Hq,topk", FORMS)
def test_large_scores_over_values_of_nothing(B, n, Hq, topk):
    # no value anywhere, by scales of 0 and by codes: o is 0, the log-sum-exp as ever
    c, gen = fill([500], 32, 1, 64, True, seed=25)
    c.vs[c.table[0, :8].long()] = 0.0
    for page in c.table[0, 8:16].long():
        c.v.view(torch.uint8)[page] = 0
    q = torch.randn(n, Hq, 64, generator=gen)
    q[:, 1::2] *= 1e28
    q = q.to(torch.bfloat16).to(DEV)
    picked = torch.randperm(500 - n, generator=gen)[:300] if topk else None
    (o, lse), want = attend(c, q, B, 500, picked)
    assert pv.device_error() == 0 and not bool(o.any())
    assert float((lse.double() / want[1] - 1).abs()[:, 1::2].max()) < 2 ** -16
    assert float((lse.double() - want[1]).abs()[:, ::2].max()) < 5e-4
