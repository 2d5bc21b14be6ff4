"""Every key counts once: a row whose score is large at one position alone
returns that position's value, and its log-sum-exp is the one score.  A key
that is lost, read twice or taken from another row at the edge of a page, a
key tile, a ring slot or a CTA's run shows as another value or as log 2."""
import pytest
import torch

from test_gpu_cache import DEV, fill, i32, offsets
from top_token_selection_b200 import pivot as pv
import paged_model as pm

pytestmark = pytest.mark.gpu


# new tokens a sequence, query heads a key head, head dim, page, length, selected
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,G,D,page,length,select", [
    (1, 4, 128, 16, 2100, False), (2, 16, 64, 64, 9000, False), (1, 1, 64, 256, 1000, False),
    (2, 16, 128, 64, 9000, False), (40, 2, 128, 64, 2100, False), (150, 4, 64, 16, 9000, False),
    (150, 4, 128, 16, 9000, False), (300, 2, 128, 128, 3000, False),
    (2, 8, 128, 64, 1500, True), (4, 40, 64, 16, 1500, True), (4, 64, 128, 128, 2100, True)])
def test_every_key_counts_once(n, G, D, page, length, select, fp8):
    # one text, seen by as many sequences as it takes to ask for each position
    c, gen = fill([length], page, 1, D, fp8, seed=30 + n)
    k = pm.tokens(c.k, c.ks, c.table, 0, length)[:, 0]
    v = pm.tokens(c.v, c.vs, c.table, 0, length)[:, 0]
    seen = length - n + 1                                  # by every new token
    B = -(-seen // (n * G))
    goal = torch.arange(B * n * G, device=DEV) % seen
    goal = goal[torch.randperm(len(goal), generator=gen).to(DEV)]
    # a score of 60 at the goal; the others' keys are random directions, their
    # scores spread by 60 / sqrt(D) (D = 128: 5.3), and by three times that for
    # the one in fifty that is three times as long.  At D = 64 those come near
    # 60 now and then: the bounds below hold all others' weight against a row
    q = (k[goal] * (60.0 / (k[goal] ** 2).sum(-1, keepdim=True))).to(torch.bfloat16)
    s = q.double() @ k.T
    s_goal = s.gather(1, goal[:, None])[:, 0]
    pos = length - n + torch.arange(B * n * G, device=DEV) // G % n
    s.masked_fill_(torch.arange(length, device=DEV)[None] > pos[:, None], -torch.inf)
    lse = torch.logsumexp(s, 1)
    rest = -torch.expm1(s_goal - lse)                      # the others' weight
    assert D == 64 or float(rest.median()) < 1e-6
    many = pv.make_cache(c.k, c.v, c.table.repeat(B, 1), c.len.repeat(B), c.refs, c.ks, c.vs)
    q = q.view(B * n, G, D)
    if select:
        topk = seen + 37
        idx = torch.full((B * n, topk), -1, dtype=torch.int32)
        for r in range(B * n):
            idx[r, torch.randperm(topk, generator=gen)[:seen]] = torch.arange(seen, dtype=torch.int32)
        s.masked_fill_(torch.arange(length, device=DEV)[None] >= seen, -torch.inf)
        lse = torch.logsumexp(s, 1)
        rest = -torch.expm1(s_goal - lse)
        o, got = pv.selected_attention(many, q, offsets([n] * B), n, idx.to(DEV), scale=1.0, with_lse=True)
    else:
        o, got = pv.paged_attention(many, q, offsets([n] * B), n, scale=1.0, with_lse=True)
    assert pv.device_error() == 0
    # fp32 products of D terms of sizes that add up to at most 60 sqrt(D): 2^-11
    # (D * 2^-24 * 60 * sqrt(D) at D = 128: 0.005 at the very most)
    assert float((got.view(-1).double() - lse).abs().max()) < 0.006
    # bf16 rounding of the weight and of the output, and the others' values (up
    # to 6, and as far from the goal's)
    off = (o.view(-1, D).double() - v[goal]).abs()
    bound = 2 * 2.0 ** -8 * v[goal].abs() + 2 ** -10 * 2 + 12.0 * rest[:, None] * 1.01
    assert bool((off <= bound).all()), float((off - bound).max())
