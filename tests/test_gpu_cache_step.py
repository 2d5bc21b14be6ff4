"""The paged cache's calls as a program uses them together: sparse decode
steps over forked, cut and compacted sequences, other streams, captured
graphs, and data that the kernels themselves refuse."""
import paged_model as pm
import pytest
import torch

from test_gpu_cache import DEV, Cache, agree, expected, fill, i32, offsets
from top_token_selection_b200 import pivot as pv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [pv.DENSE, pv.REFINE])
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_decode_steps_over_forks_cuts_and_compaction(fp8, mode):
    B, Gm, Hq, Hkv, D, H, C, topk, maxlen = 4, 2, 16, 2, 64, 4, 256, 96, 512
    gen = torch.Generator().manual_seed(11 + fp8)
    c = Cache(B, maxlen // 16, 80, 16, Hkv, D, fp8)
    keys = torch.zeros(B, maxlen, 32, device=DEV)              # the indexer's keys, fp32
    c.append([200, 333, 0, 0], gen)
    keys[:2] = torch.randint(-3, 4, (2, maxlen, 32), generator=gen).float().to(DEV)
    # two branches of sequence 1, their indexer rows copied along
    pv.pages_fork(c.c, i32([1, 1]), i32([2, 3]))
    pv.pages_copy(keys, keys, i32([1, 1]), i32([2, 3]))
    c.model.fork([1, 1], [2, 3])
    c.text[2], c.text[3] = list(c.text[1]), list(c.text[1])
    for step in range(4):
        lens = c.model.len
        for b in range(B):
            keys[b, lens[b]:lens[b] + Gm] = torch.randint(-3, 4, (Gm, 32), generator=gen).float().to(DEV)
        iq = torch.randint(-3, 4, (B, Gm, H, 32), generator=gen).float().to(DEV)
        w = torch.randint(1, 5, (B, Gm, H), generator=gen).float().to(DEV)
        q = torch.randn(B, Gm, Hq, D, generator=gen).to(torch.bfloat16)
        k, v = (torch.randn(B, Gm, Hkv, D, generator=gen).to(torch.bfloat16) for _ in range(2))
        batch = pv.make_decode(iq, None, w, keys, None, c.len)
        o, lse, idx, lack = pv.decode_attention(batch, c.c, q.to(DEV), k.to(DEV), v.to(DEV), mode, C, topk,
                                                with_lse=True)
        c.model.append([Gm] * B)
        for b in range(B):
            c.text[b] = [torch.cat([a, x[b]]) for a, x in zip(c.text[b], (k, v))]
        assert int(lack) == 0
        c.check()
        assert torch.equal(idx, pv.decode(batch, mode, C, topk)[0])
        flat = idx.view(B * Gm, topk)
        assert bool((flat >= 0).any(1).all())
        qf = q.reshape(B * Gm, Hq, D).to(DEV)
        agree((o.view(B * Gm, Hq, D), lse.view(B * Gm, Hq)),
              expected(c, qf, [Gm] * B, c.model.len, idx=flat))
        # the dense form of the same step
        agree(pv.paged_attention(c.c, qf, offsets([Gm] * B), Gm, with_lse=True),
              expected(c, qf, [Gm] * B, c.model.len))
        if step == 1:                                  # a draft token is rejected, a branch ends
            seqs, keep = [0, 2], [c.model.len[0] - 1, 0]
            pv.pages_free(c.c, i32(seqs), i32(keep))
            c.model.free(seqs, keep)
            for b, n in zip(seqs, keep):
                c.text[b] = [x[:n] for x in c.text[b]]
            pv.pages_compact(c.c)
            c.model.compact()
            c.check()
            pv.pages_fork(c.c, i32([3]), i32([2]))     # the other branch goes on twice
            pv.pages_copy(keys, keys, i32([3]), i32([2]))
            c.model.fork([3], [2])
            c.text[2] = list(c.text[3])


def run_step(c, q, new, cu, n, base, o, ws):
    pv.pages_free(c.c, i32(range(c.B)) if not isinstance(base, tuple) else base[0],
                  base if not isinstance(base, tuple) else base[1])
    lack = pv.cache_append(c.c, new, new, cu, n, ws=ws[0])
    return lack, pv.paged_attention(c.c, q, cu, n, with_lse=True, o=o, ws=ws[1])[1]


@pytest.mark.parametrize("n", [1, 40])
def test_captured_steps_sharing_a_workspace_replay(n):
    # eager, then two graphs over one workspace, replayed in turn with other inputs
    B, Hq, Hkv, D = 3, 8, 2, 64
    c, gen = fill([100, 47, 300], 16, Hkv, D, False, seed=3, spare=40)
    c.refs.zero_()
    c.refs[c.table[c.table >= 0].long()] = 1
    wide = torch.full((B, 64), -1, dtype=torch.int32, device=DEV)
    wide[:, : c.table.shape[1]] = c.table
    c.table = wide
    c.c = pv.make_cache(c.k, c.v, c.table, c.len, c.refs)
    base = (i32(range(B)), c.len.clone())
    cu = offsets([n] * B)
    qs = [torch.randn(B * n, Hq, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    new = torch.randn(B * n, Hkv, D, generator=gen).to(torch.bfloat16).to(DEV)
    ws = [torch.empty(1 << 20, dtype=torch.uint8, device=DEV), torch.empty(1 << 27, dtype=torch.uint8, device=DEV)]
    want = []
    for q in qs:
        o = torch.zeros_like(q)
        lack, lse = run_step(c, q, new, cu, n, base, o, ws)
        assert int(lack) == 0
        want.append((o, lse.clone()))
    q, outs, graphs = torch.zeros_like(qs[0]), [], []
    torch.cuda.synchronize()
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), torch.zeros_like(q)
        with torch.cuda.graph(g):
            lack, lse = run_step(c, q, new, cu, n, base, o, ws)
        outs.append((o, lse, lack))
        graphs.append(g)
    for i, q_i in enumerate([qs[0], qs[1], qs[0]]):
        q.copy_(q_i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        o, lse, lack = outs[i % 2]
        wo, wl = want[0 if i != 1 else 1]
        assert int(lack) == 0 and torch.equal(o, wo) and torch.equal(lse, wl)
    assert pv.device_error() == 0


@pytest.mark.parametrize("n,Hq", [(2, 8), (70, 16)])
def test_other_streams_and_repeated_calls_give_the_same_bits(n, Hq):
    c, gen = fill([900, 300 + n], 32, 2, 128, True, seed=4)
    q = torch.randn(2 * n, Hq, 128, generator=gen).to(torch.bfloat16).to(DEV)
    cu = offsets([n, n])
    o, lse = pv.paged_attention(c.c, q, cu, n, with_lse=True)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [pv.paged_attention(c.c, q, cu, n, with_lse=True, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert pv.device_error() == 0
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("n,Hq,topk", [(2, 4, 0), (50, 8, 0), (3, 4, 40), (3, 80, 40)])
def test_rows_behind_the_last_sequence_stay(n, Hq, topk):
    c, gen = fill([60, 90], 16, 1, 64, False, seed=5)
    total = 2 * n + 7
    q = torch.randn(total, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
    o = torch.full_like(q, 3.5)
    cu = offsets([n, n])
    if topk:
        idx = torch.randint(0, 55, (total, topk), generator=gen, dtype=torch.int32).to(DEV)
        pv.selected_attention(c.c, q, cu, n, idx, o=o)
        want = expected(c, q, [n, n], [60, 90], idx=idx)[0]
    else:
        pv.paged_attention(c.c, q, cu, n, o=o)
        want = expected(c, q, [n, n], [60, 90])[0]
    torch.cuda.synchronize()
    assert pv.device_error() == 0 and bool((o[2 * n:] == 3.5).all())
    assert float((o[: 2 * n].double() - want).abs().max()) < 0.1


@pytest.mark.parametrize("n,Hq,topk", [(2, 4, 0), (50, 8, 0), (3, 4, 40), (3, 80, 40)])
@pytest.mark.parametrize("bad", ["short", "long", "offsets"])
def test_a_bad_sequence_is_refused_alone(n, Hq, topk, bad):
    c, gen = fill([200, 150, 170], 16, 1, 64, False, seed=6)
    q = torch.randn(3 * n, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
    o = torch.full_like(q, 3.5)
    cu = offsets([n, n, n])
    idx = torch.randint(0, 99, (3 * n, topk), generator=gen, dtype=torch.int32).to(DEV) if topk else None
    want = expected(c, q, [n] * 3, [200, 150, 170], idx=idx)[0]
    if bad == "short":
        c.len[1] = n - 1                 # fewer tokens than new ones
    elif bad == "long":
        c.len[1] = c.table.shape[1] * 16 + 1
    most = n - 1 if bad == "offsets" else n              # max_new below every count
    if topk:
        pv.selected_attention(c.c, q, cu, most, idx, o=o)
    else:
        pv.paged_attention(c.c, q, cu, most, o=o)
    assert pv.device_error() == 6
    if bad == "offsets":
        assert bool((o == 3.5).all())
        return
    assert bool((o[n:2 * n] == 3.5).all())
    for a in (0, 2 * n):
        assert float((o[a:a + n].double() - want[a:a + n]).abs().max()) < 0.1


@pytest.mark.parametrize("n,Hq,topk", [(2, 4, 0), (50, 8, 0), (3, 4, 40), (3, 80, 40)])
@pytest.mark.parametrize("fp8", [False, True])
def test_tokens_of_a_bad_page_count_as_masked(n, Hq, topk, fp8):
    c, gen = fill([200], 16, 1, 64, fp8, seed=7)
    q = torch.randn(n, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
    cu = offsets([n])
    lost = torch.arange(200, device=DEV).div(16, rounding_mode="floor") == 3
    if topk:
        idx = torch.arange(30, 30 + topk, dtype=torch.int32, device=DEV).repeat(n, 1)
        want = expected(c, q, [n], [200], idx=torch.where(lost[idx.long()], -1, idx))
    else:
        pos = torch.arange(200 - n, 200, device=DEV)
        see = (torch.arange(200, device=DEV)[None] <= pos[:, None]) & ~lost
        want = pm.attention(q, pm.tokens(c.k, c.ks, c.table, 0, 200), pm.tokens(c.v, c.vs, c.table, 0, 200),
                            None, see, 0.125)
    c.table[0, 3] = c.k.shape[0]
    got = (pv.selected_attention(c.c, q, cu, n, idx, with_lse=True) if topk else
           pv.paged_attention(c.c, q, cu, n, with_lse=True))
    assert pv.device_error() == 6
    agree(got, want)


def test_pages_before_every_window_may_be_gone():
    for n, Hq in ((1, 4), (40, 8)):
        c, gen = fill([500], 16, 1, 64, False, seed=8)
        q = torch.randn(n, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
        want = expected(c, q, [n], [500], window=100)
        c.table[0, : (500 - n - 99) // 16] = -1
        agree(pv.paged_attention(c.c, q, offsets([n]), n, window=100, with_lse=True), want)


def test_scales_far_apart_and_of_zero():
    # tokens of sizes from 2^-12 to 1 and of nothing at all, in one tile
    c, gen = fill([300], 16, 2, 64, True, seed=9)
    live = c.table[0, : 19].long()
    f = 2.0 ** -torch.randint(0, 13, (19, 16), generator=gen).float()
    f[5, 3] = 0.0
    c.ks[live] *= f.to(DEV)
    c.vs[live] *= f.to(DEV).flip(0)
    for n in (1, 60):
        q = torch.randn(n, 8, 64, generator=gen).to(torch.bfloat16).to(DEV)
        agree(pv.paged_attention(c.c, q, offsets([n]), n, with_lse=True), expected(c, q, [n], [300]))


def test_large_queries_and_scale():
    c, gen = fill([700], 16, 1, 128, True, seed=10)
    for n, Hq in ((1, 4), (40, 8)):
        q = torch.randn(n, Hq, 128, generator=gen)
        q[:, 0] *= 1e20
        q[:, 1] *= 1e-20
        q[0, 2] = 0.0
        q = q.to(torch.bfloat16).to(DEV)
        o, lse = pv.paged_attention(c.c, q, offsets([n]), n, scale=0.05, with_lse=True)
        want = expected(c, q, [n], [700], scale=0.05)
        torch.cuda.synchronize()
        assert pv.device_error() == 0
        # the first head's weights are 0 or 1; the others as ever
        agree((o[:, 1:], lse[:, 1:]), tuple(x[:, 1:] for x in want))
        assert bool(torch.isfinite(o[:, 0].float()).all())
        assert float(((o[:, 0].double() - want[0][:, 0]).abs() / want[2][:, 0]).max()) < 2 ** -7


@pytest.mark.parametrize("n,Hq,topk", [(1, 4, 0), (40, 8, 0), (140, 8, 0), (2, 4, 60), (2, 40, 60)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_every_size(D, fp8, n, Hq, topk):
    # scores of up to about 1000 and 1e28: fp32 products of D terms are off by
    # about 2^-22 of the sum of their sizes (0.05 * 300 * 128 * 0.64: 3e-4
    # twice), weights by 2^-8, the output by 2^-8 again
    c, gen = fill([400], 32, 1, D, fp8, seed=12)
    q = torch.randn(n, Hq, D, generator=gen)
    q[:, 0] *= 300.0
    q[:, 1] *= 1e28
    q = q.to(torch.bfloat16).to(DEV)
    cu = offsets([n])
    if topk:
        idx = torch.randint(0, 390, (n, topk), generator=gen, dtype=torch.int32).to(DEV)
        got = pv.selected_attention(c.c, q, cu, n, idx, scale=0.05, with_lse=True)
        want = expected(c, q, [n], [400], idx=idx, scale=0.05)
    else:
        got = pv.paged_attention(c.c, q, cu, n, scale=0.05, with_lse=True)
        want = expected(c, q, [n], [400], scale=0.05)
    torch.cuda.synchronize()
    assert pv.device_error() == 0
    agree(tuple(x[:, 2:] for x in got), tuple(x[:, 2:] for x in want))
    assert float(((got[0].double() - want[0]).abs()[:, :2] / want[2][:, :2]).max()) < 2 ** -6
    assert float((got[1].double() / want[1] - 1).abs()[:, :2].max()) < 2 ** -16


@pytest.mark.parametrize("length", [-100, -1, 14 * 16 + 1, 2 ** 31 - 1])
def test_lengths_out_of_range_change_nothing(length):
    c, _ = fill([200, 150, 170], 16, 1, 64, False, seed=13)
    assert c.table.shape[1] == 14
    c.refs[c.table[c.table >= 0].long()] = 1
    c.len[1] = length
    before = [t.clone() for t in (c.table, c.len, c.refs)]
    pv.pages_free(c.c, i32([0, 1]), i32([3, 0]))
    assert pv.device_error() == 6
    pv.pages_fork(c.c, i32([1, 0]), i32([0, 2]))
    assert pv.device_error() == 6
    for a, b in zip(before, (c.table, c.len, c.refs)):
        assert torch.equal(a, b)
    pv.pages_fork(c.c, i32([0]), i32([1]))           # a sequence is mended by becoming another
    assert pv.device_error() == 0 and int(c.len[1]) == 200


@pytest.mark.parametrize("n,Hq,topk", [(2, 4, 0), (70, 8, 0), (3, 4, 150), (3, 80, 150)])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_past_4_gib_of_a_plane(fp8, n, Hq, topk):
    # the same tokens at the pool's beginning and behind 2^32 bytes of it
    # give the same bits
    Hkv, D, page = (4, 128, 64) if Hq < 80 else (1, 128, 64)
    Hq *= Hkv
    small, gen = fill([300], page, Hkv, D, fp8, seed=14)
    pages = (2 ** 32 + 2 ** 27) // (page * Hkv * D * (1 if fp8 else 2))
    k, v = (torch.empty(pages, *small.k.shape[1:], dtype=small.k.dtype, device=DEV) for _ in range(2))
    ks, vs = (torch.empty(pages, page, device=DEV) for _ in range(2)) if fp8 else (None, None)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    far = torch.arange(pages - 5, pages, dtype=torch.int32, device=DEV)
    near = small.table[0, :5].contiguous()
    for a, b in ((small.k, k), (small.v, v)):
        pv.pages_copy(a, b, near, far)
        if fp8:
            assert torch.equal(a.view(torch.uint8)[near.long()], b[-5:].view(torch.uint8))
    if fp8:
        ks[-5:], vs[-5:] = small.ks[near.long()], small.vs[near.long()]
    refs[-5:] = 1
    c = pv.make_cache(k, v, far[None].contiguous(), small.len.clone(), refs, ks, vs)
    q = torch.randn(n, Hq, D, generator=gen).to(torch.bfloat16).to(DEV)
    cu = offsets([n])
    if topk:
        idx = torch.randint(-1, 290, (n, topk), generator=gen, dtype=torch.int32).to(DEV)
        def run(x): return pv.selected_attention(x, q, cu, n, idx, with_lse=True)
    else:
        def run(x): return pv.paged_attention(x, q, cu, n, with_lse=True)
    want, got = run(small.c), run(c)
    remap, used = pv.pages_compact(c)
    after = run(c)
    assert pv.device_error() == 0 and int(used) == 5
    assert torch.equal(remap[-5:].cpu(), torch.arange(5, dtype=torch.int32))
    for a, b, d in zip(want, got, after):
        assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("G", [1, 4, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_many_short_sequences(fp8, G):
    B = 2500
    gen = torch.Generator().manual_seed(15)
    c = Cache(B, 2, 2 * B, 16, 1, 64, fp8)
    n0 = torch.randint(0, 25, (B,), generator=gen).tolist()
    n1 = [int(x) if int(x) else 0 for x in torch.randint(0, 4, (B,), generator=gen)]
    c.append(n0, gen)
    c.append(n1, gen)
    c.check()
    total = sum(n1)
    q = torch.randn(total, G, 64, generator=gen).to(torch.bfloat16).to(DEV)
    agree(pv.paged_attention(c.c, q, offsets(n1), 3, with_lse=True), expected(c, q, n1, c.model.len))
    idx = torch.randint(-1, 30, (total, 20), generator=gen, dtype=torch.int32).to(DEV)
    agree(pv.selected_attention(c.c, q, offsets(n1), 3, idx, with_lse=True),
          expected(c, q, n1, c.model.len, idx=idx))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq", [4, 40])
def test_a_bad_own_page_beside_garbage(Hq, fp8):
    # the first row of the pool is no number; the first of three new tokens is
    # on a good page, the others' own is gone: they are right or unwritten
    c, gen = fill([194], 16, 1, 64, fp8, seed=16)
    assert not bool((c.table == 0).any())
    q = torch.randn(3, Hq, 64, generator=gen).to(torch.bfloat16).to(DEV)
    idx = torch.full((3, 90), -1, dtype=torch.int32, device=DEV)
    idx[:, :50] = torch.arange(30, 80, device=DEV)
    ow, lw, size = expected(c, q, [3], [194], idx=idx)
    c.table[0, 12] = -1
    for plane in (c.k, c.v):
        plane.view(torch.uint8)[0] = 0x7F if fp8 else 0xFF
    o = torch.full_like(q, 3.5)
    _, lse = pv.selected_attention(c.c, q, offsets([3]), 3, idx, o=o, with_lse=True)
    assert pv.device_error() == (0 if Hq == 4 else 6)
    agree((o[:1], lse[:1]), (ow[:1], lw[:1], size[:1]))
    if Hq == 4:
        agree((o, lse), (ow, lw, size))
    else:
        assert bool((o[1:] == 3.5).all())
