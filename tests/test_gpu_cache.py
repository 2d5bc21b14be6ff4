"""The paged cache on the GPU: page bookkeeping against a plain model, stored
tokens bit for bit, attention against 64 bits."""
import random

import paged_model as pm
import pytest
import torch

from top_token_selection_b200 import pivot as pv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return i32(cu)


class Cache:
    """A cache on the GPU beside its plain model; unwritten slots hold NaN."""

    def __init__(self, B, columns, pages, page, Hkv=2, D=64, fp8=False):
        shape = (pages, page, Hkv, D)
        if fp8:
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(pm.E4M3)
            self.v = self.k.view(torch.uint8).clone().view(pm.E4M3)
            self.ks = torch.full(shape[:2], float("nan"), device=DEV)
            self.vs = self.ks.clone()
        else:
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
            self.v, self.ks, self.vs = self.k.clone(), None, None
        self.table = torch.full((B, columns), -1, dtype=torch.int32, device=DEV)
        self.len = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.model = pm.Pages(B, columns, pages, page)
        self.c = pv.make_cache(self.k, self.v, self.table, self.len, self.refs, self.ks, self.vs)
        self.B, self.Hkv, self.D, self.fp8 = B, Hkv, D, fp8
        self.text = [[torch.zeros(0, Hkv, D, dtype=torch.bfloat16)] * 2 for _ in range(B)]

    def append(self, counts, gen):
        new = [torch.randn(sum(counts), self.Hkv, self.D, generator=gen).to(torch.bfloat16)
               for _ in range(2)]
        lack = pv.cache_append(self.c, new[0].to(DEV), new[1].to(DEV), offsets(counts),
                               max(1, max(counts)))
        want, _ = self.model.append(counts)
        assert int(lack) == want
        at = 0
        for b, n in enumerate(counts):
            if not want:
                self.text[b] = [torch.cat([old, x[at:at + n]]) for old, x in zip(self.text[b], new)]
            at += n

    def check(self):
        torch.cuda.synchronize()
        assert pv.device_error() == 0
        assert self.table.tolist() == self.model.table()
        assert self.len.tolist() == self.model.len
        assert self.refs.tolist() == self.model.refs
        for b in range(self.B):
            n = self.model.len[b]
            for plane, scale, text in ((self.k, self.ks, self.text[b][0]), (self.v, self.vs, self.text[b][1])):
                got = pm.tokens(plane, scale, self.table, b, n).cpu()
                want = text.double()
                if self.fp8 and n:
                    codes, sc = pm.quantise(text)
                    want = codes.double() * sc.double()[:, None, None]
                assert torch.equal(got, want), b


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,seed", [(16, 0), (32, 1), (64, 2), (256, 3)])
def test_a_long_run_of_page_calls_follows_the_model(page, seed, fp8):
    r, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    B, columns, pages = 7, 6, 24
    c = Cache(B, columns, pages, page, fp8=fp8)
    full = 0
    for step in range(40):
        what = r.choice(["append", "append", "append", "fork", "free", "compact"])
        if what == "append":
            room = [columns * page - n for n in c.model.len]
            counts = [r.choice([0, 0, 1, 2, page - 1, page, r.randrange(2 * page)]) for _ in range(B)]
            counts = [min(a, b) for a, b in zip(counts, room)]
            before = list(c.model.len)
            c.append(counts, gen)
            full += c.model.len == before and sum(counts) > 0
        elif what == "fork":
            n = r.randint(1, B)
            dst = r.sample(range(B), n)
            src = [r.randrange(B) for _ in range(n)]
            pv.pages_fork(c.c, i32(src), i32(dst))
            c.model.fork(src, dst)
            now = [c.text[s] for s in src]
            for d, t in zip(dst, now):
                c.text[d] = t
        elif what == "free":
            seqs = r.sample(range(B), r.randint(1, 3))
            keep = [r.choice([0, c.model.len[b], max(0, c.model.len[b] - r.randrange(1, 2 * page)),
                              c.model.len[b] + 9]) for b in seqs]
            pv.pages_free(c.c, i32(seqs), i32(keep))
            c.model.free(seqs, keep)
            for b, n in zip(seqs, keep):
                c.text[b] = [x[:n] for x in c.text[b]]
        else:
            remap, used = pv.pages_compact(c.c)
            want, u = c.model.compact()
            assert remap.tolist() == want and int(used) == u
        c.check()
    assert full or page != 16     # the small pages' run meets a full pool


def test_append_without_pages_changes_nothing():
    gen = torch.Generator().manual_seed(5)
    c = Cache(3, 4, 5, 16)
    c.append([20, 16, 1], gen)
    k = c.k.clone()
    c.append([13, 0, 16], gen)          # three pages wanted, one free
    c.check()
    assert torch.equal(k.view(torch.int16), c.k.view(torch.int16))
    c.append([12, 0, 15], gen)          # the open pages' slots are enough
    c.check()


def test_append_over_many_sequences_and_pages():
    # more sequences than threads of the planning block, and pages past its rounds
    gen = torch.Generator().manual_seed(6)
    B, pages = 2500, 40000
    c = Cache(B, 3, pages, 16, Hkv=1, D=16)
    r = random.Random(6)
    c.refs[:17000] = 1                  # somebody else's
    for p in range(17000):
        c.model.refs[p] = 1
    c.append([r.choice([0, 1, 16, 33]) for _ in range(B)], gen)
    torch.cuda.synchronize()
    assert c.table.tolist() == c.model.table() and c.refs.tolist() == c.model.refs
    assert c.len.tolist() == c.model.len


def test_e4m3_rows_of_zeros_and_rows_behind_the_last_sequence():
    c = Cache(2, 2, 4, 16, fp8=True)
    new = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    new[1] = 3.0e38
    new[3:] = 7.0                       # rows 3 and 4 belong to nobody
    lack = pv.cache_append(c.c, new, new, i32([0, 2, 3]), 2)
    assert int(lack) == 0 and c.len.tolist() == [2, 1]
    a = pm.tokens(c.k, c.ks, c.table, 0, 2)
    assert float(c.ks[c.table[0, 0], 0]) == 1.0 and float(a[0].abs().max()) == 0.0
    assert float(a[1].min()) == pytest.approx(3.0e38, rel=2 ** -4)
    assert c.k.view(torch.uint8)[c.table[0, 0], 2:].eq(0x7F).all()      # no other slot was written


@pytest.mark.parametrize("page_bytes", [16, 48, 4096, 16384, 100_000])
def test_copy_between_planes_and_bad_ids(page_bytes):
    src = torch.randint(0, 255, (9, page_bytes), dtype=torch.uint8, device=DEV)
    dst = torch.zeros(7, page_bytes, dtype=torch.uint8, device=DEV)
    pv.pages_copy(src, dst, i32([8, 0, 3, 3]), i32([0, 6, 2, 5]))
    torch.cuda.synchronize()
    assert torch.equal(dst[[0, 6, 2, 5]], src[[8, 0, 3, 3]]) and not dst[[1, 3, 4]].any()
    before = dst.clone()
    pv.pages_copy(src, dst, i32([9, -1, 1]), i32([0, 1, 7]))
    assert pv.device_error() == 6 and torch.equal(before, dst)
    pv.pages_copy(src, dst, i32([]), i32([]))
    assert pv.device_error() == 0


@pytest.mark.parametrize("bad", ["twice", "range", "offsets", "keep", "overflow"])
def test_bad_lists_change_nothing(bad):
    gen = torch.Generator().manual_seed(7)
    c = Cache(4, 3, 12, 16)
    c.append([17, 3, 0, 40], gen)
    if bad == "twice":
        pv.pages_fork(c.c, i32([0, 1]), i32([2, 2]))
        assert pv.device_error() == 6
        pv.pages_free(c.c, i32([1, 1]), i32([0, 1]))
    elif bad == "range":
        pv.pages_fork(c.c, i32([0, 4]), i32([2, 1]))
        assert pv.device_error() == 6
        pv.pages_free(c.c, i32([-1]), i32([0]))
    elif bad == "keep":
        pv.pages_free(c.c, i32([0, 3]), i32([3, -1]))
    else:
        new = torch.zeros(9, 2, 64, dtype=torch.bfloat16, device=DEV)
        cu = [0, 2, 1, 3, 4] if bad == "offsets" else [0, 0, 0, 0, 9]     # 40 + 9 > 3 pages
        assert int(pv.cache_append(c.c, new, new, i32(cu), 9)) == -1
    assert pv.device_error() == 6
    c.check()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

# |o - exact| in units of sum p |v| (which is at least |o|): a weight's
# rounding to bf16 is off by at most 2^-8 of it, and so is the rounding of o;
# the scores' fp32 sums of up to 128 products of a size below 30 in all (after
# the scale) are off by at most 128 * 2^-24 * 30 < 2^-12, e^x with them.
O_TOL = 2 * 2.0 ** -8 + 2.0 ** -10
# the same score error, and e^x and log of fp32
LSE_TOL = 5e-4


def fill(lens, page, Hkv, D, fp8, seed, spare=3):
    """A cache whose sequences hold `lens` tokens on shuffled pages, NaN
    everywhere else."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    c = Cache(len(lens), max(need + [1]) + 1, sum(need) + spare, page, Hkv, D, fp8)
    order = torch.randperm(sum(need) + spare, generator=gen).tolist()
    for b, n in enumerate(lens):
        row = [order.pop() for _ in range(need[b])]
        c.model.rows[b] = row
        if row:
            c.table[b, : len(row)] = i32(row)
        x = [torch.randn(n, Hkv, D, generator=gen) for _ in range(2)]
        x[0][torch.rand(n, generator=gen) < 0.02] *= 3.0
        t = torch.arange(n)
        at = torch.tensor(row, dtype=torch.int64)[t // page], t % page
        at = tuple(i.to(DEV) for i in at)
        for plane, scale, y in ((c.k, c.ks, x[0]), (c.v, c.vs, x[1])):
            if fp8:
                codes, sc = pm.quantise(y.to(DEV))
                plane.view(torch.uint8)[at] = codes.view(torch.uint8)
                scale[at] = sc
            else:
                plane[at] = y.to(torch.bfloat16).to(DEV)
    c.len.copy_(i32(lens))
    return c, gen


def expected(c, q, counts, lens, window=0, idx=None, scale=None):
    o, lse, size = [], [], []
    at = 0
    scale = c.D ** -0.5 if scale is None else scale
    for b, n in enumerate(counts):
        k = pm.tokens(c.k, c.ks, c.table, b, lens[b])
        v = pm.tokens(c.v, c.vs, c.table, b, lens[b])
        pos = torch.arange(lens[b] - n, lens[b], device=DEV)
        t = torch.arange(lens[b], device=DEV)
        if idx is None:
            see = t[None] <= pos[:, None]
            if window:
                see &= t[None] > pos[:, None] - window
        else:
            rows = idx[at:at + n].long()
            ok = (rows >= 0) & (rows <= pos[:, None])
            see = torch.zeros(n, lens[b] + 1, device=DEV)
            see.scatter_add_(1, torch.where(ok, rows, lens[b]), torch.ones_like(rows, dtype=torch.float32))
            see = see[:, :-1]
        for i0 in range(0, max(n, 1), 64):
            r = pm.attention(q[at + i0:at + min(n, i0 + 64)], k, v, None, see[i0:i0 + 64], scale)
            for x, y in zip((o, lse, size), r):
                x.append(y)
        at += n
    return torch.cat(o), torch.cat(lse), torch.cat(size)


def agree(got, want):
    (o, lse), (ow, lw, size) = got, want
    torch.cuda.synchronize()
    assert pv.device_error() == 0
    assert torch.isfinite(o.float()).all()
    off = (o.double() - ow).abs() - O_TOL * size
    assert float(off.max()) <= 1e-30, float(((o.double() - ow).abs() / size.clamp(min=1e-30)).max())
    assert torch.equal(torch.isfinite(lse), torch.isfinite(lw))
    fine = torch.isfinite(lw)
    assert torch.equal(lse[~fine].double(), lw[~fine])
    if fine.any():
        assert float((lse[fine].double() - lw[fine]).abs().max()) <= LSE_TOL


PAGED = [
    # counts, lengths, Hq, Hkv, D, page, window
    ([1], [1], 8, 8, 64, 16, 0),
    ([1], [700], 32, 8, 128, 16, 0),
    ([1, 1, 1], [5, 64, 65], 4, 1, 64, 32, 0),
    ([2, 2], [2, 3000], 32, 4, 128, 64, 0),
    ([2] * 9, [300, 17, 2, 128, 129, 4000, 63, 255, 1000], 16, 2, 128, 16, 0),
    ([0, 3, 0, 1, 5], [40, 3, 0, 777, 130], 6, 2, 64, 16, 0),
    ([7], [1234], 5, 1, 128, 128, 0),
    ([300], [300], 8, 2, 128, 64, 0),
    ([257, 1, 64], [1300, 900, 64], 12, 4, 64, 16, 0),
    ([513, 40], [2049, 2000], 16, 2, 128, 256, 0),
    ([2, 2], [2000, 50], 16, 4, 128, 16, 100),
    ([1, 130, 400], [33, 1500, 400], 9, 3, 64, 32, 77),
    ([700], [1400], 24, 8, 128, 64, 1),
    ([129, 128, 127, 2], [129, 640, 500, 1026], 64, 1, 128, 64, 0),
    ([1000], [5000], 4, 4, 64, 64, 300),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", PAGED, ids=[str(i) for i in range(len(PAGED))])
def test_paged_attention(case, fp8):
    counts, lens, Hq, Hkv, D, page, window = case
    c, gen = fill(lens, page, Hkv, D, fp8, seed=len(lens) + Hq)
    q = torch.randn(sum(counts), Hq, D, generator=gen).to(torch.bfloat16).to(DEV)
    got = pv.paged_attention(c.c, q, offsets(counts), max(counts), window=window, with_lse=True)
    agree(got, expected(c, q, counts, lens, window))


SELECTED = [
    # counts, lengths, Hq, Hkv, D, page, topk
    ([1], [1], 4, 1, 64, 16, 1),
    ([1, 2], [900, 3000], 16, 2, 128, 16, 700),
    ([3, 0, 1], [5, 9, 2000], 8, 8, 64, 32, 130),
    ([40], [40], 64, 1, 128, 64, 64),
    ([2] * 5, [4000, 100, 65, 64, 2], 32, 4, 128, 64, 2048),
    ([50, 30], [800, 30], 20, 4, 64, 16, 333),
    ([9], [5000], 128, 1, 128, 64, 2048),
    ([70], [300], 7, 1, 128, 128, 100),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", SELECTED, ids=[str(i) for i in range(len(SELECTED))])
def test_selected_attention(case, fp8):
    counts, lens, Hq, Hkv, D, page, topk = case
    c, gen = fill(lens, page, Hkv, D, fp8, seed=topk + Hq)
    total = sum(counts)
    q = torch.randn(total, Hq, D, generator=gen).to(torch.bfloat16).to(DEV)
    idx = torch.full((total, topk), -1, dtype=torch.int32)
    r, at = random.Random(topk), 0
    for b, n in enumerate(counts):
        for i in range(n):
            pos = lens[b] - n + i
            pick = r.sample(range(pos + 1), min(topk, pos + 1))
            if r.random() < 0.5:
                pick.sort()
            idx[at, : len(pick)] = torch.tensor(pick, dtype=torch.int32)
            at += 1
    if total > 2:
        idx[1] = -1                                  # nothing selected
        idx[2, topk // 2:] = 2 ** 31 - 1             # positions to come, and past every page
        idx[0, 0] = lens[0] - counts[0] + 1
        idx[total - 1, : min(3, topk)] = 0           # a position named again counts again
        idx[total - 1] = idx[total - 1][torch.randperm(topk, generator=gen)]
    idx = idx.to(DEV)
    got = pv.selected_attention(c.c, q, offsets(counts), max(counts), idx, with_lse=True)
    agree(got, expected(c, q, counts, lens, idx=idx))


# Runs of many key tiles a CTA: the ring, the split key tiles and the sums
# that move, several items one after another.
LONG = [
    # counts, lengths, Hq, Hkv, D, page, window, topk
    ([60], [5000], 64, 1, 128, 64, 0, 2048),
    ([90, 40], [1500, 900], 40, 1, 64, 16, 0, 1500),
    ([2] * 40, [30000] * 40, 40, 1, 128, 128, 0, 0),
    ([20] * 12, [9000 + i for i in range(12)], 16, 4, 128, 32, 0, 0),
    ([600], [20000], 32, 8, 64, 64, 3000, 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", LONG, ids=[str(i) for i in range(len(LONG))])
def test_attention_over_many_tiles(case, fp8):
    counts, lens, Hq, Hkv, D, page, window, topk = case
    c, gen = fill(lens, page, Hkv, D, fp8, seed=Hq + topk)
    total = sum(counts)
    q = torch.randn(total, Hq, D, generator=gen).to(torch.bfloat16).to(DEV)
    # scores that climb along the sequence: the reference point moves often
    q *= torch.linspace(0.2, 6.0, total, device=DEV)[:, None, None].to(torch.bfloat16)
    idx = None
    if topk:
        rows, at = [], 0
        for b, n in enumerate(counts):
            for i in range(n):
                pos = lens[b] - n + i + 1
                pick = torch.randperm(pos, generator=gen)[:topk].sort().values
                rows.append(torch.nn.functional.pad(pick, (0, topk - len(pick)), value=-1))
        idx = torch.stack(rows).to(torch.int32).to(DEV)
        got = pv.selected_attention(c.c, q, offsets(counts), max(counts), idx, with_lse=True)
    else:
        got = pv.paged_attention(c.c, q, offsets(counts), max(counts), window=window, with_lse=True)
    (o, lse), (ow, lw, size) = got, expected(c, q, counts, lens, window, idx)
    torch.cuda.synchronize()
    assert pv.device_error() == 0
    # queries up to six times as long: six times the score error of O_TOL and LSE_TOL
    assert bool(((o.double() - ow).abs() <= (2 * 2.0 ** -8 + 6 * 2.0 ** -10) * size + 1e-30).all())
    assert float((lse.double() - lw).abs().max()) <= 6 * LSE_TOL
