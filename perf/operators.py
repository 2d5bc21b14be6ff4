"""Cases of the paged-cache operators: attention of new tokens over a paged
key/value cache, the same over the positions that the indexer selected, the
append of new tokens, and the page operations (fork, free, copy, compact).

The cache of every case: K and V planes of pages ``[pages, page, Hkv, D]``
(bf16, or e4m3 codes with one float32 scale a token), a table
``[B, columns]`` of page ids (-1: none), lengths ``[B]`` that count the new
tokens once they are appended, and one reference count a page (0: free).

``run`` computes an operator in elementary torch operations where ``own`` is
false, and by the library's calls where it is true.
"""
import math
import random

import torch

own = False

BF16, E4M3 = "bf16", "e4m3"
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(name, B, new, length, Hq, Hkv, D, page, dtype, window=0, topk=0, ragged=0):
    """new, length: (lowest, highest) new tokens and cached tokens before them
    of a sequence; topk > 0: over that many selected positions a token."""
    return dict(name=name, op="selected" if topk else "attend", B=B, new_lo=new[0], new_hi=new[1],
                len_lo=length[0], len_hi=length[1], Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                window=window, topk=topk, ragged=ragged)


def _append(name, B, new, length, Hkv, D, page, dtype, shared, ragged=0):
    return dict(name=name, op="append", B=B, new_lo=new[0], new_hi=new[1], len_lo=length[0],
                len_hi=length[1], Hkv=Hkv, D=D, page=page, dtype=dtype, shared=shared,
                ragged=ragged)


def _fork(name, parents, children, length, page, D, ragged=0):
    return dict(name=name, op="fork", parents=parents, children=children, len_lo=length[0],
                len_hi=length[1], page=page, D=D, ragged=ragged)


def _compact(name, B, length, Hkv, D, page, dtype, fill, ragged=0):
    return dict(name=name, op="compact", B=B, len_lo=length[0], len_hi=length[1], Hkv=Hkv, D=D,
                page=page, dtype=dtype, fill=fill, ragged=ragged)


def listed():
    return [
        # one user's next token early in a chat: launch latency is all there is
        _attend("one token, short cache", 1, (1, 1), (700, 700), 32, 8, 128, 16, BF16),
        # a two-token prediction step of a served batch, lengths as in the
        # repository's decode workload (32 sequences, 32K to 128K)
        _attend("two-token step, 32 long caches", 32, (2, 2), (32768, 131072), 32, 4, 128, 64, E4M3,
                ragged=1),
        # a long prompt fed in chunks: one chunk against what is cached so far
        _attend("2048-token chunk over 32K", 1, (2048, 2048), (32768, 32768), 32, 8, 128, 64, BF16),
        # chunks and single tokens of many users in one step, sliding window,
        # three query heads a key head
        _attend("mixed chunks, window 1024", 8, (1, 1500), (0, 8000), 24, 8, 64, 16, E4M3, window=1024,
                ragged=2),
        # sparse decoding: each new token reads the 2048 positions the indexer kept
        _attend("two-token step, 2048 selected", 32, (2, 2), (8192, 32768), 64, 8, 128, 64, BF16,
                topk=2048, ragged=3),
        # sparse prefill of chunks, one key head for 64 query heads
        _attend("chunks, 2048 selected", 2, (150, 700), (1000, 16000), 64, 1, 128, 64, E4M3, topk=2048,
                ragged=4),
        # decoding: the rejected draft tokens are dropped, the next two appended
        _append("two-token append, 128 caches", 128, (2, 2), (20, 150), 2, 128, 16, E4M3, False, ragged=5),
        # prompt chunks appended to forked conversations (shared last pages)
        _append("chunk append, shared pages", 6, (500, 5000), (3000, 12000), 8, 128, 64, BF16, True,
                ragged=6),
        # a beam of four branches of one conversation
        _fork("four branches of one cache", 1, 4, (900, 900), 16, 128),
        # parallel samples of served prompts, and their indexer keys
        _fork("48 branches of 16 long caches", 16, 48, (8192, 32768), 16, 128, ragged=7),
        # a small pool packed before it shrinks
        _compact("small pool", 4, (100, 900), 8, 128, 16, BF16, 0.5, ragged=8),
        # a large pool after many requests came and went
        _compact("large half-empty pool", 48, (2000, 12000), 8, 128, 64, BF16, 0.5, ragged=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "selected", "selected", "append", "fork", "compact"])
    ragged = rng.randrange(1000)
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice([BF16, E4M3])
    if op in ("attend", "selected"):
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 8, 16] + ([64] if Hkv == 1 else []))
        while True:
            if rng.random() < 0.5:      # a decode step
                B, hi, top = _log(rng, 1, 64), _log(rng, 1, 8), 65536
            else:                       # chunks
                B, hi, top = _log(rng, 1, 8), _log(rng, 16, 2048), 24000
            len_hi = _log(rng, 1, top)
            topk = rng.choice([64, 500, 1024, 2048]) if op == "selected" else 0
            window = 0 if topk or rng.random() < 0.7 else _log(rng, 16, 4096)
            kv = B * (len_hi + hi) * Hkv * D * 2
            pairs = B * hi * G * Hkv * (topk or len_hi + hi)
            if kv > 1 << 30 or pairs > 1 << 30 or B * hi * topk * Hkv * D > 1 << 29:
                continue
            return {k: v for k, v in _attend("", B, (rng.randint(1, hi), hi),
                                             (rng.randint(0, len_hi), len_hi), G * Hkv, Hkv, D, page,
                                             dtype, window, topk, ragged).items() if k != "name"}
    if op == "append":
        B, hi = _log(rng, 1, 128), _log(rng, 1, 2000)
        hi = max(1, min(hi, 20000 // B))
        len_hi = max(1, min(_log(rng, 1, 8000), 60000 // B))
        c = _append("", B, (rng.randint(1, hi), hi), (rng.randint(0, len_hi), len_hi),
                    rng.choice([1, 2, 4]), rng.choice([64, 128]), page, dtype, rng.random() < 0.5, ragged)
    elif op == "fork":
        parents = _log(rng, 1, 16)
        hi = _log(rng, 16, 20000)
        c = _fork("", parents, _log(rng, 1, 48), (rng.randint(0, hi), hi), page, 64, ragged)
    else:
        B = _log(rng, 1, 48)
        hi = _log(rng, 16, 8000)
        c = _compact("", B, (rng.randint(1, hi), hi), rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), page,
                     dtype, rng.choice([0.3, 0.5, 0.8, 0.95]), ragged)
    return {k: v for k, v in c.items() if k != "name"}


def _sizes(case):
    """(cached tokens before the call, new tokens) of each sequence, from the case alone."""
    r = random.Random(case["ragged"])
    n = case["parents"] if case["op"] == "fork" else case["B"]
    old = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0 for _ in range(n)]
    return old, new


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantise(x):
    """Rows of x [n, heads, D] as e4m3 codes with one scale a row (largest / 448)."""
    amax = x.abs().amax(dim=(1, 2))
    # divided by a tensor: a quotient by a Python number is taken as a product with its reciprocal
    scale = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    codes = (x / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, scale


def _cache(case, lengths, columns, pages, gen, B=None):
    """A cache whose sequences of `lengths` tokens sit on pages in shuffled order."""
    dev, P = "cuda", case["page"]
    Hkv, D = case["Hkv"], case["D"]
    B = len(lengths) if B is None else B
    shape = (pages, P, Hkv, D)
    k = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    # one key in fifty is "heavy", as in the repository's synthetic inputs
    heavy = torch.rand(pages * P, generator=gen, device=dev) < 0.02
    k.view(-1, Hkv, D)[heavy] *= 4.0
    s = {"k": k, "v": v, "k_scale": None, "v_scale": None}
    if case["dtype"] == E4M3:
        for n in ("k", "v"):
            codes, scale = _quantise(s[n].view(pages * P, Hkv, D).float())
            s[n], s[n + "_scale"] = codes.view(shape), scale.view(pages, P)
    used = [_ceil(x, P) for x in lengths]
    order = torch.randperm(pages, generator=gen, device=dev)[: sum(used)].to(torch.int32)
    table = torch.full((B, columns), -1, dtype=torch.int32)
    spots = []
    for b, n in enumerate(used):
        spots += [b * columns + c for c in range(n)]
    table = table.to(dev)
    table.view(-1)[torch.tensor(spots, dtype=torch.int64, device=dev)] = order
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[order.long()] = 1
    s["table"], s["refs"] = table, refs
    s["len"] = torch.tensor(list(lengths) + [0] * (B - len(lengths)), dtype=torch.int32, device=dev)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, P, op = "cuda", case["page"], case["op"]
    old, new = _sizes(case)
    if op in ("attend", "selected"):
        after = [a + b for a, b in zip(old, new)]
        columns = max(_ceil(x, P) for x in after) + 1
        s = _cache(case, after, columns, sum(_ceil(x, P) for x in after) + 3, gen)
        total, Hq, D = sum(new), case["Hq"], case["D"]
        s["q"] = torch.randn(total, Hq, D, generator=gen, device=dev, dtype=torch.bfloat16)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["max_new"], s["max_len"] = max(new), max(after)
        if op == "selected":
            K = case["topk"]
            idx = torch.full((total, K), -1, dtype=torch.int32, device=dev)
            for b, n in enumerate(new):
                # distinct positions of each token's own prefix, ascending
                for i0 in range(0, n, 256):
                    i1 = min(n, i0 + 256)
                    draws = torch.rand(i1 - i0, after[b], generator=gen, device=dev)
                    pos = torch.arange(old[b] + i0, old[b] + i1, device=dev)
                    draws.masked_fill_(torch.arange(after[b], device=dev)[None] > pos[:, None], 2.0)
                    kk = min(K, after[b])
                    val, at = draws.topk(kk, dim=1, largest=False)
                    at = torch.where(val < 1.5, at, after[b]).sort(dim=1).values
                    idx[cu[b] + i0:cu[b] + i1, :kk] = torch.where(at < after[b], at, -1).to(torch.int32)
            if total > 40:
                idx[17] = -1     # a token that selected nothing
            s["idx"] = idx
    elif op == "append":
        after = [a + b for a, b in zip(old, new)]
        columns = max(_ceil(x, P) for x in after) + 2
        pages = sum(_ceil(x, P) + 2 for x in after)
        s = _cache(case, old, columns, pages, gen)
        if case["shared"]:
            # odd sequences go on from their neighbour's pages: shared, the last one too
            for b in range(1, len(old), 2):
                s["refs"][s["table"][b, : _ceil(old[b], P)].long()] -= 1
                s["table"][b] = s["table"][b - 1]
                s["len"][b] = s["len"][b - 1]
                s["refs"][s["table"][b, : _ceil(old[b - 1], P)].long()] += 1
        s["base"] = s["len"].clone()
        s["seqs"] = torch.arange(len(old), dtype=torch.int32, device=dev)
        total = sum(new)
        for n in ("k_new", "v_new"):
            s[n] = torch.randn(total, case["Hkv"], case["D"], generator=gen, device=dev,
                               dtype=torch.bfloat16)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"], s["max_new"] = torch.tensor(cu, dtype=torch.int32, device=dev), max(new)
    elif op == "fork":
        parents, children = case["parents"], case["children"]
        columns = max(1, max(_ceil(x, P) for x in old))
        c = dict(case, Hkv=1, dtype=BF16, D=8)
        s = _cache(c, old, columns, sum(_ceil(x, P) for x in old) + 2, gen, B=parents + children)
        # the rows' indexer keys, one contiguous row a sequence
        s["keys"] = torch.randn(parents + children, columns * P, case["D"], generator=gen, device=dev,
                                dtype=torch.bfloat16)
        r = random.Random(seed)
        src = [r.randrange(parents) for _ in range(children)]
        s["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
        s["dst"] = torch.tensor(range(parents, parents + children), dtype=torch.int32, device=dev)
        # a branch leaves its parent up to three tokens back
        s["keep"] = torch.tensor([max(0, old[p] - r.randrange(4)) for p in src], dtype=torch.int32,
                                 device=dev)
    else:
        pages = max(2, int(sum(_ceil(x, P) for x in old) / case["fill"]))
        s = _cache(case, old, max(_ceil(x, P) for x in old), pages, gen)
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rows(s, n):
    """A plane as float32 token rows [pages * page, Hkv, D], or a float view of given rows of it."""
    x = s[n].view(-1, s[n].shape[2], s[n].shape[3])
    scale = s[n + "_scale"]
    return x, None if scale is None else scale.view(-1)


def _take(s, n, rows):
    x, scale = _rows(s, n)
    if x.dtype == torch.float8_e4m3fn:
        y = x.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float()
        return y * scale[rows][..., None, None]
    return x[rows].float()


def _softmax_rows(scores, ok):
    """exp(scores - max), its sum, and the log-sum-exp over the last axis; rows with nothing left give 0, 0, -inf."""
    scores = torch.where(ok, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return p, total, lse[..., 0]


def _plain_attend(s):
    c = s["case"]
    P, Hq, Hkv, D = c["page"], c["Hq"], c["Hkv"], c["D"]
    G, B, n, L = Hq // Hkv, c["B"], s["max_new"], s["max_len"]
    dev = s["q"].device
    t = torch.arange(L, device=dev)
    page = s["table"][:, t // P].clamp(min=0).long()
    rows = page * P + t % P                                    # [B, L]
    k, v = _take(s, "k", rows), _take(s, "v", rows)            # [B, L, Hkv, D]
    i = torch.arange(n, device=dev)
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)    # [B, n]
    q = s["q"][at].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    scores = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, G, n, L) * (1.0 / math.sqrt(D))
    pos = s["len"].long()[:, None] - count[:, None] + i        # [B, n]
    ok = (t <= pos[..., None]) & (i < count[:, None])[..., None]
    if c["window"]:
        ok &= t > pos[..., None] - c["window"]
    p, total, lse = _softmax_rows(scores, ok[:, None, None])
    o = (p.view(B, Hkv, G * n, L) @ v.permute(0, 2, 1, 3)).view(B, Hkv, G, n, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)
    live = i < count[:, None]
    return {"o": o[live].to(torch.bfloat16), "lse": lse[live]}


def _plain_selected(s):
    c = s["case"]
    P, Hq, Hkv, D = c["page"], c["Hq"], c["Hkv"], c["D"]
    G, T = Hq // Hkv, s["q"].shape[0]
    dev = s["q"].device
    r = torch.arange(T, device=dev)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], r, right=True)
    pos = s["len"].long()[b] - (cu[1:][b] - r)
    idx = s["idx"].long()
    ok = (idx >= 0) & (idx <= pos[:, None])
    t = torch.where(ok, idx, 0)
    rows = s["table"][b[:, None], t // P].clamp(min=0).long() * P + t % P
    k, v = _take(s, "k", rows), _take(s, "v", rows)            # [T, K, Hkv, D]
    q = s["q"].float().view(T, Hkv, G, D)
    scores = (q @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    p, total, lse = _softmax_rows(scores, ok[:, None, None])
    o = torch.where(total > 0, p @ v.permute(0, 2, 1, 3) / total, 0.0)
    return {"o": o.reshape(T, Hq, D).to(torch.bfloat16), "lse": lse.reshape(T, Hq)}


def _plain_free(s, seqs, keep):
    """Drops the tokens from `keep` on of the sequences `seqs`."""
    P = s["case"]["page"]
    q = seqs.long()
    n = torch.minimum(s["len"][q], keep)
    col = torch.arange(s["table"].shape[1], device=q.device)
    rows = s["table"][q]
    drop = (col >= ((n + P - 1) // P)[:, None]) & (rows >= 0)
    s["refs"].index_add_(0, rows.clamp(min=0).view(-1).long(), -drop.view(-1).to(torch.int32))
    s["table"][q] = torch.where(drop, -1, rows)
    s["len"][q] = n


def _plain_append(s):
    P, dev = s["case"]["page"], s["cu"].device
    cu = s["cu"].long()
    count, length = cu[1:] - cu[:-1], s["len"].long()
    B, columns = s["table"].shape
    have, want = (length + P - 1) // P, (length + count + P - 1) // P
    last = s["table"][torch.arange(B, device=dev), (have - 1).clamp(min=0)].clamp(min=0).long()
    fresh = (length % P != 0) & (count > 0) & (s["refs"][last] > 1)   # a shared last page is copied first
    first = have - fresh.long()
    need = want - first
    start = need.cumsum(0) - need
    free = torch.argsort((s["refs"] != 0).to(torch.int8), stable=True)
    col = torch.arange(columns, device=dev)
    gets = (col >= first[:, None]) & (col < want[:, None])
    pick = free[(start[:, None] + col - first[:, None]).clamp(0, free.shape[0] - 1)]
    s["table"].copy_(torch.where(gets, pick.to(torch.int32), s["table"]))
    s["refs"].index_add_(0, pick.view(-1), gets.view(-1).to(torch.int32))
    s["refs"].index_add_(0, last, -fresh.to(torch.int32))
    # the shared pages' tokens
    slot = torch.arange(P, device=dev)
    copied = fresh[:, None] & (slot < (length % P)[:, None])
    now = s["table"][torch.arange(B, device=dev), (have - 1).clamp(min=0)].clamp(min=0).long()
    to, of = (now[:, None] * P + slot)[copied], (last[:, None] * P + slot)[copied]
    # the new tokens
    r = torch.arange(s["k_new"].shape[0], device=dev)
    b = torch.searchsorted(cu[1:], r, right=True)
    pos = length[b] + r - cu[:-1][b]
    rows = s["table"][b, pos // P].long() * P + pos % P
    s["len"].copy_((length + count).to(torch.int32))
    _write(s, "k", to, of, rows)
    _write(s, "v", to, of, rows)
    return {**_state(s), "lack": torch.zeros(1, dtype=torch.int32, device=dev)}


def _write(s, n, to, of, rows):
    x, scale = _rows(s, n)
    if scale is not None:
        codes, sc = _quantise(s[n + "_new"].float())
        scale[to] = scale[of]
        scale[rows] = sc
        x, new = x.view(torch.uint8), codes.view(torch.uint8)
    else:
        new = s[n + "_new"]
    x[to] = x[of]
    x[rows] = new


def _state(s):
    """The cache's state, 8-bit codes as the values they stand for."""
    return {**{n: s[n] for n in ("table", "len", "refs")}, "k": _values(s, "k"), "v": _values(s, "v")}


def _values(s, n):
    return s[n] if s[n + "_scale"] is None else s[n].float() * s[n + "_scale"][..., None, None]


def _plain_fork(s):
    P = s["case"]["page"]
    src, dst = s["src"].long(), s["dst"].long()
    old, rows = s["table"][dst], s["table"][src]
    s["refs"].index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).view(-1).to(torch.int32))
    s["refs"].index_add_(0, old.clamp(min=0).view(-1).long(), -(old >= 0).view(-1).to(torch.int32))
    s["table"][dst] = rows
    s["len"][dst] = s["len"][src]
    _plain_free(s, s["dst"], s["keep"])
    s["keys"][dst] = s["keys"][src]
    return {n: s[n] for n in ("table", "len", "refs", "keys")}


def _move(plane, to, of):
    x = plane.view(torch.uint8) if plane.dtype == torch.float8_e4m3fn else plane
    x[to] = x[of]


def _plain_compact(s):
    used = s["refs"] > 0
    n = used.sum()
    ids = torch.arange(used.shape[0], device=used.device)
    of, to = (used & (ids >= n)).nonzero()[:, 0], (~used & (ids < n)).nonzero()[:, 0]
    remap = torch.where(used, ids, -1).to(torch.int32)
    remap[of] = to.to(torch.int32)
    _move(s["k"], to, of)
    _move(s["v"], to, of)
    if s["k_scale"] is not None:
        _move(s["k_scale"], to, of)
        _move(s["v_scale"], to, of)
    s["refs"][to] = s["refs"][of]
    s["refs"][of] = 0
    t = s["table"]
    t.copy_(torch.where(t >= 0, remap[t.clamp(min=0).long()], -1))
    return {**_state(s), "remap": remap, "used": n.to(torch.int32).view(1)}


def run(s):
    op = s["case"]["op"]
    if op == "compact":          # the fragmented state again: its pages are still where they were
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
    if own:
        from top_token_selection_b200 import pivot as pv
        if op == "fork":
            cache = pv.make_cache(s["k"], s["v"], s["table"], s["len"], s["refs"])
            pv.pages_fork(cache, s["src"], s["dst"])
            pv.pages_free(cache, s["dst"], s["keep"])
            pv.pages_copy(s["keys"], s["keys"], s["src"], s["dst"])
            return {n: s[n] for n in ("table", "len", "refs", "keys")}
        cache = pv.make_cache(s["k"], s["v"], s["table"], s["len"], s["refs"], s["k_scale"], s["v_scale"])
        if op == "attend":
            o, lse = pv.paged_attention(cache, s["q"], s["cu"], s["max_new"], window=s["case"]["window"],
                                        with_lse=True)
            return {"o": o, "lse": lse}
        if op == "selected":
            o, lse = pv.selected_attention(cache, s["q"], s["cu"], s["max_new"], s["idx"], with_lse=True)
            return {"o": o, "lse": lse}
        if op == "append":
            pv.pages_free(cache, s["seqs"], s["base"])       # the rejected tokens of the last pass
            lack = pv.cache_append(cache, s["k_new"], s["v_new"], s["cu"], s["max_new"])
            return {**_state(s), "lack": lack}
        remap, used = pv.pages_compact(cache)
        return {**_state(s), "remap": remap, "used": used}
    if op == "attend":
        return _plain_attend(s)
    if op == "selected":
        return _plain_selected(s)
    if op == "append":
        _plain_free(s, s["seqs"], s["base"])
        return _plain_append(s)
    return _plain_fork(s) if op == "fork" else _plain_compact(s)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    old, new = _sizes(case)
    op, P = case["op"], case["page"]
    if op == "fork":
        # the parents' table rows read once, the children's old and new rows, the keys of each child
        # read from its parent and written
        columns = max(1, max(_ceil(x, P) for x in old))
        keys = columns * P * case["D"] * 2
        kids = case["children"]
        distinct = min(kids, case["parents"])
        return {"bytes": (distinct + kids) * keys + (distinct + 2 * kids) * columns * 4, "flops": 0}
    size = 2 if case["dtype"] == BF16 else 1
    token = 2 * (case["Hkv"] * case["D"] * size + (4 if size == 1 else 0))     # K and V of a token
    if op in ("attend", "selected"):
        D, Hq = case["D"], case["Hq"]
        pairs, read = 0, 0
        for a, n in zip(old, new):
            if op == "selected":
                pairs += sum(min(case["topk"], a + i + 1) for i in range(n))
                read += min(a + n, case["topk"] * n)
            else:
                w = case["window"] or a + n
                pairs += sum(min(w, a + i + 1) for i in range(n))
                read += min(a + n, w + n - 1)
        rows = sum(new)
        return {"bytes": read * token + rows * Hq * (D * 4 + 4) + rows * case["topk"] * 4,
                "flops": 4.0 * D * Hq * pairs}
    if op == "append":
        rows = sum(new)
        return {"bytes": rows * (2 * case["Hkv"] * case["D"] * 2 + token), "flops": 0}
    # compact: the used pages above the used count move (their share of the pool is random: the mean)
    used = sum(_ceil(x, P) for x in old)
    pages = max(2, int(used / case["fill"]))
    return {"bytes": 2 * used * (1 - used / pages) * P * token + pages * 12, "flops": 0}


def _exact_rows(s, plane, b, positions):
    """K or V of positions of sequence b in 64 bits, one gather by page and slot."""
    P = s["case"]["page"]
    pages = s["table"][b].long()[positions.div(P, rounding_mode="floor")]
    slots = positions.remainder(P)
    x = s[plane]
    if x.dtype == torch.float8_e4m3fn:
        vals = x.view(torch.uint8)[pages, slots].view(torch.float8_e4m3fn).to(torch.float64)
        return vals * s[plane + "_scale"][pages, slots].to(torch.float64)[:, None, None]
    return x[pages, slots].to(torch.float64)


def exact(case, seed):
    if case["op"] not in ("attend", "selected"):
        # moved bits and whole numbers; a quantised token's nearest code has no value besides itself
        return None
    s = prepare(case, seed)
    old, new = _sizes(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    total = sum(new)
    out = torch.zeros(total, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((total, Hq), -math.inf, dtype=torch.float64, device="cuda")
    root = math.sqrt(D)
    row = 0
    for b, (a, n) in enumerate(zip(old, new)):
        q = s["q"][row:row + n].to(torch.float64)
        if case["op"] == "attend":
            every = torch.arange(a + n, device="cuda")
            kk, vv = _exact_rows(s, "k", b, every), _exact_rows(s, "v", b, every)
            for i0 in range(0, n, 128):
                i1 = min(n, i0 + 128)
                lo = max(0, a + i0 + 1 - case["window"]) if case["window"] else 0
                hi = a + i1
                at = torch.arange(a + i0, a + i1, device="cuda")[:, None]
                seen = every[lo:hi][None]
                hidden = seen > at
                if case["window"]:
                    hidden = hidden | (at - seen >= case["window"])
                for h in range(Hq):
                    x = q[i0:i1, h] @ kk[lo:hi, h // G].T / root
                    x = x.masked_fill(hidden, -math.inf)
                    z = torch.logsumexp(x, dim=1)
                    lse[row + i0:row + i1, h] = z
                    out[row + i0:row + i1, h] = torch.exp(x - z[:, None]) @ vv[lo:hi, h // G]
        else:
            for i in range(n):
                chosen = s["idx"][row + i].long()
                chosen = chosen[(chosen >= 0) & (chosen <= a + i)]
                if chosen.numel() == 0:
                    continue
                kk, vv = _exact_rows(s, "k", b, chosen), _exact_rows(s, "v", b, chosen)
                x = torch.einsum("hgd,thd->hgt", q[i].view(Hkv, G, D), kk) / root
                z = torch.logsumexp(x, dim=-1)
                lse[row + i] = z.reshape(Hq)
                out[row + i] = torch.einsum("hgt,thd->hgd", torch.exp(x - z[..., None]), vv).reshape(Hq, D)
        row += n
    return {"o": out, "lse": lse}
