"""Plain models of the paged cache for the tests: the page bookkeeping in
Python integers, and attention in 64 bits."""
import math

import torch

E4M3 = torch.float8_e4m3fn


class Pages:
    """Table, lengths and reference counts as the page calls keep them."""

    def __init__(self, B, columns, pages, page):
        self.B, self.columns, self.pages, self.page = B, columns, pages, page
        self.rows = [[] for _ in range(B)]
        self.len = [0] * B
        self.refs = [0] * pages

    def table(self):
        return [r + [-1] * (self.columns - len(r)) for r in self.rows]

    def append(self, counts):
        """(missing pages, copies [(from page, to page, tokens)])."""
        P = self.page
        shared = [r and self.len[b] % P and self.refs[r[-1]] > 1 for b, r in enumerate(self.rows)]
        fresh = [bool(n and s) for n, s in zip(counts, shared)]
        need = [-(-(l + n) // P) - -(-l // P) + f for l, n, f in zip(self.len, counts, fresh)]
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        if sum(need) > len(free):
            return sum(need) - len(free), []
        copies, old = [], list(self.len)
        for b, n in enumerate(counts):
            take, free = free[: need[b]], free[need[b]:]
            if fresh[b]:
                last = self.rows[b].pop()
                self.refs[last] -= 1
                copies.append((last, take[0], old[b] % P))
            self.rows[b] += take
            for p in take:
                self.refs[p] = 1
            self.len[b] += n
        return 0, copies

    def fork(self, src, dst):
        new = [(list(self.rows[s]), self.len[s]) for s in src]
        for row, _ in new:
            for p in row:
                self.refs[p] += 1
        for d, (row, n) in zip(dst, new):
            for p in self.rows[d]:
                self.refs[p] -= 1
            self.rows[d], self.len[d] = row, n

    def free(self, seqs, keep):
        for b, n in zip(seqs, keep):
            self.len[b] = min(self.len[b], n)
            held = -(-self.len[b] // self.page)
            for p in self.rows[b][held:]:
                self.refs[p] -= 1
            self.rows[b] = self.rows[b][:held]

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        of = [p for p in range(used, self.pages) if self.refs[p] > 0]
        to = [p for p in range(used) if self.refs[p] == 0]
        remap = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        for a, b in zip(of, to):
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[remap[p] for p in r] for r in self.rows]
        return remap, used


def tokens(plane, scale, table, b, n):
    """Tokens 0 .. n - 1 of sequence b in 64 bits: [n, Hkv, D]."""
    P = plane.shape[1]
    t = torch.arange(n, device=plane.device)
    page, slot = table[b].long()[t // P], t % P
    if plane.dtype == E4M3:
        x = plane.view(torch.uint8)[page, slot].view(E4M3).double()
        return x * scale[page, slot].double()[:, None, None]
    return plane[page, slot].double()


def attention(q, k, v, positions, see, scale):
    """q [n, Hq, D], k and v [t, Hkv, D]; see [n, t] (how often a token sees a
    position).  Returns o, lse, and sum p |v|, the size that rounding errors
    of o go by; all in 64 bits."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    k, v = (x.repeat_interleave(G, dim=1).permute(1, 0, 2) for x in (k, v))
    s = (q.double().permute(1, 0, 2) @ k.transpose(1, 2)) * scale
    s = s + torch.log(see.double())[None]
    top = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full((Hq, n, 1), -math.inf)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    p = torch.where(total > 0, p / total, 0.0)
    return (p @ v).permute(1, 0, 2), lse.T, (p @ v.abs()).permute(1, 0, 2)


def quantise(x):
    """e4m3 codes and one scale a token of x [n, heads, D]: largest / 448."""
    x = x.float()
    amax = x.abs().amax(dim=(1, 2))
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / scale[:, None, None]).clamp(-448.0, 448.0).to(E4M3), scale
