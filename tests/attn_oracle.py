"""Plain 64-bit oracle of the cached-attention operators, on the CPU, from
their definitions alone (loops over sequences, heads and tokens), and builders
of small paged problems.

Tolerances of the attention output (per element), with u = eps / 2 of the
payload type, M = sum_j w_j |v_j| and dS the error bound of a score:
  u |o|        the final rounding
  u M          every weight rounded once to the payload type for the product
               (fp16 weights keep 11 bits down to 2^-22 of the largest; what
               lies below adds less than 2^-33 n M, inside the fp32 term)
  2 dS M       a score off by dS changes its weight and the sum by e^(dS)
  2^-20 M      exponentials, sums and the rescaling in fp32
dS = (Dk + 4) 2^-24 max_j scale sum_i |q_i k_ij|: a product sum in fp32 in any
order, then one rounding by the scale.  The log-sum-exp is off by at most
dS + 2^-20 + 2^-22 |lse|.
"""
from __future__ import annotations

import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def owned(x, rank, N, inter):
    """Positions p < x with (p // inter) % N == rank, counted one by one."""
    return sum(1 for p in range(max(x, 0)) if p // inter % N == rank)


def owned_fast(x, rank, N, inter):
    block = N * inter
    return x // block * inter + min(max(x % block - rank * inter, 0), inter)


class Problem:
    """A batch over one rank's paged cache, on the CPU.

    seqs: (new tokens, whole length) of each sequence.  cut: keys dropped from
    the front of every sequence's cache (as an eviction leaves it)."""

    def __init__(self, seqs, Hq, Hkv, Dk, Dv, *, dtype=torch.bfloat16, cache=None, page=16, N=1, rank=0, inter=1,
                 causal=True, shared=False, seed=0, cut=0, lead=0, tail=0, spare=2, cross=None):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.Dk, self.Dv = seqs, Hq, Hkv, Dk, Dv
        self.dtype, self.cache, self.page = dtype, cache or dtype, page
        self.N, self.rank, self.inter, self.causal, self.shared = N, rank, inter, causal, shared
        self.B = len(seqs)
        self.lead = lead
        self.T = lead + sum(n for n, _ in seqs) + tail
        cu = [lead]
        for n, _ in seqs:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        if cross is not None:
            kv = list(cross)
        else:
            kv = [max(0, owned(length, rank, N, inter) - cut) for _, length in seqs]
        self.kv = torch.tensor(kv, dtype=torch.int32)
        self.seq = torch.tensor([length for _, length in seqs], dtype=torch.int32)
        need = [-(-n // page) for n in kv]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(need + [1]) + 1
        self.table = torch.full((self.B, width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = order.pop()
        self.q = torch.randn(self.T, Hq, Dk, generator=g).to(dtype)
        self.k = torch.randn(self.pages, page, Hkv, Dk, generator=g).to(self.cache)
        self.v = None if shared else torch.randn(self.pages, page, Hkv, Dv, generator=g).to(self.cache)
        fp8 = self.cache == torch.float8_e4m3fn
        self.ks, self.vs = (0.75, 1.25) if fp8 else (1.0, 1.0)
        self.scale = Dk ** -0.5

    def place(self, b, j):
        return int(self.table[b, j // self.page]), j % self.page

    def rows(self, b):
        """(page, place) index tensors of sequence b's cached keys, and which of them exist."""
        j = torch.arange(int(self.kv[b]))
        page = self.table[b].long()[j // self.page]
        there = (page >= 0) & (page < self.pages)
        return page.clamp(0, self.pages - 1), j % self.page, there

    def seen(self, b):
        """[new tokens, keys] truth: does the token see the key?"""
        n, length = self.seqs[b]
        kv = int(self.kv[b])
        _, _, there = self.rows(b)
        m = there[None].repeat(n, 1)
        if self.causal:
            for i in range(n):
                t = length - n + i
                hidden = sum(1 for p in range(t + 1, length) if p // self.inter % self.N == self.rank)
                m[i, max(0, kv - hidden):] = False
        return m

    def keys(self, b, h):
        page, place, _ = self.rows(b)
        return self.k.double()[page, place, h] * self.ks

    def values(self, b, h):
        page, place, _ = self.rows(b)
        if self.shared:
            return self.keys(b, h)[:, :self.Dv]
        return self.v.double()[page, place, h] * self.vs

    def attention(self):
        """(out, lse, out tolerance, lse tolerance), rows outside the sequences NaN."""
        G = self.Hq // self.Hkv
        u = U[self.dtype]
        out = torch.full((self.T, self.Hq, self.Dv), math.nan, dtype=torch.float64)
        lse = torch.full((self.T, self.Hq), math.nan, dtype=torch.float64)
        tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (n, _) in enumerate(self.seqs):
            m = self.seen(b)
            at = slice(int(self.cu[b]), int(self.cu[b]) + n)
            for h in range(self.Hq):
                q = self.q[at, h].double()
                k, v = self.keys(b, h // G), self.values(b, h // G)
                kk = torch.where(torch.isfinite(k), k, 0.0)
                ds = (self.Dk + 4) * 2.0 ** -24 * self.scale * ((q.abs() @ kk.abs().t()) * m).amax(1, keepdim=True) \
                    if k.shape[0] else torch.zeros(n, 1, dtype=torch.float64)
                for i in range(n):
                    s = self.scale * (k[m[i]] @ q[i])
                    w = torch.exp(s - (s.max() if len(s) else 0.0))
                    total = w.sum()
                    row = at.start + i
                    if len(s) == 0 or bool((s == -math.inf).all()):
                        out[row, h], lse[row, h] = 0.0, -math.inf
                        continue
                    out[row, h] = (w / total) @ v[m[i]]
                    lse[row, h] = s.max() + torch.log(total)
                    M = (w / total) @ v[m[i]].abs()
                    tol[row, h] = u * (out[row, h].abs() + M) + (2 * ds[i] + 2.0 ** -20) * M + FLOOR[self.dtype]
                    tol_l[row, h] = ds[i, 0] + 2.0 ** -20 + 2.0 ** -22 * lse[row, h].abs()
        return out, lse, tol, tol_l

    def mass(self, lse, before):
        """(mass, tolerance): before [pages,page,Hkv] plus the weights of every row."""
        G = self.Hq // self.Hkv
        got, tol = before.double().clone(), torch.full(before.shape, 2.0 ** -60, dtype=torch.float64)
        for b, (n, _) in enumerate(self.seqs):
            m = self.seen(b)
            page, place, there = self.rows(b)
            at = slice(int(self.cu[b]), int(self.cu[b]) + n)
            for h in range(self.Hq):
                q, k = self.q[at, h].double(), self.keys(b, h // G)
                kk = torch.where(torch.isfinite(k), k, 0.0)
                s = self.scale * (q @ kk.t())
                ds = (self.Dk + 4) * 2.0 ** -24 * self.scale * (q.abs() @ kk.abs().t())
                g = lse[at, h].double()[:, None]
                w = torch.where(m & (g != -math.inf), torch.exp(s - g), 0.0)
                # the score's error, the scaled log-sum-exp's rounding, the exponential and the sum in fp32
                e = w * (ds + 2.0 ** -22 * (g.abs() * 1.5 + s.abs()) + 2.0 ** -20)
                e = torch.where(torch.isfinite(e), e, 0.0)
                got[page[there], place[there], h // G] += w.sum(0)[there]
                tol[page[there], place[there], h // G] += e.sum(0)[there]
        return got, tol + 2.0 ** -23 * got.abs()


def evict(mass, table, kv, budget, sink, recent, pages):
    """(new_len, kept) by sorting: NaN first, then by weight, ties to the oldest."""
    B, Hkv = table.shape[0], mass.shape[2]
    page = mass.shape[1]
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    new = []
    for b in range(B):
        L = int(kv[b])
        new.append(min(L, budget))
        for h in range(Hkv):
            def weight(j):
                if j < sink or j >= L - recent:
                    return (2, 0.0)
                p = int(table[b, j // page])
                if not 0 <= p < pages:
                    return (0, -math.inf)
                x = float(mass[p, j % page, h])
                return (1, 0.0) if math.isnan(x) else (0, x)
            order = list(range(L))
            if L > budget:
                order.sort(key=lambda j: (-weight(j)[0], -weight(j)[1], j))
                order = sorted(order[:budget])
            kept[b, h, :len(order)] = torch.tensor(order, dtype=torch.int32)
    return torch.tensor(new, dtype=torch.int32), kept


def norm_rope(x, w, eps, cos_sin, pos, off, pairs):
    """[T, H, D] in 64 bits, one column pair at a time."""
    x = x.double().clone()
    if w is not None:
        n = w.numel()
        r = 1.0 / torch.sqrt((x[..., :n] ** 2).mean(-1, keepdim=True) + eps)
        x[..., :n] = x[..., :n] * r * w.double()
    half = cos_sin.shape[1] // 2
    y = x.clone()
    for t in range(x.shape[0]):
        p = min(max(int(pos[t]), 0), cos_sin.shape[0] - 1)
        for j in range(half):
            a, b = (off + 2 * j, off + 2 * j + 1) if pairs else (off + j, off + j + half)
            c, s = float(cos_sin[p, j]), float(cos_sin[p, half + j])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y
