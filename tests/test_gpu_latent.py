"""latent_queries, latent_values, latent_expand and dcp_latent_attn against their definitions in 64 bits.

Tolerances.  A product sum of K terms in fp32, in any order: (K + 2) 2^-24 sum |x w|.  The result rounded once to the
payload type: u |y|, u = eps / 2, and half the smallest subnormal.  An 8-bit cache's values are exact in 16 bits; the
scale is one more fp32 rounding.  A result in two parts is off by u^2 |y| (the rest of at most u |y| is rounded once more)
and half the smallest subnormal.  Attention over expanded rows is checked against the exact definition with what the keys'
and values' rounding r can do (r = u^2 in two parts, u rounded): keys off by r |k| move a score by dS = r scale sum |q k|,
values by r |v|."""
import math

import pytest
import torch

from attn_oracle import FLOOR, U, Problem
from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rand(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def close(got, want, tol):
    got = got.cpu().double()
    assert got.shape == want.shape
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    off = torch.where(nan | (got == want), 0.0, (got - want).abs() - tol)       # (equal infinities)
    assert not bool((off > 0).any()) and not bool(torch.isnan(off).any()), float(off.max())


def product(x, w):
    """x [T,H,K], w [H,N,K] -> (y [T,H,N], its tolerance)."""
    xd, wd = x.double().transpose(0, 1), w.double().transpose(1, 2)
    y = torch.bmm(xd, wd.contiguous()).transpose(0, 1)
    m = torch.bmm(xd.abs(), wd.abs().contiguous()).transpose(0, 1)
    return y, U[x.dtype] * y.abs() + (x.shape[2] + 2) * 2.0 ** -24 * m * (1 + U[x.dtype]) + FLOOR[x.dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 2, 31, 64, 65, 129, 300])
@pytest.mark.parametrize("Dn,Dr,Dc", [(128, 64, 512), (8, 0, 8), (72, 8, 456), (192, 32, 320)])
def test_queries(T, Dn, Dr, Dc, dtype):
    g = torch.Generator().manual_seed(T)
    H = 3
    q, w = rand(g, T, H, Dn + Dr, dtype=dtype), rand(g, H, Dn, Dc, dtype=dtype, scale=Dc ** -0.5)
    y, tol = product(q[..., :Dn], w.transpose(1, 2))
    for weights in (w.to(DEV), w.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)):
        got = attn.latent_queries(q.to(DEV), weights)
        assert got.shape == (T, H, Dc + Dr)
        close(got[..., :Dc], y, tol)
        assert torch.equal(got[..., Dc:].cpu(), q[..., Dn:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 17, 64, 128, 129, 257])
@pytest.mark.parametrize("Dv,Dc", [(128, 512), (8, 8), (136, 72), (64, 1000)])
def test_values(T, Dv, Dc, dtype):
    g = torch.Generator().manual_seed(T)
    H = 5
    o, w = rand(g, T, H, Dc, dtype=dtype), rand(g, H, Dv, Dc, dtype=dtype, scale=Dc ** -0.5)
    y, tol = product(o, w)
    close(attn.latent_values(o.to(DEV), w.to(DEV)), y, tol)
    close(attn.latent_values(o.to(DEV), w.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)), y, tol)


@pytest.mark.parametrize("T", [3, 200])
def test_products_of_strided_rows(T):
    """Rows within wider ones, heads outermost, weights inside one projection, an output within a larger buffer whose rest
    stays as it was."""
    g = torch.Generator().manual_seed(1)
    H, Dn, Dr, Dv, Dc = 4, 64, 16, 96, 160
    whole = rand(g, H, Dn + Dv, Dc, scale=Dc ** -0.5)
    kv_b = whole.to(DEV)
    qkv = rand(g, T, H * (Dn + Dr) + 24)
    q = qkv[:, 16:16 + H * (Dn + Dr)].unflatten(1, (H, Dn + Dr))
    buf = torch.full((T + 2, H + 1, Dc + Dr + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[1:T + 1, 1:, 8:]
    got = attn.latent_queries(qkv.to(DEV)[:, 16:16 + H * (Dn + Dr)].unflatten(1, (H, Dn + Dr)), kv_b[:, :Dn], out=out)
    assert got.data_ptr() == out.data_ptr()
    y, tol = product(q[..., :Dn], whole[:, :Dn].transpose(1, 2))
    close(got[..., :Dc], y, tol)
    assert torch.equal(got[..., Dc:].cpu(), q[..., Dn:])
    assert bool((buf[0] == 7).all() and (buf[T + 1] == 7).all() and (buf[:, 0] == 7).all() and (buf[..., :8] == 7).all())
    o = rand(g, H, T, Dc)                                                   # heads outermost
    got = attn.latent_values(o.to(DEV).transpose(0, 1), kv_b[:, Dn:])
    close(got, *product(o.transpose(0, 1), whole[:, Dn:]))


def test_rows_of_one_token_do_not_reach_another():
    """NaN and infinities in one row or one head stay there; no tokens write nothing."""
    g = torch.Generator().manual_seed(2)
    for T in (70, 200):
        o, w = rand(g, T, 3, 64), rand(g, 3, 40, 64)
        o[5, 1] = math.nan
        o[T - 1, 2, 3] = math.inf
        w[0, 7, 60] = math.inf
        got = attn.latent_values(o.to(DEV), w.to(DEV)).cpu()
        y = torch.bmm(o.double().transpose(0, 1), w.double().transpose(1, 2).contiguous()).transpose(0, 1)
        assert torch.equal(torch.isnan(got), torch.isnan(y)) and torch.equal(torch.isinf(got), torch.isinf(y))
    assert attn.latent_values(torch.empty(0, 3, 64, dtype=torch.float16, device=DEV), w.to(DEV, torch.float16)).shape == (0, 3, 40)


class Rows:
    """Cached latent rows of a few sequences, and a projection's weights."""

    def __init__(self, kv, H, Dn, Dr, Dv, Dc, dtype=torch.bfloat16, cache=None, page=16, seed=0, missing=()):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.H, self.Dn, self.Dr, self.Dv, self.Dc = kv, H, Dn, Dr, Dv, Dc
        self.dtype, self.page = dtype, page
        need = [-(-n // page) for n in kv]
        self.pages = sum(need) + 1
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((len(kv), max(need + [1])), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = order.pop()
        for b, i in missing:
            self.table[b, i] = -1 if b % 2 == 0 else self.pages + 3
        self.cache = rand(g, self.pages, page, 1, Dc + Dr, dtype=cache or dtype)
        self.ks = 0.75 if cache == torch.float8_e4m3fn else 1.0
        self.w = rand(g, H, Dn + Dv, Dc, dtype=dtype, scale=Dc ** -0.5)
        self.len = torch.tensor(kv, dtype=torch.int32)

    def gpu(self):
        w = self.w.to(DEV)
        return self.cache.to(DEV), w[:, :self.Dn], w[:, self.Dn:], self.table.to(DEV), self.len.to(DEV)

    def exact(self, most):
        """(k, v, their tolerances, which keys there are)."""
        B, H = len(self.kv), self.H
        k = torch.zeros(B, most, H, self.Dn + self.Dr, dtype=torch.float64)
        v = torch.zeros(B, most, H, self.Dv, dtype=torch.float64)
        tk, tv, there = torch.zeros_like(k), torch.zeros_like(v), torch.zeros(B, most, dtype=torch.bool)
        wd = self.w.double()
        for b, n in enumerate(self.kv):
            n = min(n, most, self.table.shape[1] * self.page)
            j = torch.arange(n)
            pg = self.table[b].long()[j // self.page]
            there[b, :n] = (pg >= 0) & (pg < self.pages)
            row = self.cache.double()[pg.clamp(0, self.pages - 1), j % self.page, 0] * self.ks
            c = row[:, :self.Dc]
            y = torch.einsum("jc,hnc->jhn", c, wd)
            m = torch.einsum("jc,hnc->jhn", c.abs(), wd.abs())
            t = U[self.dtype] * y.abs() + (self.Dc + 3) * 2.0 ** -24 * m * 1.01 + FLOOR[self.dtype]
            k[b, :n, :, :self.Dn], tk[b, :n, :, :self.Dn] = y[..., :self.Dn], t[..., :self.Dn]
            v[b, :n], tv[b, :n] = y[..., self.Dn:], t[..., self.Dn:]
            k[b, :n, :, self.Dn:] = row[:, None, self.Dc:]
            tk[b, :n, :, self.Dn:] = (U[self.dtype] + 2.0 ** -24) * row[:, None, self.Dc:].abs() + FLOOR[self.dtype]
        return k, v, tk, tv, there


DIMS = [(3, 128, 64, 128, 512), (1, 8, 0, 8, 8), (5, 40, 24, 72, 200), (2, 192, 64, 64, 256), (16, 64, 32, 64, 512)]


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, torch.float8_e4m3fn),
                                         (torch.float16, torch.float8_e4m3fn)])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("kv,page", [([1], 1), ([300, 0, 5, 257], 24), ([256, 255], 64)])
def test_expand(kv, page, dims, dtype, cache):
    p = Rows(kv, *dims, dtype=dtype, cache=cache, page=page, missing=[(0, 0)] if len(kv) == 4 else ())
    most = max(kv) + 3
    k = torch.full((len(kv), most, dims[0], dims[1] + dims[2]), 9.0, dtype=dtype, device=DEV)
    v = torch.full((len(kv), most, dims[0], dims[3]), 9.0, dtype=dtype, device=DEV)
    places = torch.full((len(kv), most), -77, dtype=torch.int32, device=DEV)
    got = attn.latent_expand(*p.gpu(), most, k_scale=p.ks, k_out=k, v_out=v, places=places)
    assert got[0].data_ptr() == k.data_ptr() and got[1].data_ptr() == v.data_ptr()
    ek, ev, tk, tv, there = p.exact(most)
    m = there[:, :, None, None]
    close(k, torch.where(m, ek, 9.0), torch.where(m, tk, 0.0))
    close(v, torch.where(m, ev, 9.0), torch.where(m, tv, 0.0))
    # in two parts
    k2, v2 = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    kr, vr = torch.full_like(k[..., :dims[1]], 9.0).contiguous(), torch.full_like(v, 9.0)
    attn.latent_expand(*p.gpu(), most, k_scale=p.ks, k_out=k2, v_out=v2, k_rest=kr, v_rest=vr)
    assert torch.equal(k2, k) and torch.equal(v2, v)
    for whole, rest, want, tol, c in ((k[..., :dims[1]], kr, ek[..., :dims[1]], tk[..., :dims[1]], dims[1]), (v, vr, ev, tv, dims[3])):
        both = whole.cpu().double() + rest.cpu().double()
        fine = tol - U[dtype] * want.abs() + U[dtype] ** 2 * want.abs()
        close(both, torch.where(m, want, 18.0), torch.where(m, fine, 0.0))
    at = torch.arange(len(kv) * most).view(len(kv), most)
    want = torch.where(there, at, -1)
    counted = torch.arange(most)[None] < p.len[:, None]
    assert torch.equal(places.cpu().long(), torch.where(counted, want, -77))


def test_expand_clamps_lengths():
    """Lengths beyond the buffers and beyond the page table; strided caches, weights and outputs."""
    p = Rows([100, 70, 10], 3, 16, 8, 24, 40, page=16)
    cache, wk, wv, table, _ = p.gpu()
    for most, width in ((50, 7), (200, 3), (64, 4)):
        p.kv = [500, -3, 10]
        wide = torch.zeros(p.pages, 20, 2, 56, dtype=torch.bfloat16, device=DEV)[:, 2:18, :1, :48]
        wide.copy_(cache)
        k = torch.full((4, 3, most, 32), 9.0, dtype=torch.bfloat16, device=DEV)         # heads outermost
        v = torch.full((3, most, 3, 32), 9.0, dtype=torch.bfloat16, device=DEV)
        places = torch.full((3, most), -77, dtype=torch.int32, device=DEV)
        full = p.table
        p.table = full[:, :width]
        ko = torch.as_strided(k, (3, most, 3, 24), (most * 32, 32, 3 * most * 32, 1), 3 * most * 32 + 8)
        attn.latent_expand(wide, wk, wv, table[:, :width], torch.tensor(p.kv, dtype=torch.int32, device=DEV), most,
                           k_out=ko, v_out=v[..., 8:], places=places)
        p.kv = [500, 0, 10]
        ek, ev, tk, tv, there = p.exact(most)
        m = there[:, :, None, None]
        close(ko, torch.where(m, ek, 9.0), torch.where(m, tk, 0.0))
        close(v[..., 8:], torch.where(m, ev, 9.0), torch.where(m, tv, 0.0))
        assert bool((v[..., :8] == 9).all() and (k[0] == 9).all() and (k[..., :8] == 9).all())
        at = torch.where(there, torch.arange(3 * most).view(3, most), -1)
        counted = torch.arange(most)[None] < torch.tensor([500, 0, 10])[:, None]
        assert torch.equal(places.cpu().long(), torch.where(counted, at, -77))
        p.table = full
    p.kv = [500, -3, 10]
    empty = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    places.fill_(-77)
    attn.latent_expand(wide, wk, wv, empty, torch.tensor(p.kv, dtype=torch.int32, device=DEV), 64, k_out=ko, v_out=v[..., 8:],
                       places=places)
    assert places.cpu().tolist() == [[-1] * 64, [-77] * 64, [-1] * 10 + [-77] * 54]
    attn.latent_expand(wide, wk, wv, table, torch.tensor(p.kv, dtype=torch.int32, device=DEV), 0)


def test_one_key_does_not_reach_another():
    p = Rows([300, 40], 3, 32, 16, 32, 64)
    p.cache[int(p.table[0, 0]), 3] = math.nan
    p.cache[int(p.table[1, 1]), 5, 0, 2] = math.inf
    k, v = attn.latent_expand(*p.gpu(), 300)
    assert int(torch.isnan(k[0]).sum()) == 3 * 48 and int(torch.isnan(v[0]).sum()) == 3 * 32
    assert bool(torch.isnan(k[0, 3]).all()) and not bool(torch.isfinite(v[1, 21]).any())
    assert bool(torch.isfinite(v[1, :21]).all()) and bool(torch.isfinite(v[1, 22:40]).all())


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, None), (torch.float16, torch.float8_e4m3fn)])
@pytest.mark.parametrize("N,rank,inter", [(1, 0, 1), (4, 2, 1), (2, 1, 16)])
@pytest.mark.parametrize("mode", ["parts", "wide", "rounded"])
@pytest.mark.parametrize("dims", [(64, 16, 48, 128), (128, 64, 128, 64), (96, 32, 128, 72), (160, 64, 200, 64), (8, 0, 8, 16)])
def test_latent_attention(N, rank, inter, mode, dims, dtype, cache):
    """The expanded form against the definition, and against the absorbed form over the same cache."""
    Dn, Dr, Dv, Dc = dims
    H = 3
    seqs = [(40, 300), (1, 90), (7, 7), (0, 50)]
    lat = Problem(seqs, H, 1, Dc + Dr, Dc, dtype=dtype, cache=cache, page=16, N=N, rank=rank, inter=inter, shared=True, seed=3)
    if N == 1:
        lat.table[0, 2] = -1
    g = torch.Generator().manual_seed(4)
    w = rand(g, H, Dn + Dv, Dc, dtype=dtype, scale=Dc ** -0.5)
    q = rand(g, lat.T, H, Dn + Dr, dtype=dtype)
    most = int(lat.kv.max())
    wg = w.to(DEV)
    scale = (Dn + Dr) ** -0.5
    args = dict(seq_len=lat.seq.to(DEV), scale=scale, rank=rank, n_ranks=N, interleave=inter)
    cache_g, table, cu, kv = lat.k.to(DEV), lat.table.to(DEV), lat.cu.to(DEV), lat.kv.to(DEV)
    out, lse = attn.dcp_latent_attn(q.to(DEV), cache_g, wg[:, :Dn], wg[:, Dn:], table, cu, kv, most, k_scale=lat.ks,
                                    rounded=mode == "rounded", wide_weights=mode == "wide", **args)
    out, lse = out.cpu().double(), lse.cpu().double()
    u = U[dtype]
    ur = u if mode == "rounded" else u * u
    for b, (n, _) in enumerate(seqs):
        m = lat.seen(b)
        row = lat.keys(b, 0)
        for h in range(H):
            key = torch.cat([row[:, :Dc] @ w[h, :Dn].double().t(), row[:, Dc:]], 1)
            val = row[:, :Dc] @ w[h, Dn:].double().t()
            mag = row[:, :Dc].abs() @ w[h, Dn:].double().abs().t() * (Dc + 3) * 2.0 ** -24
            kmag = torch.cat([row[:, :Dc].abs() @ w[h, :Dn].double().abs().t() * (Dc + 3) * 2.0 ** -24, 0 * row[:, Dc:]], 1)
            at = slice(int(lat.cu[b]), int(lat.cu[b]) + n)
            for i in range(n):
                r, qd = at.start + i, q[at.start + i, h].double()
                if not bool(m[i].any()):
                    assert bool((out[r, h] == 0).all()) and float(lse[r, h]) == -math.inf
                    continue
                s = scale * (key[m[i]] @ qd)
                ds = float((scale * ((ur * key[m[i]].abs() + kmag[m[i]] + FLOOR[dtype]) @ qd.abs() +
                                     (2 * Dn + Dr + 4) * 2.0 ** -24 * (key[m[i]].abs() @ qd.abs()))).max())
                p = torch.softmax(s, 0)
                o, M = p @ val[m[i]], p @ val[m[i]].abs()
                # the output's and a weight's rounding (a wide weight's rest, 2^-16 or less), the values' and their sums', the scores'
                tol = u * o.abs() + ((u * u if mode == "wide" and ur == u * u else u) + ur) * M + p @ mag[m[i]] + FLOOR[dtype] + (2 * ds * (1 + 2 * ds) + 2.0 ** -20) * M * (1 + 2 * u) + FLOOR[dtype]
                assert bool(((out[r, h] - o).abs() <= tol).all())
                assert abs(float(lse[r, h] - torch.logsumexp(s, 0))) <= ds + 2.0 ** -20 + 2.0 ** -22 * abs(float(lse[r, h]))
    # the absorbed form: other roundings (the latent queries' and outputs'), the same attention
    ql = attn.latent_queries(q.to(DEV), wg[:, :Dn])
    ol, lse2 = attn.dcp_paged_attn(ql, cache_g, None, table, cu, kv, v_dim=Dc, k_scale=lat.ks, **args)
    got = attn.latent_values(ol, wg[:, Dn:]).cpu().double()
    # (a score off by 2^-8 of sum |q k| scale, of scores near 1; values of magnitude near 1)
    tol = 64 * u
    seen = torch.isfinite(lse)
    assert torch.equal(seen, torch.isfinite(lse2.cpu()))
    assert float((got - out)[seen].abs().max()) <= tol and float((lse2.cpu().double() - lse)[seen].abs().max()) <= tol


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("dims", [(64, 64, 64), (128, 64, 128), (192, 64, 200)])
def test_latent_rows_that_are_masked_reach_no_token(dims, what):
    """Not finite: a latent row that the first tokens of a chunk do not see, one behind the length, and buffers that hold
    anything before the call."""
    Dn, Dr, Dv, Dc, H = *dims, 96, 2
    p = Rows([100], H, Dn, Dr, Dv, Dc, page=16, seed=7)
    p.cache[int(p.table[0, 6]), 3] = what                       # key 99: seen by the last token alone
    p.cache[int(p.table[0, 6]), 4:] = what
    g = torch.Generator().manual_seed(8)
    q = rand(g, 40, H, Dn + Dr).to(DEV)
    cu = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    full = lambda d: torch.full((1, 128, H, d), what, dtype=torch.bfloat16, device=DEV)       # noqa: E731
    for rounded in (False, True):
        more = {} if rounded else dict(k_rest=full(Dn), v_rest=full(Dv))
        out, lse = attn.dcp_latent_attn(q, *p.gpu()[:4], cu, p.len.to(DEV), 128, rounded=rounded, k_out=full(Dn + Dr),
                                        v_out=full(Dv), **more)
        ref, rl = attn.dcp_latent_attn(q[:39], *p.gpu()[:4], torch.tensor([0, 39], dtype=torch.int32, device=DEV),
                                       p.len.to(DEV) - 1, 128, rounded=rounded)
        assert bool(torch.isfinite(out[:39]).all()) and bool(torch.isfinite(lse[:39]).all())
        assert float((out[:39].float() - ref.float()).abs().max()) <= 2.0 ** -6 and float((lse[:39] - rl).abs().max()) <= 2.0 ** -14
        assert not bool(torch.isfinite(out[39]).all())


def test_layer_captured_and_replayed():
    """Queries into latent space, append, attention, values, and the expanded form, as one graph on new inputs."""
    H, Dn, Dr, Dv, Dc, page, B = 4, 64, 64, 64, 128, 16, 3
    g = torch.Generator().manual_seed(5)
    w = rand(g, H, Dn + Dv, Dc, scale=Dc ** -0.5).to(DEV)
    cache = rand(g, 20, page, 1, Dc + Dr).to(DEV)
    table = torch.arange(15, dtype=torch.int32, device=DEV).view(3, 5)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    kv = torch.tensor([70, 33, 1], dtype=torch.int32, device=DEV)
    pos = kv - 1
    slots = attn.cache_slots(pos, torch.arange(3, device=DEV), table, page)
    angle = torch.arange(80.0)[:, None] * 0.1 ** torch.arange(Dr // 2)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(DEV)
    q, k = rand(g, B, H, Dn + Dr).to(DEV), rand(g, B, 1, Dc + Dr).to(DEV)
    new = [(rand(g, B, H, Dn + Dr).to(DEV), rand(g, B, 1, Dc + Dr).to(DEV)) for _ in range(3)]
    ql = torch.empty(B, H, Dc + Dr, dtype=torch.bfloat16, device=DEV)
    rot = torch.empty_like(ql)
    ol, lse = torch.empty(B, H, Dc, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, device=DEV)
    y, y2 = (torch.empty(B, H, Dv, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qe = torch.empty(B, H, Dn + Dr, dtype=torch.bfloat16, device=DEV)
    lse2 = torch.empty_like(lse)
    ke, ve = (torch.zeros(B, 80, H, d, dtype=torch.bfloat16, device=DEV) for d in (Dn + Dr, Dv))
    kr, vr = (torch.zeros(B, 80, H, d, dtype=torch.bfloat16, device=DEV) for d in (Dn, Dv))
    places = torch.empty(B, 80, dtype=torch.int32, device=DEV)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)

    def layer():
        attn.latent_queries(q, w[:, :Dn], out=ql)
        attn.qk_norm_rope_append(ql, k, None, None, None, pos, cos_sin, slots, cache, None, rope_offset=Dc, q_out=rot)
        attn.dcp_paged_attn(rot, cache, None, table, cu, kv, v_dim=Dc, scale=0.1, out=ol, out_lse=lse, workspace=ws)
        attn.latent_values(ol, w[:, Dn:], out=y)
        qe[..., :Dn].copy_(q[..., :Dn])
        qe[..., Dn:].copy_(rot[..., Dc:])
        attn.dcp_latent_attn(qe, cache, w[:, :Dn], w[:, Dn:], table, cu, kv, 80, scale=0.1, out=y2, out_lse=lse2, k_out=ke,
                             v_out=ve, k_rest=kr, v_rest=vr, places=places, workspace=ws)

    layer()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        layer()
    for nq, nk in new:
        q.copy_(nq)
        k.copy_(nk)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (y, lse, y2, lse2, ke, ve)]
        layer()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, lse, y2, lse2, ke, ve)))
        assert float((y.double() - y2.double()).abs().max()) <= 0.25 and float((lse - lse2).abs().max()) <= 0.1
