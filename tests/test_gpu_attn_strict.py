"""The cached-attention operators against the 64-bit oracle where a NaN may not
pass for a right answer, and on paths that only callers of other layouts take:
base-2 log-sum-exp in the weights, 8-bit appends of every kind, strided caches,
weights and tables, full attention over several ranks.  Tolerances:
tests/attn_oracle.py, and near() of test_gpu_attn_cache.py."""
import math

import pytest
import torch

import attn_oracle as oracle
from attn_oracle import Problem
from lse_weighted_merge_dcp_amd import attn
from test_gpu_attn import call
from test_gpu_attn_cache import check_evict, evict_problem, mass_call, rope_table

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def strict(p, got, ref=None):
    """Every element within its tolerance, NaN and -inf exactly where the oracle has them."""
    want, want_l, tol, tol_l = ref or p.attention()
    a, b = int(p.cu[0]), int(p.cu[-1])
    for x, w, t in ((got[0], want, tol), (got[1], want_l, tol_l)):
        x, w, t = x.cpu().double()[a:b], w[a:b], t[a:b]
        same = torch.isnan(x) & torch.isnan(w) | (x == w)
        ok = same | ((x - w).abs() <= t)       # (False for a NaN on one side, and for -inf)
        assert bool(ok.all()), (torch.nonzero(~ok)[:4].tolist(), x[~ok][:4].tolist(), w[~ok][:4].tolist())


FORMS = {
    "decode": dict(seqs=[(1, 100), (1, 37)], Hq=8, Hkv=2, Dk=64, Dv=64),
    "decode fp16": dict(seqs=[(1, 700), (1, 37)], Hq=8, Hkv=2, Dk=128, Dv=128, dtype=HF),
    "decode fp8": dict(seqs=[(1, 100), (1, 37)], Hq=8, Hkv=2, Dk=128, Dv=128, cache=F8),
    "two": dict(seqs=[(2, 100), (3, 37)], Hq=8, Hkv=2, Dk=64, Dv=64),
    "chunk": dict(seqs=[(80, 100), (37, 37)], Hq=8, Hkv=2, Dk=128, Dv=128, N=2, rank=0),
    "chunk fp8": dict(seqs=[(80, 100), (37, 37)], Hq=8, Hkv=2, Dk=128, Dv=128, cache=F8),
    "wide chunk": dict(seqs=[(80, 100)], Hq=4, Hkv=2, Dk=192, Dv=128, dtype=HF),
    "latent": dict(seqs=[(5, 100), (2, 37)], Hq=12, Hkv=1, Dk=576, Dv=512, shared=True),
    "latent fp8": dict(seqs=[(5, 100), (2, 37)], Hq=12, Hkv=1, Dk=576, Dv=512, shared=True, cache=F8),
}


def unused(p):
    """Places that belong to no cached key."""
    free = torch.ones(p.pages, p.page, dtype=torch.bool)
    for b in range(p.B):
        page, place, there = p.rows(b)
        free[page[there], place[there]] = False
    return free


def fill(cache, where, what):
    """what in the places of `where`; an 8-bit cache holds no infinity, its largest value instead."""
    if cache.dtype == F8:
        cache.view(torch.uint8)[where] = 0x7f if what != what else 0x7e if what > 0 else 0xfe
    else:
        cache[where] = what


@pytest.mark.parametrize("wide", [False, True], ids=["", "wide"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", list(FORMS))
def test_masked_places_reach_neither_output_nor_sum(dev, form, what, wide):
    p = Problem(seed=70, **FORMS[form])
    clean = p.attention()
    free = unused(p)
    fill(p.k, free, what)
    if p.v is not None:
        fill(p.v, free, what)
    strict(p, call(p, dev, wide_weights=wide), clean)
    # a key that the last token alone sees: the others' rows stay
    hit = []
    for b, (n, _) in enumerate(p.seqs):
        seen, j = p.seen(b), int(p.kv[b]) - 1
        if n > 1 and not bool(seen[0, j]):
            last = torch.zeros_like(free)
            last[p.place(b, j)] = True
            fill(p.k, last, what)
            if p.v is not None:
                fill(p.v, last, what)
            hit += [int(p.cu[b]) + i for i in range(n) if bool(seen[i, j])]
    out, lse = call(p, dev, wide_weights=wide)
    for row in hit:                            # (not compared here)
        out[row], lse[row] = clean[0][row].to(out), clean[1][row].to(lse)
    strict(p, (out, lse), clean)


@pytest.mark.parametrize("form", list(FORMS))
def test_missing_pages(dev, form):
    p = Problem(seed=71, **FORMS[form])
    p.table[0, 1], p.table[0, 2], p.table[1 % p.B, 0] = -1, p.pages, 2 ** 31 - 1
    strict(p, call(p, dev))
    p.table[0, :] = -1
    strict(p, call(p, dev))


@pytest.mark.parametrize("form", list(FORMS))
def test_a_seen_nan(dev, form):
    p = Problem(seed=72, **FORMS[form])
    page, at = p.place(0, int(p.kv[0]) // 2)
    p.k[page, at, 0, 1] = math.nan
    strict(p, call(p, dev))


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("form", list(FORMS))
def test_weights_of_masked_places(dev, form, what):
    kw = dict(FORMS[form])
    kw.update(Dv=8, shared=False)
    p = Problem(seed=73, **kw)
    lse = torch.full((p.T, p.Hq), 5.0)
    before = torch.rand(p.pages, p.page, p.Hkv, generator=torch.Generator().manual_seed(4))
    want, tol = p.mass(lse, before)
    fill(p.k, unused(p), what)
    skip = torch.zeros(p.pages, p.page, dtype=torch.bool)
    for b in range(p.B):
        page, at = p.place(b, int(p.kv[b]) - 1)
        if not bool(p.seen(b)[0, -1]):         # seen by the last token alone: its own weight is lost, no other
            one = torch.zeros_like(skip)
            one[page, at] = True
            fill(p.k, one, what)
            skip |= one
    got = mass_call(p, lse, before.to(dev), dev).cpu().double()
    ok = ((got - want).abs() <= tol) | skip[..., None]
    assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()


# ---------------------------------------------------------------------------
# other layouts
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("form", ["decode", "chunk", "latent"])
def test_weights_from_base_2(dev, form):
    kw = dict(FORMS[form])
    kw.update(Dv=8, shared=False)
    p = Problem(seed=74, **kw)
    lse = 5.0 + 0.1 * torch.randn(p.T, p.Hq, generator=torch.Generator().manual_seed(5))
    before = torch.zeros(p.pages, p.page, p.Hkv)
    two = (lse.double() / math.log(2.0)).float()
    want, tol = p.mass((two.double() * math.log(2.0)), before)
    got = mass_call(p, two, before.to(dev), dev, is_lse_base_on_e=False).cpu().double()
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("form", ["decode", "chunk", "latent", "chunk fp8"])
@pytest.mark.parametrize("N,rank", [(3, 1), (2, 0)])
def test_full_attention_over_several_ranks(dev, form, N, rank):
    """causal = False: a rank's keys are all there is, whatever the ranks' number."""
    kw = dict(FORMS[form])
    kw.update(N=N, rank=rank, causal=False, cross=[77, 300][:len(kw["seqs"])])
    p = Problem(seed=75, **kw)
    strict(p, call(p, dev))
    strict(p, call(p, dev, seq_len=None))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,Dv,off,rot", [(64, 64, 0, 64), (128, 64, 0, 128), (192, 128, 64, 128), (256, 256, 0, 256),
                                          (576, 0, 512, 64), (576, 512, 8, 200), (1024, 1000, 0, 1024), (80, 80, 0, 40)])
def test_append_to_8_bit_caches(dev, D, Dv, off, rot, pairs, dtype):
    g = torch.Generator().manual_seed(D + rot)
    T, Hq, Hkv, page, pages = 21, 3, 2, 4, 8
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    q, k, v, w = r(T, Hq, D), r(T, Hkv, D), r(T, Hkv, Dv) if Dv else None, (1 + 0.2 * r(D)).to(dtype)
    cs, pos = rope_table(50, rot), torch.randint(0, 50, (T,), generator=g).to(torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[3] = -1
    ks, vs = 0.02, 0.05
    kd, vd = (torch.zeros(pages, page, Hkv, n, device=dev).to(F8) if n else None for n in (D, Dv))
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    got = attn.qk_norm_rope_append(d(q), d(k), d(v), d(w), d(w), d(pos), d(cs), d(slots), kd, vd, rope_offset=off,
                                   interleaved=pairs, k_scale=ks, v_scale=vs)
    want = oracle.norm_rope(q, w, 1e-6, cs, pos, off, pairs)
    tol = oracle.U[dtype] * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True) + oracle.FLOOR[dtype]
    assert bool(((got.cpu().double() - want).abs() <= tol).all())
    keep = slots >= 0
    want = (oracle.norm_rope(k, w, 1e-6, cs, pos, off, pairs) / ks)[keep]
    flat = kd.cpu().float().view(-1, Hkv, D)
    err = (flat[slots[keep]].double() - want.clamp(-448, 448)).abs()
    # half a step of e4m3 (2^-4 of the value, 2^-10 in the subnormals) and the fp32 arithmetic before it
    assert bool((err <= want.abs() * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10 + want.abs().amax(-1, keepdim=True) * 2.0 ** -20).all())
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots[keep]] = False
    assert not bool(flat[rest].any())
    if Dv:
        ref = (v.float() * torch.tensor(1.0 / vs, dtype=torch.float32)).clamp(-448, 448).to(F8).float()
        assert torch.equal(vd.cpu().float().view(-1, Hkv, Dv)[slots[keep]], ref[keep])


@pytest.mark.parametrize("form", ["decode", "chunk", "latent", "decode fp8"])
def test_weights_of_strided_tensors(dev, form):
    """A head-major cache with padded rows, weights of another order, a table cut out of a wider one, lse transposed."""
    kw = dict(FORMS[form])
    kw.update(Dv=8, shared=False)
    p = Problem(seed=76, **kw)
    lse = 5.0 + 0.1 * torch.randn(p.T, p.Hq, generator=torch.Generator().manual_seed(6))
    before = torch.rand(p.pages, p.page, p.Hkv, generator=torch.Generator().manual_seed(7))
    kc = torch.zeros(p.Hkv, p.pages, p.page, p.Dk + 16, dtype=p.cache, device=dev)[..., :p.Dk].permute(1, 2, 0, 3)
    kc.copy_(p.k)
    mass = torch.full((p.Hkv, p.page, 2 * p.pages), 9.0, device=dev)
    view = mass[:, :, ::2].permute(2, 1, 0)
    view.copy_(before)
    table = torch.full((p.B, 50), -1, dtype=torch.int32, device=dev)[:, 3:3 + p.table.shape[1]]
    table.copy_(p.table)
    turned = lse.t().contiguous().to(dev).t()
    assert turned.stride() == (1, p.T)
    got = mass_call(p, turned, view, dev, k_cache=kc, block_table=table)
    want, tol = p.mass(lse, before)
    assert bool(((got.cpu().double() - want).abs() <= tol).all()) and bool((mass[:, :, 1::2] == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, F8, torch.float32], ids=["16-bit", "8-bit", "32-bit"])
@pytest.mark.parametrize("wide", [16, 8], ids=["16-byte rows", "8-byte rows"])
def test_evict_strided_tensors(dev, dtype, wide):
    es = torch.empty(0, dtype=dtype).element_size()
    table, dst, kv, k, v, mass = evict_problem([200, 60, 131], 48, 3, 64 // es, 32 // es, dtype, 16, 9)
    pad = wide // es

    def heads_first(t):
        x = torch.zeros(t.shape[2], t.shape[0], t.shape[1], t.shape[3] + pad, dtype=t.dtype, device=dev)
        x = x[..., :t.shape[3]].permute(1, 2, 0, 3)
        x.copy_(t)
        return x

    kd, vd = heads_first(k), heads_first(v)
    md = torch.zeros(mass.shape[2], mass.shape[1], mass.shape[0], device=dev).permute(2, 1, 0)
    md.copy_(mass)
    wider = lambda t: torch.full((t.shape[0], 40), -1, dtype=torch.int32, device=dev)[:, 5:5 + t.shape[1]].copy_(t)  # noqa: E731
    kept = torch.zeros(3, 3, 60, dtype=torch.int32, device=dev)[:, :, 7:55]
    plain = [t.to(dev) for t in (mass, k, v)]
    want = attn.dcp_cache_evict(plain[0], plain[1], plain[2], table.to(dev), kv.to(dev), dst.to(dev), 48, n_sink=2, n_recent=3)
    new, got = attn.dcp_cache_evict(md, kd, vd, wider(table), kv.to(dev), wider(dst), 48, n_sink=2, n_recent=3, kept=kept)
    assert got is kept and torch.equal(new, want[0]) and torch.equal(kept, want[1])
    for x, y in zip((md, kd, vd), plain):
        assert torch.equal(x.float(), y.float())
    check_evict(dev, table, dst, kv, k, v, mass, 48, 2, 3)
