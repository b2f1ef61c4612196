"""The cache's other operators against the 64-bit oracle: norm, rotation and
append (qk_norm_rope_append), accumulated weights (dcp_attn_mass), eviction
(dcp_cache_evict), and the whole path of a layer over several ranks."""
import math

import pytest
import torch

import attn_oracle as oracle
from attn_oracle import Problem
from lse_weighted_merge_dcp_amd import attn, ops

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


# ---------------------------------------------------------------------------
# norm, rotation, append
# ---------------------------------------------------------------------------
def rope_table(P, rot):
    half = max(rot // 2, 1)
    a = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], 1).float()[:, :rot].contiguous()


def near(got, want, dtype, fp32=2.0 ** -20):
    """One rounding to dtype, plus the fp32 arithmetic: a rotated element is a
    sum of two products of normed elements, each within 2^-21 of their size."""
    scale = want.abs().amax(-1, keepdim=True)
    tol = oracle.U[dtype] * want.abs() + fp32 * scale + oracle.FLOOR.get(dtype, 2.0 ** -10)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err - tol).max()))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,Dv,nq,nk,off,rot,pairs", [
    (1, 1, 1, 64, 64, 64, 64, 0, 64, False),
    (5, 8, 2, 128, 128, 128, 128, 0, 128, False),
    (7, 6, 3, 128, 64, 128, 128, 0, 64, False),
    (33, 5, 1, 80, 80, 80, 0, 16, 64, True),
    (9, 3, 1, 576, 0, 0, 512, 512, 64, True),
    (4, 2, 2, 576, 0, 576, 576, 0, 576, False),
    (3, 2, 1, 1024, 1024, 1024, 1000, 8, 1008, False),
    (6, 4, 2, 256, 8, 0, 0, 0, 0, False),
    (2, 2, 1, 192, 256, 64, 192, 64, 128, False),
    (3, 1, 1, 8, 24, 8, 8, 0, 0, True),
    # half a range that is no whole piece of eight columns
    (9, 5, 5, 80, 80, 80, 80, 0, 40, False),
    (9, 5, 5, 80, 80, 80, 80, 0, 40, True),
    (6, 3, 1, 64, 64, 64, 40, 8, 8, False),
    (4, 2, 1, 96, 96, 0, 96, 16, 72, False),
    (3, 2, 1, 576, 0, 576, 512, 24, 200, False),
    (3, 2, 2, 8, 8, 8, 8, 0, 8, False),
])
def test_norm_rope(dev, dtype, T, Hq, Hkv, D, Dv, nq, nk, off, rot, pairs):
    g = torch.Generator().manual_seed(T * D)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    page, pages = 4, T // 3 + 2
    q, k = r(T, Hq, D), r(T, Hkv, D)
    v = r(T, Hkv, Dv) if Dv else None
    wq, wk = (1 + 0.2 * r(nq)).to(dtype) if nq else None, (1 + 0.2 * r(nk)).to(dtype) if nk else None
    cs = rope_table(50, rot)
    pos = torch.randint(0, 50, (T,), generator=g).to(torch.int32)
    pos[0] = 49
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 2] = -1
    if T > 2:
        slots[1] = pages * page            # behind the cache: skipped too
    kc, vc = r(pages, page, Hkv, D), r(pages, page, Hkv, Dv) if Dv else None
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    kd, vd = d(kc), d(vc)
    got = attn.qk_norm_rope_append(d(q), d(k), d(v), d(wq), d(wk), d(pos), d(cs), d(slots), kd, vd, rope_offset=off,
                                   interleaved=pairs, eps=1e-5)
    near(got.cpu(), oracle.norm_rope(q, wq, 1e-5, cs, pos, off, pairs), dtype)
    want = oracle.norm_rope(k, wk, 1e-5, cs, pos, off, pairs)
    keep = (slots >= 0) & (slots < pages * page)
    flat, kflat = kd.cpu().view(-1, Hkv, D), kc.clone().view(-1, Hkv, D)
    near(flat[slots[keep]], want[keep], dtype)
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots[keep]] = False
    assert torch.equal(flat[rest], kflat[rest])
    if Dv:
        vflat = vc.clone().view(-1, Hkv, Dv)
        vflat[slots[keep]] = v[keep]
        assert torch.equal(vd.cpu().view(-1, Hkv, Dv), vflat)


def test_norm_rope_8_bit_cache(dev):
    g = torch.Generator().manual_seed(3)
    T, Hq, Hkv, D, page, pages = 40, 4, 2, 128, 16, 4
    q, k, v = (torch.randn(T, h, D, generator=g).to(BF) for h in (Hq, Hkv, Hkv))
    v[3] *= 1000.0                          # saturates
    v[4, 0, 0] = math.nan
    v[4, 0, 1], v[4, 0, 2] = math.inf, -math.inf
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(BF)
    cs, pos = rope_table(64, D), torch.arange(T, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    ks, vs = 0.02, 0.05
    kd, vd = (torch.zeros(pages, page, Hkv, D, dtype=F8, device=dev) for _ in range(2))
    attn.qk_norm_rope_append(q.to(dev), k.to(dev), v.to(dev), w.to(dev), w.to(dev), pos.to(dev), cs.to(dev),
                             slots.to(dev), kd, vd, k_scale=ks, v_scale=vs)
    want = oracle.norm_rope(k, w, 1e-6, cs, pos, 0, False) / ks
    got = kd.cpu().float().view(-1, Hkv, D)[slots].double()
    err = (got - want.clamp(-448, 448)).abs()
    # half a step of e4m3 (2^-4 of the value, 2^-10 in the subnormals) and the fp32 arithmetic before it
    assert bool((err <= want.abs() * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10 + want.abs().amax(-1, keepdim=True) * 2.0 ** -20).all())
    x = v.float() * torch.tensor(1.0 / vs, dtype=torch.float32)
    ref = x.clamp(-448, 448).to(F8)
    got = vd.cpu().view(torch.uint8).view(-1, Hkv, D)[slots].view(F8)
    nan = torch.isnan(ref.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(got.float()[~nan], ref.float()[~nan])


def test_norm_rope_in_place_strided_and_far_positions(dev):
    g = torch.Generator().manual_seed(4)
    T, Hq, Hkv, D = 11, 4, 2, 64
    fused = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g).to(HF)
    view = lambda f: (f[:, :Hq * D].view(T, Hq, D), f[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),  # noqa: E731
                      f[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D))
    q, k, v = view(fused)
    fd = fused.to(dev)
    qd, kd, vd = view(fd)
    cs = rope_table(100, D)
    pos = torch.tensor([-5, 0, 99, 100, 1 << 30] + [7] * 6, dtype=torch.int32)    # outside: the nearest row
    slots = torch.arange(T)
    kc = torch.zeros(2, Hkv, 16, D, dtype=HF, device=dev).transpose(1, 2)
    vc = torch.zeros(2, 16, Hkv, D + 8, dtype=HF, device=dev)[..., :D]
    got = attn.qk_norm_rope_append(qd, kd, vd, None, None, pos.to(dev), cs.to(dev), slots.to(dev), kc, vc, q_out=qd)
    assert got.data_ptr() == fd.data_ptr()
    near(got.cpu(), oracle.norm_rope(q, None, 0, cs, pos, 0, False), HF)
    near(kc.cpu().reshape(-1, Hkv, D)[:T], oracle.norm_rope(k, None, 0, cs, pos, 0, False), HF)
    assert torch.equal(vc.cpu().reshape(-1, Hkv, D)[:T], v)
    assert torch.equal(fd.cpu()[:, Hq * D:], fused[:, Hq * D:])


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,off,rot", [(64, 0, 64), (256, 0, 256), (576, 64, 512), (1024, 0, 1024), (512, 480, 32), (80, 0, 40),
                                       (576, 8, 520), (128, 0, 104)])
def test_norm_rope_in_place_of_every_width(dev, D, off, rot, pairs):
    """In place and into a tensor of its own give the same bits: no piece is read after it was turned."""
    g = torch.Generator().manual_seed(D)
    T, Hq = 300, 3
    q, k = torch.randn(T, Hq, D, generator=g).to(BF), torch.randn(T, 1, D, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(BF)
    cs, pos = rope_table(64, rot), torch.randint(0, 64, (T,), generator=g).to(torch.int32)
    d = lambda t: t.to(dev)  # noqa: E731
    qd, kc, slots = d(q), torch.zeros(T, 1, 1, D, dtype=BF, device=dev), torch.arange(T, device=dev)
    kw = dict(rope_offset=off, interleaved=pairs)
    apart = attn.qk_norm_rope_append(qd, d(k), None, d(w), d(w), d(pos), d(cs), slots, kc, None, **kw)
    near(apart.cpu(), oracle.norm_rope(q, w, 1e-6, cs, pos, off, pairs), BF)
    attn.qk_norm_rope_append(qd, d(k), None, d(w), d(w), d(pos), d(cs), slots, kc, None, q_out=qd, **kw)
    assert torch.equal(qd, apart)


def test_norm_without_rotation_needs_no_positions(dev, monkeypatch):
    """The C call with null positions and table."""
    g = torch.Generator().manual_seed(9)
    q, k = torch.randn(7, 2, 64, generator=g).to(BF), torch.randn(7, 1, 64, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(64, generator=g)).to(BF)
    cs, pos = torch.zeros(1, 0), torch.zeros(7, dtype=torch.int32)
    d = lambda t: t.to(dev)  # noqa: E731
    kc = torch.zeros(7, 1, 1, 64, dtype=BF, device=dev)

    def without(fn, name, device, args):
        fields = list(attn.ROPE_ARGS.unpack(args))
        fields[11] = fields[12] = 0            # positions, cos_sin
        assert fn(attn.ROPE_ARGS.pack(*fields), torch.cuda.current_stream().cuda_stream) == 0

    monkeypatch.setattr(attn, "_call", without)
    got = attn.qk_norm_rope_append(d(q), d(k), None, d(w), d(w), d(pos), d(cs), torch.arange(7, device=dev), kc, None)
    near(got.cpu(), oracle.norm_rope(q, w, 1e-6, cs, pos, 0, False), BF)
    near(kc.view(7, 1, 64).cpu(), oracle.norm_rope(k, w, 1e-6, cs, pos, 0, False), BF)


def test_norm_rope_of_more_rows_than_a_launch(dev):
    """2^23 workgroups of 32 rows of 8 columns: the tokens behind them go to a second launch."""
    Hq, D = 512, 8
    per = (32 << 23) // (Hq + 2)
    T = per + 5
    q = torch.randn(T, Hq, D, dtype=BF, device=dev)
    k, v = torch.randn(T, 1, D, dtype=BF, device=dev), torch.randn(T, 1, D, dtype=BF, device=dev)
    w = torch.full((D,), 1.5, dtype=BF, device=dev)
    cs, pos = rope_table(4, 0).to(dev), torch.zeros(T, dtype=torch.int32, device=dev)
    kc, vc = torch.zeros(T, 1, 1, D, dtype=BF, device=dev), torch.zeros(T, 1, 1, D, dtype=BF, device=dev)
    slots = torch.arange(T, device=dev)
    got = attn.qk_norm_rope_append(q, k, v, w, w, pos, cs, slots, kc, vc)
    at = torch.tensor([0, 1, per - 1, per, per + 1, T - 1])
    for x, y in ((q, got), (k, kc.view(T, 1, D))):
        near(y[at.to(dev)].cpu(), oracle.norm_rope(x[at.to(dev)].cpu(), w.cpu(), 1e-6, cs.cpu(), pos[:6].cpu(), 0, False), BF)
    assert torch.equal(vc.view(T, 1, D), v)


# ---------------------------------------------------------------------------
# accumulated weights
# ---------------------------------------------------------------------------
def mass_call(p, lse, mass, dev, **over):
    a = dict(q=p.q.to(dev), k_cache=p.k.to(dev), lse=lse.to(dev), mass=mass, block_table=p.table.to(dev),
             cu_q=p.cu.to(dev), kv_len=p.kv.to(dev), seq_len=p.seq.to(dev), scale=p.scale, rank=p.rank, n_ranks=p.N,
             interleave=p.inter, causal=p.causal, k_scale=p.ks)
    a.update(over)
    return attn.dcp_attn_mass(**a)


def check_mass(p, lse, dev, seed=0, **over):
    g = torch.Generator().manual_seed(seed)
    before = torch.rand(p.pages, p.page, p.Hkv, generator=g) * 0.01
    got = mass_call(p, lse, before.to(dev), dev, **over).cpu().double()
    want, tol = p.mass(lse, before)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    err = (got - want).abs()
    bad = (err > tol) & ~nan
    assert not bool(bad.any()), (float(err[bad].max()), float(tol[bad].min()), torch.nonzero(bad)[:4].tolist())
    untouched = torch.ones(p.pages, p.page, dtype=torch.bool)
    for b in range(p.B):
        page, place, there = p.rows(b)
        untouched[page[there], place[there]] = False
    assert torch.equal(got[untouched], before.double()[untouched])


MASS = [
    dict(seqs=[(1, 1), (1, 300), (1, 129)], Hq=8, Hkv=2, Dk=64),
    dict(seqs=[(1, 200)], Hq=7, Hkv=1, Dk=128, dtype=HF),
    dict(seqs=[(40, 90), (3, 3), (1, 500)], Hq=4, Hkv=2, Dk=128, N=2, rank=1),
    dict(seqs=[(130, 300)], Hq=8, Hkv=1, Dk=80, cache=F8, page=24),
    dict(seqs=[(3, 100), (1, 40)], Hq=40, Hkv=1, Dk=576, N=3, rank=2, inter=4),
    dict(seqs=[(20, 20)], Hq=6, Hkv=2, Dk=256, dtype=HF, page=1),
    dict(seqs=[(1, 70)] * 70, Hq=2, Hkv=1, Dk=8, page=8),
    dict(seqs=[(50, 60)], Hq=2, Hkv=2, Dk=576, cache=F8),
    dict(seqs=[(9, 9), (5, 5)], Hq=4, Hkv=2, Dk=64, causal=False, cross=[200, 0]),
    dict(seqs=[(60, 140)], Hq=4, Hkv=2, Dk=64, N=2, rank=0, cut=25),
    dict(seqs=[(1, 90), (1, 700)], Hq=16, Hkv=2, Dk=128, cache=F8),
    dict(seqs=[(1, 90), (1, 33)], Hq=4, Hkv=2, Dk=72, cache=F8),
    dict(seqs=[(1, 90), (1, 33)], Hq=4, Hkv=1, Dk=192, dtype=HF, cache=F8, page=4),
    dict(seqs=[(9, 90), (0, 3), (0, 40), (0, 7)], Hq=8, Hkv=1, Dk=64, page=4),   # many rows in one sequence of few
    dict(seqs=[(1, 3000)], Hq=8, Hkv=1, Dk=64, page=16),
    dict(seqs=[(1, 40)] * 66 + [(50, 600)], Hq=7, Hkv=1, Dk=128, page=16),
    dict(seqs=[(300, 700), (33, 1400)], Hq=6, Hkv=2, Dk=128, N=2, rank=1, inter=16),
    dict(seqs=[(97, 97)], Hq=5, Hkv=5, Dk=256, dtype=HF),
]


@pytest.mark.parametrize("i", range(len(MASS)))
def test_mass(dev, i):
    p = Problem(Dv=8, seed=100 + i, lead=i % 3, tail=i % 2, **MASS[i])
    lse = torch.full((p.T, p.Hq), math.nan)
    for b, (n, length) in enumerate(p.seqs):
        lse[int(p.cu[b]):int(p.cu[b + 1])] = math.log(max(length, int(p.kv[b]), 1)) + 0.5
    g = torch.Generator().manual_seed(i)
    lse += 0.1 * torch.randn(lse.shape, generator=g)
    lse[int(p.cu[0]), 0] = -math.inf        # this row saw nothing anywhere
    check_mass(p, lse, dev, i)


@pytest.mark.parametrize("token", [0, 20, 39])
def test_mass_of_a_row_without_a_sum(dev, token):
    """A row whose log-sum-exp is NaN gives NaN to the keys that it sees and nothing to those that it does not."""
    p = Problem([(40, 340)], 4, 1, 64, 8, seed=140)
    lse = torch.full((p.T, p.Hq), 6.0)
    lse[int(p.cu[0]) + token, 2] = math.nan
    mass = torch.zeros(p.pages, p.page, 1, device=dev)
    got = mass_call(p, lse, mass, dev).cpu()
    page, place, _ = p.rows(0)
    assert torch.equal(torch.isnan(got[page, place, 0]), torch.arange(340) <= 300 + token)


def test_mass_sums_to_one_over_the_ranks(dev):
    """With the merged log-sum-exp, the weights of every row over all ranks sum to 1."""
    N, total = 4, 0.0
    seqs = [(5, 5), (17, 300), (1, 2)]
    lses, parts = [], []
    for r in range(N):
        p = Problem(seqs, 8, 2, 64, 64, N=N, rank=r, seed=111)
        parts.append(p)
        a = dict(q=p.q.to(dev), k_cache=p.k.to(dev), v_cache=p.v.to(dev), block_table=p.table.to(dev),
                 cu_q=p.cu.to(dev), kv_len=p.kv.to(dev), seq_len=p.seq.to(dev), rank=r, n_ranks=N)
        parts[-1].q = parts[0].q
        a["q"] = parts[0].q.to(dev)
        lses.append(attn.dcp_paged_attn(**a)[1])
    merged = torch.logsumexp(torch.stack(lses).double(), 0).float()
    for p in parts:
        m = mass_call(p, merged, torch.zeros(p.pages, p.page, 2, device=dev), dev)
        total = total + m.double().sum((0, 1)).cpu()
    rows = sum(n for n, _ in seqs) * 4
    assert bool((total - rows).abs().max() <= rows * 2.0 ** -18), total


@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_mass_of_masked_places(dev, what):
    p = Problem([(30, 60), (1, 20)], 4, 2, 64, 8, seed=112)
    lse = torch.full((p.T, 4), 4.0)
    before = torch.zeros(p.pages, p.page, 2)
    want, tol = p.mass(lse, before)
    dirty = torch.ones(p.pages, p.page, dtype=torch.bool)
    for b in range(p.B):
        page, place, _ = p.rows(b)
        dirty[page, place] = False
    p.k[dirty] = what
    page, at = p.place(0, 59)               # seen by the last token alone
    p.k[page, at] = what
    got = mass_call(p, lse, before.to(dev), dev).cpu().double()
    far = (got - want).abs() > tol
    far[page, at] = False
    assert not bool(far.any())


def test_mass_missing_pages_and_graph(dev):
    p = Problem([(60, 200), (2, 50)], 4, 1, 128, 8, seed=113)
    p.table[0, 2], p.table[0, 5], p.table[1, 1] = -1, p.pages, 1 << 30
    lse = torch.full((p.T, 4), 4.0)
    check_mass(p, lse, dev)
    before = torch.rand(p.pages, p.page, 1)
    mass = before.to(dev)
    st = dict(q=p.q.to(dev), k_cache=p.k.to(dev), lse=lse.to(dev), block_table=p.table.to(dev), cu_q=p.cu.to(dev),
              kv_len=p.kv.to(dev), seq_len=p.seq.to(dev))
    once = attn.dcp_attn_mass(mass=before.to(dev), scale=p.scale, **st) - before.to(dev)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        attn.dcp_attn_mass(mass=mass, scale=p.scale, **st)
    for turn in range(3):
        mass.copy_(before)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(mass, attn.dcp_attn_mass(mass=before.to(dev), scale=p.scale, **st)), turn
    assert float(once.sum()) > 0


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def evict_problem(lens, budget, Hkv, Dk, Dv, dtype, page, seed):
    g = torch.Generator().manual_seed(seed)
    need, new = [-(-n // page) for n in lens], -(-budget // page)
    pages = sum(need) + len(lens) * new + 1
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    dst = torch.empty(len(lens), new, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
        for i in range(new):
            dst[b, i] = order.pop()
    k = torch.randn(pages, page, Hkv, Dk, generator=g).to(dtype)
    v = torch.randn(pages, page, Hkv, Dv, generator=g).to(dtype) if Dv else None
    mass = torch.exp(2 * torch.randn(pages, page, Hkv, generator=g))
    return table, dst, torch.tensor(lens, dtype=torch.int32), k, v, mass


def bits(t):
    return t.view(torch.uint8) if t.dtype == F8 else t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


def check_evict(dev, table, dst, kv, k, v, mass, budget, sink, recent):
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    kd, vd, md = d(k), d(v), d(mass)
    new, kept = attn.dcp_cache_evict(md, kd, vd, d(table), d(kv), d(dst), budget, n_sink=sink, n_recent=recent)
    pages, page, Hkv = mass.shape
    want_new, want_kept = oracle.evict(mass, table, kv, budget, sink, recent, pages)
    assert torch.equal(new.cpu(), want_new)
    assert torch.equal(kept.cpu(), want_kept)
    pools = [(bits(x).clone(), bits(y.cpu())) for x, y in ((k, kd), (v, vd), (mass, md)) if x is not None]
    empty = torch.tensor(-math.inf).view(torch.int32).item()
    for b in range(table.shape[0]):
        for h in range(Hkv):
            for i in range(int(want_new[b])):
                j = int(want_kept[b, h, i])
                src, to = int(table[b, j // page]), int(dst[b, i // page])
                if not 0 <= to < pages:
                    continue
                for n, (x, _) in enumerate(pools):
                    last = n == len(pools) - 1
                    x[to, i % page, h] = x[src, j % page, h] if 0 <= src < pages else (empty if last else 0)
    for x, y in pools:
        assert torch.equal(x, y)


@pytest.mark.parametrize("lens,budget,Hkv,Dk,Dv,dtype,page,sink,recent", [
    ([1], 1, 1, 8, 8, BF, 16, 0, 0),
    ([100, 64, 65, 0, 63], 64, 2, 64, 64, BF, 16, 0, 0),
    ([500, 33], 32, 3, 128, 64, HF, 24, 4, 8),
    ([300], 128, 1, 576, 0, F8, 16, 0, 128),
    ([2000, 1025, 3000], 1024, 2, 16, 8, BF, 64, 1, 1),
    ([200], 50, 2, 4, 2, torch.float32, 1, 50, 0),
    ([77, 80], 40, 1, 40, 24, F8, 5, 10, 30),
])
def test_evict(dev, lens, budget, Hkv, Dk, Dv, dtype, page, sink, recent):
    table, dst, kv, k, v, mass = evict_problem(lens, budget, Hkv, Dk, Dv, dtype, page, sum(lens))
    check_evict(dev, table, dst, kv, k, v, mass, budget, sink, recent)


def test_evict_ties_and_special_weights(dev):
    """Equal weights keep the oldest; NaN above +infinity, both zeros equal."""
    table, dst, kv, k, v, mass = evict_problem([900, 1500], 300, 2, 16, 16, BF, 16, 5)
    g = torch.Generator().manual_seed(6)
    mass = torch.randint(0, 4, mass.shape, generator=g).float() * torch.where(torch.rand(mass.shape, generator=g) < 0.5, -1.0, 1.0)
    mass[torch.rand(mass.shape, generator=g) < 0.02] = math.nan
    mass[torch.rand(mass.shape, generator=g) < 0.02] = -math.nan
    mass[torch.rand(mass.shape, generator=g) < 0.02] = math.inf
    mass[torch.rand(mass.shape, generator=g) < 0.02] = -math.inf
    check_evict(dev, table, dst, kv, k, v, mass, 300, 3, 5)
    check_evict(dev, table, dst, kv, k, v, torch.zeros_like(mass), 300, 3, 5)


def test_evict_long(dev):
    """More keys than a workgroup holds in registers: 70000, with ties across the turns."""
    L, budget, page = 70000, 40000, 64
    table, dst, kv, k, v, mass = evict_problem([L], budget, 1, 8, 0, BF, page, 8)
    mass = torch.randint(0, 50, mass.shape, generator=torch.Generator().manual_seed(1)).float()
    md, kd = mass.to(dev), k.to(dev)
    new, kept = attn.dcp_cache_evict(md, kd, None, table.to(dev), kv.to(dev), dst.to(dev), budget, n_sink=3, n_recent=9)
    j = torch.arange(L)
    w = mass[table[0].long()[j // page], j % page, 0].double()
    w[:3] = w[L - 9:] = math.inf
    want = torch.argsort(-w, stable=True)[:budget].sort().values
    assert int(new[0]) == budget and torch.equal(kept[0, 0].cpu().long(), want)
    i = torch.arange(budget)
    got = kd.cpu()[dst[0].long()[i // page], i % page, 0]
    assert torch.equal(got.view(torch.int16), k[table[0].long()[want // page], want % page, 0].view(torch.int16))


def test_evict_bad_pages(dev):
    table, dst, kv, k, v, mass = evict_problem([300, 200], 64, 2, 16, 16, BF, 16, 7)
    table[0, 2], table[0, 3], table[1, 0] = -1, mass.shape[0], 1 << 30
    dst[0, 1], dst[1, 3] = -5, mass.shape[0]
    check_evict(dev, table, dst, kv, k, v, mass, 64, 40, 4)


# ---------------------------------------------------------------------------
# a layer's path
# ---------------------------------------------------------------------------
def test_layer_over_several_ranks(dev):
    """New tokens normed, rotated and cached on the ranks that own them,
    attention on every rank, pack and merge, the weights from the merged
    log-sum-exp, caches cut, and a second step over the cut caches: each
    against the whole computed in 64 bits."""
    from lse_weighted_merge_dcp_amd import sim

    N, Hq, Hkv, D, page, inter = 4, 8, 2, 64, 8, 2
    layer = sim.StackedAttention(N, Hq, Hkv, D, D, page_size=page, pages=40, sequences=2, max_pages=8,
                                 dtype=BF, device=dev, interleave=inter)
    g = torch.Generator().manual_seed(9)
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(BF).to(dev) for _ in range(2))
    cs = rope_table(256, D).to(dev)
    lens = [0, 0]
    keys, values = [[], []], [[], []]       # what a single rank would hold, in 64 bits as cached

    def step(new):
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=g).to(BF).to(dev) for h in (Hq, Hkv, Hkv))
        out, lse = layer.step(q, k, v, new, wq, wk, cs, eps=1e-6)
        at = 0
        for b, n in enumerate(new):
            pos = torch.arange(lens[b], lens[b] + n)
            lens[b] += n
            qr = oracle.norm_rope(q[at:at + n].cpu(), wq.cpu(), 1e-6, cs.cpu(), pos, 0, False).to(BF).double()
            kr = oracle.norm_rope(k[at:at + n].cpu(), wk.cpu(), 1e-6, cs.cpu(), pos, 0, False).to(BF).double()
            keys[b] += list(kr)
            values[b] += list(v[at:at + n].cpu().double())
            K, V = torch.stack(keys[b]), torch.stack(values[b])
            for i in range(n):
                seen = lens[b] - n + i + 1
                for h in range(Hq):
                    s = (K[:seen, h // 4] @ qr[i, h]) * D ** -0.5
                    w = torch.softmax(s, 0)
                    want = w @ V[:seen, h // 4]
                    M = w @ V[:seen, h // 4].abs()
                    err = (out[at + i, h].cpu().double() - want).abs()
                    # q, k may round the other way (2 u of |q||k|); weights, partials, merge: u M each
                    u = 2.0 ** -8
                    ds = float((2 * u * D ** -0.5 * (K[:seen, h // 4].abs() @ qr[i, h].abs())).max())
                    assert bool((err <= 4 * u * M + 2 * ds * M).all()), (b, i, h, float(err.max()))
                    assert abs(float(lse[at + i, h]) - float(torch.logsumexp(s, 0))) <= ds + 1e-5
            at += n
        return q

    step([30, 5])
    step([1, 1])
    step([4, 60])
    # every row gave the keys of all ranks a weight of 1
    rows = (30 + 5 + 2 + 64) * 4
    got = sum(layer.mass[r].double().sum((0, 1)) for r in range(N)).cpu()
    assert bool(((got - rows).abs() <= rows * 2.0 ** -12).all()), got
    before = layer.kv_len.cpu().clone()
    layer.evict(budget=6, n_sink=1, n_recent=2)
    assert torch.equal(layer.kv_len.cpu(), before.clamp(max=6))
    # a step over the cut caches against attention over what is cached
    q, k, v = (torch.randn(2, h, D, generator=g).to(BF).to(dev) for h in (Hq, Hkv, Hkv))
    out, lse = layer.step(q, k, v, [1, 1], wq, wk, cs, eps=1e-6)
    for b in range(2):
        qr = oracle.norm_rope(q[b:b + 1].cpu(), wq.cpu(), 1e-6, cs.cpu(), [lens[b]], 0, False).to(BF).double()
        for h in range(Hq):
            K, V = [], []
            for r in range(N):
                for j in range(int(layer.kv_len[r, b])):
                    pg = int(layer.table[r, b, j // page])
                    K.append(layer.k_cache[r, pg, j % page, h // 4].cpu().double())
                    V.append(layer.v_cache[r, pg, j % page, h // 4].cpu().double())
            K, V = torch.stack(K), torch.stack(V)
            s = (K @ qr[0, h]) * D ** -0.5
            w = torch.softmax(s, 0)
            u = 2.0 ** -8
            ds = float((u * D ** -0.5 * (K.abs() @ qr[0, h].abs())).max())
            assert bool(((out[b, h].cpu().double() - w @ V).abs() <= (4 * u + 2 * ds) * (w @ V.abs())).all())
            assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= ds + 1e-5


def test_partial_feeds_the_pack(dev):
    """The attention's neutral rows and LSE go through pack and combine as they are."""
    N = 4
    seqs = [(1, 2), (1, 90)]
    parts = [Problem(seqs, 8, 2, 64, 64, N=N, rank=r, seed=120) for r in range(N)]
    q = parts[0].q.to(dev)
    out = torch.empty(N, 2, 8, 64, dtype=BF, device=dev)
    lse = torch.empty(N, 2, 8, device=dev)
    for r, p in enumerate(parts):
        attn.dcp_paged_attn(q, p.k.to(dev), p.v.to(dev), p.table.to(dev), p.cu.to(dev), p.kv.to(dev),
                            seq_len=p.seq.to(dev), rank=r, n_ranks=N, out=out[r], out_lse=lse[r])
    assert bool((lse[2:, 0] == -math.inf).all()) and bool((out[2:, 0] == 0).all())
    merged, g = ops.dcp_lse_combine(out, lse)
    want = torch.logsumexp(lse.double(), 0)
    assert bool(((g.double() - want).abs() <= 1e-5).all())
    w = torch.exp(lse.double() - want)[..., None]
    assert bool(((merged.double() - (w * out.double()).sum(0)).abs() <= 2.0 ** -7 * (w * out.double().abs()).sum(0) + 1e-30).all())
