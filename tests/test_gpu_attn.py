"""Attention over a paged cache (dcp_paged_attn) against the 64-bit oracle:
decode and chunks, grouped and latent head layouts, every column count, 8-bit
caches, several ranks with blocks of positions, cut caches, absent pages, rows
that see nothing, values that are not finite in masked places, rows outside the
sequences, strides, streams and graphs.  Tolerances: tests/attn_oracle.py."""
import math

import pytest
import torch

from attn_oracle import Problem
from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def call(p, dev, **over):
    a = dict(q=p.q.to(dev), k_cache=p.k.to(dev), v_cache=None if p.shared else p.v.to(dev),
             block_table=p.table.to(dev), cu_q=p.cu.to(dev), kv_len=p.kv.to(dev), seq_len=p.seq.to(dev),
             scale=p.scale, v_dim=p.Dv, rank=p.rank, n_ranks=p.N, interleave=p.inter, causal=p.causal, k_scale=p.ks,
             v_scale=p.vs)
    a.update(over)
    return attn.dcp_paged_attn(**a)


def check(p, out, lse, ref=None):
    want, want_l, tol, tol_l = ref or p.attention()
    out, lse = out.cpu().double(), lse.cpu().double()
    a, b = int(p.cu[0]), int(p.cu[-1])
    bad = (out - want).abs()[a:b] > tol[a:b]
    bad &= ~(torch.isnan(out[a:b]) & torch.isnan(want[a:b]))
    same_kind = torch.isnan(out[a:b]) == torch.isnan(want[a:b])
    assert bool(same_kind.all()), "NaN in other places: %s" % torch.nonzero(~same_kind)[:4].tolist()
    assert not bool(bad.any()), ("out off by %.3g where %.3g is allowed, at %s" % (
        float((out - want).abs()[a:b][bad].max()), float(tol[a:b][bad].min()), torch.nonzero(bad)[:4].tolist()))
    neutral = want_l[a:b] == -math.inf
    assert torch.equal(lse[a:b] == -math.inf, neutral)
    assert bool((out[a:b][neutral] == 0).all())
    far = (lse - want_l).abs()[a:b] > tol_l[a:b]
    far &= ~neutral & ~torch.isnan(want_l[a:b])
    assert not bool(far.any()), "lse off by %.3g" % float((lse - want_l).abs()[a:b][far].max())


SHAPES = [
    # seqs, Hq, Hkv, Dk, Dv
    ([(1, 1)], 1, 1, 64, 64),
    ([(1, 37), (1, 200), (1, 1)], 8, 2, 64, 64),
    ([(1, 300), (1, 64), (1, 65)], 16, 2, 128, 128),
    ([(1, 129), (1, 500)], 7, 1, 128, 64),
    ([(1, 70), (1, 33)], 5, 5, 80, 80),
    ([(1, 90)], 4, 2, 256, 256),
    ([(2, 40), (3, 90), (1, 17)], 8, 2, 128, 128),
    ([(5, 5), (64, 100), (33, 33)], 8, 2, 64, 64),
    ([(130, 200), (1, 64), (17, 300)], 4, 2, 128, 128),
    ([(70, 131), (129, 129)], 3, 1, 192, 128),
    ([(40, 90)], 6, 2, 256, 240),
    ([(20, 20), (1, 300)], 12, 4, 8, 16),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(dev, i, dtype):
    seqs, Hq, Hkv, Dk, Dv = SHAPES[i]
    p = Problem(seqs, Hq, Hkv, Dk, Dv, dtype=dtype, page=[16, 1, 24, 64][i % 4], seed=i)
    check(p, *call(p, dev))


LATENT = [([(1, 300), (1, 1), (1, 65)], 16, 576, 512), ([(1, 700)], 128, 576, 512), ([(3, 40), (2, 2)], 96, 576, 512),
          ([(9, 100)], 5, 320, 256), ([(2, 33)], 3, 64, 64)]


@pytest.mark.parametrize("cache", [BF, F8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(LATENT)))
def test_latent_layout(dev, i, cache):
    seqs, Hq, Dk, Dv = LATENT[i]
    p = Problem(seqs, Hq, 1, Dk, Dv, cache=cache, shared=True, page=[16, 64][i % 2], seed=20 + i)
    check(p, *call(p, dev))


def test_latent_layout_with_two_key_heads_fp16(dev):
    p = Problem([(2, 60), (1, 9)], 6, 2, 96, 64, dtype=HF, shared=True, seed=30)
    check(p, *call(p, dev))


@pytest.mark.parametrize("i,dtype", [(1, BF), (2, HF), (4, BF), (5, HF), (8, BF), (9, HF), (10, BF)])
def test_8_bit_cache(dev, i, dtype):
    seqs, Hq, Hkv, Dk, Dv = SHAPES[i]
    p = Problem(seqs, Hq, Hkv, Dk, Dv, dtype=dtype, cache=F8, page=16, seed=40 + i)
    check(p, *call(p, dev))


@pytest.mark.parametrize("Dk,Dv,Hkv", [(72, 72, 2), (64, 40, 1), (136, 128, 3), (24, 24, 1)])
def test_8_bit_rows_of_half_pieces(dev, Dk, Dv, Hkv):
    """8-bit rows that are not whole pieces of 16 bytes, in every kernel."""
    p = Problem([(1, 70), (1, 33)], 4 * Hkv, Hkv, Dk, Dv, cache=F8, seed=56)
    check(p, *call(p, dev))
    p = Problem([(40, 70), (1, 33)], 2 * Hkv, Hkv, Dk, Dv, cache=F8, dtype=HF, seed=57)
    check(p, *call(p, dev))
    p = Problem([(2, 70), (1, 33)], 5, 1, 264 + Dk, Dv, cache=F8, shared=True, seed=58)
    check(p, *call(p, dev))


@pytest.mark.parametrize("N,rank,inter", [(2, 0, 1), (2, 1, 1), (3, 2, 4), (8, 7, 16), (16, 15, 1), (4, 1, 64)])
@pytest.mark.parametrize("form", ["decode", "chunk", "latent"])
def test_ranks(dev, N, rank, inter, form):
    """Some sequences leave this rank without a key, some tokens of a chunk too."""
    if form == "decode":
        p = Problem([(1, 1), (1, 300), (1, 7), (1, 65)], 8, 2, 64, 64, N=N, rank=rank, inter=inter, seed=50)
    elif form == "chunk":
        p = Problem([(50, 50), (20, 300), (1, 7)], 4, 1, 128, 128, N=N, rank=rank, inter=inter, seed=51)
    else:
        p = Problem([(2, 2), (3, 200), (1, 1)], 20, 1, 576, 512, N=N, rank=rank, inter=inter, shared=True, seed=52)
    check(p, *call(p, dev))


@pytest.mark.parametrize("n", [1, 60])
def test_cut_cache(dev, n):
    """A cache that lost 25 keys: what is there stays visible, the new tokens in order."""
    p = Problem([(n, 140), (min(n, 9), 90)], 4, 2, 64, 64, N=2, rank=1, cut=25, seed=60)
    check(p, *call(p, dev))


def test_not_causal(dev):
    """Every token sees the whole cache (another sequence's states, say)."""
    p = Problem([(40, 40), (1, 1), (7, 7)], 4, 2, 128, 128, causal=False, cross=[77, 0, 300], seed=61)
    check(p, *call(p, dev, seq_len=None))
    p = Problem([(1, 1), (1, 1)], 8, 2, 64, 64, causal=False, cross=[131, 0], seed=62)
    check(p, *call(p, dev, seq_len=None))


def test_one_rank_needs_no_lengths(dev):
    p = Problem([(30, 90), (1, 4)], 4, 2, 64, 64, seed=63)
    check(p, *call(p, dev, seq_len=None))


def test_base_2(dev):
    p = Problem([(1, 90), (3, 50)], 8, 2, 64, 64, seed=64)
    out, lse = call(p, dev, is_lse_base_on_e=False)
    check(p, out, lse * math.log(2.0))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_long_decode_and_far_apart_scores(dev, dtype):
    """Keys split over workgroups; one row's scores span a wide range."""
    p = Problem([(1, 5000), (1, 3)], 8, 1, 64, 64, dtype=dtype, page=32, seed=65)
    p.q[0] *= 30
    check(p, *call(p, dev))


def test_growing_scores_rescale(dev):
    """Each tile's maximum lies far above the last one's."""
    p = Problem([(1, 400), (40, 400)], 4, 1, 64, 64, page=16, seed=66)
    for b in range(2):
        for j in range(int(p.kv[b])):
            page, at = p.place(b, j)
            p.k[page, at] = 0.0
            p.k[page, at, :, 0] = j / 4.0
    p.q[:, :, 0] = 8.0
    check(p, *call(p, dev))


@pytest.mark.parametrize("form", ["decode", "chunk", "latent", "fp8"])
def test_absent_pages(dev, form):
    """Table entries of -1, of num_pages and far outside: their keys are not there."""
    kw = dict(decode=dict(seqs=[(1, 300), (1, 90)]), chunk=dict(seqs=[(70, 300), (3, 90)]),
              latent=dict(seqs=[(2, 300), (1, 90)]), fp8=dict(seqs=[(1, 300), (40, 90)]))[form]
    if form == "latent":
        p = Problem(kw["seqs"], 8, 1, 576, 512, shared=True, seed=67)
    else:
        p = Problem(kw["seqs"], 8, 2, 128, 128, cache=F8 if form == "fp8" else None, seed=67)
    p.table[0, 3] = -1
    p.table[0, 7] = p.pages
    p.table[1, 0] = 2 ** 31 - 1
    p.table[1, 5] = -(2 ** 31)
    check(p, *call(p, dev))
    p.table[1, :] = -1                     # a sequence without any page: the neutral pair
    check(p, *call(p, dev))


@pytest.mark.parametrize("form", ["decode", "chunk", "latent", "two"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_masked_places_never_reach_a_row(dev, form, what):
    """Whatever lies behind the end of a sequence, in unused places and pages,
    and in keys and values that a token does not see, its row stays as it is."""
    if form == "decode":
        p = Problem([(1, 100), (1, 37)], 8, 2, 64, 64, seed=70)
    elif form == "two":
        p = Problem([(2, 100), (3, 37)], 8, 2, 64, 64, seed=70)
    elif form == "chunk":
        p = Problem([(80, 100), (37, 37)], 8, 2, 128, 128, N=2, rank=0, seed=71)
    else:
        p = Problem([(5, 100), (2, 37)], 12, 1, 576, 512, shared=True, seed=72)
    clean = p.attention()
    dirty = torch.ones(p.pages, p.page, dtype=torch.bool)
    for b in range(p.B):
        page, place, _ = p.rows(b)
        dirty[page, place] = False
    p.k[dirty] = what
    if p.v is not None:
        p.v[dirty] = what
    out, lse = call(p, dev)
    check(p, out, lse, clean)
    # the last key of each sequence is seen by the last token alone
    rows = []
    for b in range(p.B):
        n, length = p.seqs[b]
        if n > 1:
            seen = p.seen(b)
            j = int(p.kv[b]) - 1
            page, at = p.place(b, j)
            (p.k if p.v is None else p.v)[page, at, :, 3] = what
            rows += [(int(p.cu[b]) + i) for i in range(n) if not bool(seen[i, j])]
    if rows:
        out2, lse2 = call(p, dev)
        for r in rows:
            err = (out2[r].cpu().double() - clean[0][r]).abs()
            assert bool((err <= clean[2][r]).all()), (r, float(err.max()))
            assert bool(((lse2[r].cpu().double() - clean[1][r]).abs() <= clean[3][r]).all())


def test_seen_nan_makes_its_rows_nan_alone(dev):
    p = Problem([(30, 60), (1, 60)], 4, 2, 64, 64, seed=73)
    page, at = p.place(0, 45)              # seen by the tokens at positions 45 and behind: rows 15 ..
    p.v[page, at, 1, 5] = math.nan
    out, lse = call(p, dev)
    out = out.cpu()
    hit = torch.isnan(out)
    want = torch.zeros_like(hit)
    want[15:30, 2:4, 5] = True
    assert torch.equal(hit, want)
    p.v[page, at, 1, 5] = 0.0
    p.k[page, at, 0, 0] = math.nan         # a score of NaN: the whole row
    out, lse = call(p, dev)
    hit = torch.isnan(lse.cpu())
    want = torch.zeros_like(hit)
    want[15:30, 0:2] = True
    assert torch.equal(hit, want) and torch.equal(torch.isnan(out.cpu()).all(-1), want)


def test_rows_outside_the_sequences_stay(dev):
    for seqs in ([(1, 50), (1, 9)], [(40, 60), (1, 9), (0, 30), (5, 5)]):
        p = Problem(seqs, 4, 2, 64, 64, lead=3, tail=4, seed=74)
        out = torch.full((p.T, 4, 64), 7.0, dtype=BF, device=dev)
        lse = torch.full((p.T, 4), 7.0, device=dev)
        call(p, dev, out=out, out_lse=lse)
        check(p, out, lse)
        for t in (out, lse):
            t = t.float().cpu()
            assert bool((t[:3] == 7.0).all()) and bool((t[-4:] == 7.0).all())


def test_strided_tensors(dev):
    """Queries out of a fused projection, head-major caches, an output slice."""
    p = Problem([(20, 60), (1, 200)], 8, 2, 64, 64, seed=75)
    fused = torch.zeros(p.T, 8 * 64 + 24, dtype=BF, device=dev)
    q = fused[:, 8:8 + 512].view(p.T, 8, 64)
    q.copy_(p.q)
    kc = torch.empty(2, p.pages, p.page, 72, dtype=BF, device=dev)[..., :64].permute(1, 2, 0, 3)
    vc = torch.empty(p.pages, 2, p.page, 64, dtype=BF, device=dev).transpose(1, 2)
    kc.copy_(p.k)
    vc.copy_(p.v)
    out = torch.zeros(8, p.T, 66, dtype=BF, device=dev)[..., :64].transpose(0, 1)
    lse = torch.zeros(8, p.T, device=dev).t()
    table = torch.full((p.B, 40), -1, dtype=torch.int32, device=dev)[:, :p.table.shape[1]]
    table.copy_(p.table)
    check(p, *call(p, dev, q=q, k_cache=kc, v_cache=vc, out=out, out_lse=lse, block_table=table))


def test_many_sequences(dev):
    """More sequences than a wave has lanes, empty ones among them."""
    seqs = [((i * 7) % 4, 1 + (i * 13) % 90) for i in range(150)]
    seqs = [(min(n, length), length) for n, length in seqs]
    p = Problem(seqs, 4, 2, 64, 64, page=8, seed=76)
    check(p, *call(p, dev))
    p = Problem([(1, 1 + (i * 13) % 90) for i in range(130)], 16, 1, 64, 64, page=8, shared=True, seed=77)
    check(p, *call(p, dev))


@pytest.mark.parametrize("form", ["decode", "chunk", "latent"])
def test_sequences_without_tokens(dev, form):
    """A padded batch: sequences of no new tokens, with and without a cache, among the others."""
    seqs = [(0, 50), (1, 300), (0, 0), (3 if form == "decode" else 40, 340), (0, 9), (0, 0)]
    p = Problem(seqs, 8, 1, *((576, 512) if form == "latent" else (128, 128)), shared=form == "latent", seed=120)
    check(p, *call(p, dev))


def test_long_sequences_behind_64_others(dev):
    """Split keys of a sequence that is not among the first 64."""
    p = Problem([(1, 20)] * 67 + [(1, 3000), (2, 90)] + [(1, 1)] * 3, 4, 2, 64, 64, seed=121)
    check(p, *call(p, dev))
    p = Problem([(1, 9)] * 66 + [(3, 900)], 48, 1, 128, 64, shared=True, seed=122)
    check(p, *call(p, dev))


def test_many_rows_of_split_keys(dev):
    """More rows than the join has waves."""
    p = Problem([(600, 900)], 16, 1, 64, 64, seed=123)
    check(p, *call(p, dev))


@pytest.mark.parametrize("cache", [BF, F8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (192, 128), (192, 192), (160, 48), (256, 256), (64, 64), (72, 128)])
def test_row_tiles_of_every_width(dev, Dk, Dv, cache):
    """Several tiles of keys, whole ones and the diagonal's, pages that end inside them and one that is not there."""
    p = Problem([(150, 420), (37, 37)], 2, 1, Dk, Dv, cache=cache, page=24, seed=124)
    p.table[0, 3] = -1
    check(p, *call(p, dev))


def test_deterministic(dev):
    p = Problem([(1, 3000), (1, 900)], 16, 2, 128, 128, seed=78)
    a = call(p, dev)
    for _ in range(3):
        b = call(p, dev)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_two_streams_and_a_graph(dev):
    """Calls at once on two streams, and a captured call replayed on changed
    inputs with eager work between the replays."""
    ps = [Problem([(1, 2000), (1, 40)], 8, 2, 128, 128, seed=80 + i) for i in range(2)]
    refs = [p.attention() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    args = [dict(q=p.q.to(dev), k_cache=p.k.to(dev), v_cache=p.v.to(dev)) for p in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for p, s, a in zip(ps, streams, args):
            with torch.cuda.stream(s):
                got.append((p, call(p, dev, **a)))
    torch.cuda.synchronize()
    for p, (out, lse) in got:
        check(p, out, lse, refs[ps.index(p)])
    p = ps[0]
    st = {k: t.clone() for k, t in args[0].items()}
    st.update(block_table=p.table.to(dev), cu_q=p.cu.to(dev), kv_len=p.kv.to(dev), seq_len=p.seq.to(dev))
    out, lse = torch.empty(p.T, 8, 128, dtype=BF, device=dev), torch.empty(p.T, 8, device=dev)
    call(p, dev, **st, out=out, out_lse=lse)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        attn.dcp_paged_attn(**st, scale=p.scale, out=out, out_lse=lse)
    for turn in range(4):
        other = Problem([(1, 2000 - 300 * turn), (1, 40 + turn)], 8, 2, 128, 128, seed=90 + turn)
        st["q"].copy_(other.q)
        st["k_cache"][:other.pages].copy_(other.k[:p.pages]) if other.pages <= p.pages else None
        st["v_cache"][:other.pages].copy_(other.v[:p.pages]) if other.pages <= p.pages else None
        st["block_table"].fill_(-1)
        st["block_table"][:, :other.table.shape[1]] = other.table.to(dev)[:, :p.table.shape[1]]
        st["kv_len"].copy_(other.kv)
        st["seq_len"].copy_(other.seq)
        out.fill_(5.0)
        g.replay()
        eager = call(other, dev)
        torch.cuda.synchronize()
        assert other.pages <= p.pages
        check(other, out, lse)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_offsets_past_32_bits(dev):
    """A cache of more than 4 GiB: pages at its far end."""
    pages, page = 70000, 64
    kc = torch.empty(pages, page, 1, 512, dtype=BF, device=dev)    # 4.6 GB
    p = Problem([(1, 200), (3, 90)], 8, 1, 512, 256, shared=True, page=page, seed=95)
    kc[-p.pages:] = p.k.to(dev)
    table = torch.where(p.table >= 0, p.table + (pages - p.pages), p.table).to(dev)
    check(p, *call(p, dev, k_cache=kc, block_table=table))
