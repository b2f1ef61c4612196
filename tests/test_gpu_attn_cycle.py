"""A cache's life across calls: lengths updated in place by the eviction, weights
of new keys, and appends, attention, weights and cuts in turn."""
import pytest
import torch

import attn_oracle as oracle
from lse_weighted_merge_dcp_amd import attn, ops
from test_gpu_attn_cache import check_evict, evict_problem

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("lens,budget,Hkv", [([5000, 64, 0, 65, 700, 63], 64, 8), ([300] * 40, 128, 16), ([0, 0], 8, 2), ([9, 3], 1, 3)])
def test_lengths_in_place(dev, lens, budget, Hkv):
    """new_len = kv_len: the heads of a sequence are cut at different times, and every one by its old length."""
    table, dst, kv, k, v, mass = evict_problem(lens, budget, Hkv, 16, 8, BF, 16, budget)
    want_new, want_kept = oracle.evict(mass, table, kv, budget, 1, 0, mass.shape[0])
    d = lambda t: t.to(dev)  # noqa: E731
    for _ in range(3):
        length = d(kv)
        new, kept = attn.dcp_cache_evict(d(mass), d(k), d(v), d(table), length, d(dst), budget, n_sink=1, new_len=length)
        assert new is length and torch.equal(length.cpu(), want_new) and torch.equal(kept.cpu(), want_kept)
    check_evict(dev, table, dst, kv, k, v, mass, budget, 1, 0)


@pytest.mark.parametrize("D,pairs", [(8, False), (64, True), (128, False), (256, False), (576, True), (1024, False)])
def test_a_new_key_starts_without_weight(dev, D, pairs):
    """Weights of the rows that are written become 0, whatever lies there; all others stay."""
    g = torch.Generator().manual_seed(D)
    T, Hkv, page, pages = 37, 3, 4, 15
    q, k = torch.randn(T, 6, D, generator=g).to(BF).to(dev), torch.randn(T, Hkv, D, generator=g).to(BF).to(dev)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[5], slots[9] = -1, pages * page
    old = torch.randn(pages, page, Hkv, generator=g)
    old[0, 0], old[1, 1] = float("nan"), float("inf")
    store = torch.full((Hkv, pages, page + 3), 7.0, device=dev)     # a stride of its own for every dimension
    mass = store[:, :, 1:1 + page].permute(1, 2, 0)
    mass.copy_(old)
    kc = torch.zeros(pages, page, Hkv, D, dtype=BF, device=dev)
    cs, pos = torch.zeros(1, 0, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    for v, vc in ((None, None), (k, kc.clone())):
        attn.qk_norm_rope_append(q, k, v, None, None, pos, cs, slots.to(dev), kc, vc, interleaved=pairs, mass=mass)
        want = old.clone().view(-1, Hkv)
        want[slots[(slots >= 0) & (slots < pages * page)]] = 0.0
        assert torch.equal(torch.nan_to_num(mass.cpu(), 99.0).reshape(-1, Hkv), torch.nan_to_num(want, 99.0))
        assert bool((store[:, :, 0] == 7.0).all()) and bool((store[:, :, 1 + page:] == 7.0).all())
        mass.copy_(old)


def test_append_attend_weigh_cut_and_on(dev):
    """Three rounds of a cache through the public calls alone: slots, append, attention, merge, weights and cut, each
    against what is cached (64 bits), with pages handed out again without being cleared."""
    N, Hq, Hkv, D, page, budget, inter, B = 2, 4, 2, 64, 4, 8, 2, 2
    g = torch.Generator().manual_seed(11)
    width, pages = 12, 2 * 2 * 12 + 1
    kc, vc = (torch.randn(N, pages, page, Hkv, D, generator=g).to(BF).to(dev) for _ in range(2))
    mass = torch.full((N, pages, page, Hkv), 55.0, device=dev)     # old weights everywhere
    half = torch.arange(B * width, dtype=torch.int32, device=dev).view(B, width)
    tables = [half, half + B * width]                              # in turn, one cut's destination the next one's source
    kv = torch.zeros(N, B, dtype=torch.int32, device=dev)
    seq = torch.zeros(B, dtype=torch.int32, device=dev)
    still = torch.zeros(1, 0, device=dev)
    for turn, new in enumerate(([40, 23], [1, 3], [5, 30])):
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=g).to(BF).to(dev) for h in (Hq, Hkv, Hkv))
        n = torch.tensor(new, dtype=torch.int32, device=dev)
        cu = torch.tensor([0, new[0], T], dtype=torch.int32, device=dev)
        of = torch.repeat_interleave(torch.arange(B, device=dev), n.long())
        pos = (seq[of] + torch.arange(T, device=dev) - cu[of]).int()
        table = tables[turn % 2]
        parts, before = [], mass.clone()
        grown = torch.zeros_like(kv)
        for r in range(N):
            slots = attn.cache_slots(pos, of, table, page, r, N, inter, kv_len=kv[r], seq_len=seq)
            grown[r] = kv[r] + attn.owned_positions(seq + n, r, N, inter) - attn.owned_positions(seq, r, N, inter)
            attn.qk_norm_rope_append(q, k, v, None, None, pos, still, slots, kc[r], vc[r], mass=mass[r])
            before[r].view(-1, Hkv)[slots[slots >= 0]] = 0.0
        kv, seq = grown, seq + n
        for r in range(N):
            parts.append(attn.dcp_paged_attn(q, kc[r], vc[r], table, cu, kv[r], seq_len=seq, rank=r, n_ranks=N, interleave=inter))
        out, lse = ops.dcp_lse_combine(torch.stack([o for o, _ in parts]), torch.stack([x for _, x in parts]))
        for r in range(N):
            attn.dcp_attn_mass(q, kc[r], lse, mass[r], table, cu, kv[r], seq_len=seq, rank=r, n_ranks=N, interleave=inter)
        u = 2.0 ** -8
        for b in range(B):
            for h in range(Hq):
                kd, vd, at = [], [], []
                for r in range(N):
                    j = torch.arange(int(kv[r, b]))
                    place = (table[b].cpu().long()[j // page], j % page)
                    kd.append(kc[r].cpu().double()[place[0], place[1], h // 2])
                    vd.append(vc[r].cpu().double()[place[0], place[1], h // 2])
                for i in range(new[b]):
                    # a token sees of each rank all but the keys of the tokens behind it
                    later = [int(attn.owned_positions(int(seq[b]), r, N, inter) -
                                 attn.owned_positions(int(seq[b]) - new[b] + i + 1, r, N, inter)) for r in range(N)]
                    K = torch.cat([x[:len(x) - m] for x, m in zip(kd, later)])
                    V = torch.cat([x[:len(x) - m] for x, m in zip(vd, later)])
                    row = int(cu[b]) + i
                    x = q[row, h].cpu().double()
                    s = (K @ x) * D ** -0.5
                    w = torch.softmax(s, 0)
                    ds = float((u * 2.0 ** -8 + (D + 4) * 2.0 ** -24) * D ** -0.5 * (K.abs() @ x.abs()).max())
                    # weights, partials and the merge are rounded once each
                    assert bool(((out[row, h].cpu().double() - w @ V).abs() <= (4 * u + 2 * ds) * (w @ V.abs())).all())
                    assert abs(float(lse[row, h]) - float(torch.logsumexp(s, 0))) <= ds + 1e-5
        # every row gave the keys of all ranks a weight of 1, on top of what was there
        assert bool(((mass - before).double().sum((0, 1, 2)).cpu() - T * 2).abs().max() <= T * 2 * 2.0 ** -12)
        for r in range(N):
            want_new, want_kept = oracle.evict(mass[r].cpu(), table.cpu(), kv[r].cpu(), budget, 1, 2, pages)
            _, kept = attn.dcp_cache_evict(mass[r], kc[r], vc[r], table, kv[r], tables[(turn + 1) % 2], budget, n_sink=1,
                                           n_recent=2, new_len=kv[r])
            assert torch.equal(kv[r].cpu(), want_new) and torch.equal(kept.cpu(), want_kept)


def test_a_large_budget(dev):
    """64 sequences of 8 heads with room for 131072 keys each, 2^26 rows of the list, most of them empty."""
    lens, budget, page = [100 + b for b in range(64)], 131072, 256
    table, dst, kv, k, v, mass = evict_problem(lens, page, 8, 4, 4, torch.float32, page, 12)
    wide = torch.full((64, budget // page), -1, dtype=torch.int32)
    wide[:, :1] = dst
    d = lambda t: t.to(dev)  # noqa: E731
    kd, vd, md = d(k), d(v), d(mass)
    new, kept = attn.dcp_cache_evict(md, kd, vd, d(table), d(kv), d(wide), budget)
    assert torch.equal(new.cpu(), kv)
    for b in (0, 31, 63):
        n = lens[b]
        assert torch.equal(kept[b, :, :n].cpu(), torch.arange(n, dtype=torch.int32).expand(8, n)) and bool((kept[b, :, n:] == -1).all())
        for x, y in ((k, kd), (v, vd), (mass, md)):
            assert torch.equal(y[int(dst[b, 0]), :n].cpu(), x[int(table[b, 0]), :n])


@pytest.mark.parametrize("wide", [False, True], ids=["", "wide"])
@pytest.mark.parametrize("latent", [False, True], ids=["grouped", "latent"])
def test_a_captured_step(dev, latent, wide):
    """Slots, append, attention, weights and a cut in one graph: replayed on new inputs and lengths, with eager work
    between, it does what the eager calls do, bit for bit."""
    g = torch.Generator().manual_seed(5)
    B, page, pages, budget = 3, 16, 60, 40
    Hq, Hkv, D, Dv = (20, 1, 576, 512) if latent else (8, 2, 128, 128)
    T = 9
    d = lambda *s: torch.randn(*s, generator=g).to(BF).to(dev)  # noqa: E731
    still = torch.zeros(1, 0, device=dev)
    table = torch.randperm(pages, generator=g)[:B * 15].to(torch.int32).view(B, 15).to(dev)
    dst = torch.tensor([i for i in range(pages) if i not in table.cpu().flatten().tolist()][:3 * B], dtype=torch.int32, device=dev).view(B, 3)
    st = dict(q=d(T, Hq, D), k=d(T, Hkv, D), v=None if latent else d(T, Hkv, Dv), kc=d(pages, page, Hkv, D),
              vc=None if latent else d(pages, page, Hkv, Dv), mass=torch.rand(pages, page, Hkv, generator=g).to(dev),
              cu=torch.tensor([0, 1, 6, 8], dtype=torch.int32, device=dev), kv=torch.tensor([200, 17, 90], dtype=torch.int32, device=dev),
              pos=torch.tensor([199, 12, 13, 14, 15, 16, 88, 89, -1], dtype=torch.int32, device=dev),
              of=torch.tensor([0, 1, 1, 1, 1, 1, 2, 2, -1], device=dev))

    def step(s):
        slots = attn.cache_slots(s["pos"], s["of"], table, page)
        q = attn.qk_norm_rope_append(s["q"], s["k"], s["v"], None, None, s["pos"], still, slots, s["kc"], s["vc"], mass=s["mass"])
        out, lse = torch.zeros(T, Hq, Dv, dtype=BF, device=dev), torch.zeros(T, Hq, device=dev)
        attn.dcp_paged_attn(q, s["kc"], s["vc"], table, s["cu"], s["kv"], v_dim=Dv, wide_weights=wide, out=out, out_lse=lse)
        attn.dcp_attn_mass(q, s["kc"], lse, s["mass"], table, s["cu"], s["kv"])
        new, kept = attn.dcp_cache_evict(s["mass"], s["kc"], s["vc"], table, s["kv"], dst, budget, n_sink=1, n_recent=2, new_len=s["kv"])
        return [out, lse, kept, new] + [t for t in (s["kc"], s["vc"], s["mass"]) if t is not None]

    copy = lambda: {k: None if t is None else t.clone() for k, t in st.items()}  # noqa: E731
    step(copy())
    torch.cuda.synchronize()
    held = copy()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        got = step(held)
    for turn in range(4):
        for k in ("q", "k", "v", "kc", "vc"):
            if st[k] is not None:
                st[k].copy_(d(*st[k].shape))
        st["mass"].uniform_()
        st["kv"].copy_(torch.tensor([200 - 50 * turn, 17, 90 + turn], dtype=torch.int32))
        st["pos"][0] = 199 - 50 * turn
        for k, t in st.items():
            if t is not None:
                held[k].copy_(t)
        graph.replay()
        want = step(copy())
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), turn
