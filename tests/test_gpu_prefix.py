"""Attention behind shared prefixes (dcp_prefix_attn) against the 64-bit oracle of the attention call: what a group
shares changes how the keys are read, not the result.  Tolerances: tests/attn_oracle.py."""
import math
import random

import pytest
import torch

from attn_oracle import Problem
from lse_weighted_merge_dcp_amd import attn
from test_gpu_attn import check

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
DEV = "cuda"


def share(p, groups):
    """Let the sequences of each group (b0, b1, keys) have the group's pages in front; returns (cu_group, shared_len)."""
    cu, same = [groups[0][0] if groups else 0], []
    for b0, b1, keys in groups:
        assert b0 == cu[-1] and (keys % p.page == 0 or b1 - b0 <= 1)
        for b in range(b0, b1):
            held = -(-int(p.kv[b]) // p.page)
            n = min(keys // p.page, held) if b1 - b0 > 1 else 0
            p.table[b, :n] = p.table[b0, :n]
        cu.append(b1)
        same.append(keys)
    return torch.tensor(cu, dtype=torch.int32), torch.tensor(same, dtype=torch.int32)


def call(p, cu_group, same, **over):
    a = dict(q=p.q.to(DEV), k_cache=p.k.to(DEV), v_cache=None if p.shared else p.v.to(DEV), block_table=p.table.to(DEV),
             cu_q=p.cu.to(DEV), kv_len=p.kv.to(DEV), cu_group=cu_group.to(DEV), shared_len=same.to(DEV),
             seq_len=p.seq.to(DEV), scale=p.scale, v_dim=p.Dv, rank=p.rank, n_ranks=p.N, interleave=p.inter,
             causal=p.causal, k_scale=p.ks, v_scale=p.vs)
    a.update(over)
    return attn.dcp_prefix_attn(**a)


SHAPES = [
    # seqs, groups, Hq, Hkv, Dk, Dv
    ([(1, 70), (1, 100), (1, 65)], [(0, 3, 64)], 8, 2, 64, 64),
    ([(1, 300), (1, 290), (1, 257), (1, 40), (1, 41)], [(0, 3, 256), (3, 5, 32)], 16, 2, 128, 128),
    ([(4, 300), (3, 290), (5, 261), (1, 64), (9, 200)], [(0, 3, 240), (3, 4, 48), (4, 5, 16)], 8, 2, 128, 128),
    ([(40, 300), (70, 290), (5, 261)], [(0, 3, 144)], 6, 1, 80, 72),
    ([(1, 200), (2, 210), (1, 230), (1, 5)], [(0, 2, 192), (2, 4, 0)], 5, 5, 192, 128),
    ([(3, 150), (2, 170), (1, 133)], [(0, 3, 128)], 4, 2, 256, 240),
    ([(2, 90), (1, 95), (1, 99)], [(0, 3, 80)], 12, 3, 136, 200),
    ([(1, 17), (1, 18)], [(0, 2, 16)], 1, 1, 8, 16),
]
FORMS = {"narrow": (8, 2, 64, 64, False), "rows": (8, 2, 128, 128, False), "latent": (16, 1, 576, 512, True)}


@pytest.mark.parametrize("dtype,cache", [(BF, None), (HF, None), (BF, F8)], ids=["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i, dtype, cache):
    seqs, groups, Hq, Hkv, Dk, Dv = SHAPES[i]
    p = Problem(seqs, Hq, Hkv, Dk, Dv, dtype=dtype, cache=cache, page=16, seed=i)
    check(p, *call(p, *share(p, groups)))


@pytest.mark.parametrize("dtype,cache", [(BF, None), (HF, None), (HF, F8)], ids=["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("seqs,Hq,Dk,Dv", [([(1, 300), (1, 290), (1, 257), (1, 256)], 16, 576, 512), ([(2, 300), (5, 270)], 96, 576, 512),
                                           ([(3, 260), (1, 256)], 5, 320, 256), ([(2, 300), (1, 299)], 3, 64, 64)])
def test_latent_layout(seqs, Hq, Dk, Dv, dtype, cache):
    p = Problem(seqs, Hq, 1, Dk, Dv, dtype=dtype, cache=cache, shared=True, page=64, seed=20)
    check(p, *call(p, *share(p, [(0, len(seqs), 192)])))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("N,rank,inter", [(2, 1, 1), (4, 0, 3), (8, 7, 16)])
def test_ranks(form, N, rank, inter):
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    seqs = [(2, 400), (1, 390), (3, 407), (1, 30), (1, 1)]
    p = Problem(seqs, Hq, Hkv, Dk, Dv, page=4, N=N, rank=rank, inter=inter, shared=latent, seed=31)
    keys = min(int(p.kv[b]) for b in range(3)) // 4 * 4
    check(p, *call(p, *share(p, [(0, 3, max(0, keys - 4)), (3, 5, 0)])))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_rows_that_see_part_of_what_is_shared(form, wide):
    """Groups whose new tokens, shorter caches and padding lie within the shared keys; full attention over them."""
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    seqs = [(30, 100), (100, 110), (1, 40), (0, 64), (1, 70)]
    for causal in (True, False):
        p = Problem(seqs, Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=32, causal=causal)
        p.kv[4] = 0                                                # a padded sequence of the batch
        check(p, *call(p, *share(p, [(0, 5, 96)]), wide_weights=wide))


@pytest.mark.parametrize("form", FORMS)
def test_lengths_and_groups_at_their_limits(form):
    """Shared lengths beyond the table and below 0, empty groups, sequences outside the groups, no group, groups of one."""
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    seqs = [(1, 50), (2, 60), (1, 64), (1, 100)]
    for groups in ([(1, 3, 48)], [(0, 0, 32), (0, 2, 48), (2, 2, 16), (2, 4, 64)], [], [(3, 4, 100)], [(0, 1, 33), (1, 2, 16)]):
        p = Problem(seqs, Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=33)
        check(p, *call(p, *share(p, groups)))
    p = Problem(seqs, Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=33)
    cu, same = share(p, [(0, 1, 10 ** 9), (1, 4, 48)])
    check(p, *call(p, cu, torch.tensor([10 ** 9, 48], dtype=torch.int32)))
    p = Problem(seqs, Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=33)
    check(p, *call(p, torch.tensor([0, 4], dtype=torch.int32), torch.tensor([-5], dtype=torch.int32)))


@pytest.mark.parametrize("form", FORMS)
def test_cut_caches_and_missing_pages(form):
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    p = Problem([(1, 200), (2, 230), (1, 190)], Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=34, cut=37)
    cu, same = share(p, [(0, 3, 128)])
    p.table[:, 2] = -1
    p.table[1, 9] = p.pages + 2
    check(p, *call(p, cu, same))


@pytest.mark.parametrize("form", FORMS)
def test_padding_in_front_of_a_group(form):
    """The group's first sequences hold nothing, or less than is shared, and their table rows name no pages."""
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    p = Problem([(1, 90), (1, 40), (2, 120), (1, 100)], Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=42)
    cu, same = share(p, [(0, 4, 96)])
    p.kv[0] = 0
    p.table[0] = -1
    p.table[1, 3:] = -1
    check(p, *call(p, cu, same))


def test_more_groups_and_sequences_than_a_workgroup_has_threads():
    """Lists of more than 1024 entries, with groups across the border of what one pass holds, and padding among them."""
    r = random.Random(43)
    seqs, groups, b = [], [], 0
    while b < 1100:
        n = min(r.choice([1, 3, 40, 200]), 1100 - b)
        keys = 16 * r.randint(0, 3)
        groups.append((b, b + n, keys))
        seqs += [(r.choice([0, 1, 1]), keys + 2 + r.randint(0, 20)) for _ in range(n)]
        b += n
    p = Problem(seqs, 1, 1, 16, 16, page=16, seed=43)
    cu, same = share(p, groups)
    for g0, g1, keys in groups:
        if g1 - g0 > 2:
            p.kv[g0] = 0
            p.table[g0] = -1
    check(p, *call(p, cu, same))


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("form", FORMS)
def test_masked_places_never_reach_a_row(form, what):
    """Not finite: the shared page of which a short sequence sees the first half alone, and places behind the ends."""
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    p = Problem([(1, 100), (1, 40), (2, 120)], Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=35)
    cu, same = share(p, [(0, 3, 96)])
    for b, n in enumerate(p.kv.tolist()):
        if n % 16 and (b != 1):
            at = int(p.table[b, n // 16])
            p.k[at, n % 16:] = what
            if p.v is not None:
                p.v[at, n % 16:] = what
    check(p, *call(p, cu, same))
    # key 45: hidden from sequence 1 (40 keys), seen by the others
    page, place = p.place(0, 45)
    (p.k if latent else p.v)[page, place, 0, 3] = what
    want = p.attention()
    out, lse = call(p, cu, same)
    out, lse = out.cpu().double(), lse.cpu().double()
    row = slice(1, 2)                                           # sequence 1's
    assert bool(((out[row] - want[0][row]).abs() <= want[2][row]).all()) and bool(((lse[row] - want[1][row]).abs() <= want[3][row]).all())
    heads = slice(0, Hq // Hkv)
    if not latent:
        assert not bool(torch.isfinite(out[0, heads, 3]).any())
    else:
        assert not bool(torch.isfinite(out[0, heads]).all(-1).any())


@pytest.mark.parametrize("B", [63, 64, 65, 200])
def test_many_sequences_and_groups(B):
    r = random.Random(B)
    seqs, groups, b = [], [], 0
    while b < B:
        n = min(r.choice([1, 2, 5, 40]), B - b)
        keys = 16 * r.randint(0, 6)
        groups.append((b, b + n, keys))
        seqs += [(r.choice([0, 1, 1, 2]), keys + 3 + r.randint(0, 50)) for _ in range(n)]
        b += n
    p = Problem(seqs, 2, 1, 64, 64, page=16, seed=B, lead=2, tail=3)
    out = torch.full((p.T, 2, 64), 7.0, dtype=BF, device=DEV)
    lse = torch.full((p.T, 2), 7.0, device=DEV)
    cu, same = share(p, groups)
    check(p, *call(p, cu, same, out=out, out_lse=lse))
    assert bool((out[:2] == 7).all() and (out[-3:] == 7).all() and (lse[:2] == 7).all() and (lse[-3:] == 7).all())


@pytest.mark.parametrize("form", FORMS)
def test_long_prefix_of_many_rows(form):
    """Rows beyond a tile of a group and a join of many rows, keys split over many workgroups."""
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    seqs = [(1, 2048 + 3 * i + 1) for i in range(40)]
    p = Problem(seqs, Hq, Hkv, Dk, Dv, page=64, shared=latent, seed=36)
    check(p, *call(p, *share(p, [(0, 39, 2048), (39, 40, 0)]), is_lse_base_on_e=True))


def test_strided_tensors_and_base_2():
    p = Problem([(2, 100), (1, 90), (3, 97)], 4, 2, 64, 64, page=16, seed=37)
    cu, same = share(p, [(0, 3, 80)])
    q = torch.zeros(p.T + 1, 6, 72, dtype=BF, device=DEV)[1:, 1:5, 8:]
    q.copy_(p.q)
    k = torch.zeros(2, p.pages, 18, 72, dtype=BF, device=DEV).permute(1, 2, 0, 3)[:, 1:17, :, :64]
    k.copy_(p.k)
    v = torch.zeros(p.pages, 16, 3, 64, dtype=BF, device=DEV)[:, :, 1:]
    v.copy_(p.v)
    table = torch.zeros(3, p.table.shape[1] + 2, dtype=torch.int32, device=DEV)[:, 1:-1]
    table.copy_(p.table)
    out = torch.full((p.T, 4, 80), 5.0, dtype=BF, device=DEV)
    lse = torch.zeros(4, p.T, device=DEV).t()
    got, l = call(p, cu, same, q=q, k_cache=k, v_cache=v, block_table=table, out=out[..., 8:72], out_lse=lse, is_lse_base_on_e=False)
    check(p, got, l * math.log(2))
    assert bool((out[..., :8] == 5).all() and (out[..., 72:] == 5).all())


def test_deterministic_and_no_rows():
    p = Problem([(1, 700 + i) for i in range(20)], 8, 2, 128, 128, page=16, seed=38)
    cu, same = share(p, [(0, 20, 688)])
    a, b = call(p, cu, same), call(p, cu, same)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    e = call(p, cu, same, q=p.q[:0].to(DEV))
    assert e[0].shape == (0, 8, 128)


def test_two_streams_a_workspace_and_a_graph():
    """Calls on two streams with workspaces of their own; one captured, and replayed on new queries, caches and lengths."""
    p = Problem([(1, 300), (1, 310), (1, 305), (2, 90)], 8, 2, 128, 128, page=16, seed=39)
    cu, same = share(p, [(0, 3, 288), (3, 4, 16)])
    base = dict(q=p.q.to(DEV), k_cache=p.k.to(DEV), v_cache=p.v.to(DEV), block_table=p.table.to(DEV), cu_q=p.cu.to(DEV),
                kv_len=p.kv.to(DEV), cu_group=cu.to(DEV), shared_len=same.to(DEV), seq_len=p.seq.to(DEV), scale=p.scale)
    want = attn.dcp_prefix_attn(**base)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([attn.dcp_prefix_attn(**base) for _ in range(3)][-1])
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    streams[0].wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(streams[0]), torch.cuda.graph(g, stream=streams[0]):
        attn.dcp_prefix_attn(**base, out=out, out_lse=lse, workspace=ws)
    gen = torch.Generator().manual_seed(40)
    for step in range(3):
        base["q"].copy_(torch.randn(p.q.shape, generator=gen).to(BF))
        base["shared_len"].copy_(torch.tensor([288 - 16 * step, 16], dtype=torch.int32))
        base["kv_len"].sub_(step)
        g.replay()
        torch.cuda.synchronize()
        o, l = attn.dcp_prefix_attn(**base)
        assert torch.equal(o, out) and torch.equal(l, lse)
        ref, rl = attn.dcp_paged_attn(*[base[k] for k in ("q", "k_cache", "v_cache", "block_table", "cu_q", "kv_len")],
                                      seq_len=base["seq_len"], scale=p.scale)
        assert float((ref.float() - out.float()).abs().max()) <= 2.0 ** -5 and float((rl - lse).abs().max()) <= 2.0 ** -16


def test_binding_checks():
    p = Problem([(1, 20)], 2, 1, 64, 64, page=16, seed=41)
    for cu, same in (([0, 1, 1], [16]), ([[0, 1]], [16]), ([0, 1], [[16]])):
        with pytest.raises(ValueError):
            call(p, torch.tensor(cu, dtype=torch.int32), torch.tensor(same, dtype=torch.int32))
    with pytest.raises(ValueError):
        call(p, torch.tensor([0, 1]), torch.tensor([16], dtype=torch.int32))
    with pytest.raises(attn.AttnError):
        call(p, torch.tensor([0, 1], dtype=torch.int32), torch.tensor([16], dtype=torch.int32),
             workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
