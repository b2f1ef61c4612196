"""The plan, the latent projections, the expansion and the expanded and shared-prefix attention: offsets that pass 32 bits,
calls on two streams at once, rows behind the last sequence, strided tensors and the two bases of the log-sum-exp."""
import math

import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def rand(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF16).to(DEV)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def layer(seed, H=3, Dn=64, Dr=32, Dv=48, Dc=96, page=16):
    w = rand(seed, H, Dn + Dv, Dc, scale=Dc ** -0.5)
    return dict(cache=rand(seed + 1, 12, page, 1, Dc + Dr), w_uk=w[:, :Dn], w_uv=w[:, Dn:],
                table=torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6), q=rand(seed + 2, 45, H, Dn + Dr),
                cu=ints(0, 37, 43), kv=ints(90, 61))


def expanded(x, **more):
    return attn.dcp_latent_attn(x["q"], x["cache"], x["w_uk"], x["w_uv"], x["table"], x["cu"], x["kv"], 90, **more)


def test_expansion_of_far_pages_into_far_rows():
    """A cache of more than 4 GB whose last pages are used, and results more than 4 GB apart."""
    Dr, Dc, page, H, Dn, Dv = 64, 512, 64, 3, 128, 128
    pages = (1 << 32) // (page * (Dc + Dr) * 2) + 40
    cache = torch.empty(pages, page, 1, Dc + Dr, dtype=BF16, device=DEV)
    last = rand(1, 8, page, 1, Dc + Dr)
    cache[-8:] = last
    assert cache.numel() * 2 > 1 << 32
    w = rand(2, H, Dn + Dv, Dc, scale=Dc ** -0.5)
    kv = ints(200, 130)
    small = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    rests = [torch.zeros(2, 200, H, d, dtype=BF16, device=DEV) for d in (Dn, Dv)]
    k = [torch.zeros(2, 200, H, d, dtype=BF16, device=DEV) for d in (Dn + Dr, Dv)]
    attn.latent_expand(last, w[:, :Dn], w[:, Dn:], small, kv, 200, k_out=k[0], v_out=k[1], k_rest=rests[0], v_rest=rests[1])
    apart = (1 << 31) + 4096
    big = torch.zeros(apart + 200 * H * (Dn + Dr) + 64, dtype=BF16, device=DEV)
    far = [big.as_strided((2, 200, H, d), (apart, H * d, d, 1)) for d in (Dn + Dr, Dv)]
    for rest in (False, True):
        for i in range(2):                     # (keys far apart, then values)
            out = [x.clone().zero_() for x in k]
            out[i] = far[i]
            big.zero_()
            more = dict(k_rest=torch.zeros_like(rests[0]), v_rest=torch.zeros_like(rests[1])) if rest else {}
            attn.latent_expand(cache, w[:, :Dn], w[:, Dn:], small + (pages - 8), kv, 200, k_out=out[0], v_out=out[1], **more)
            assert torch.equal(out[0], k[0]) and torch.equal(out[1], k[1])
            if rest:
                assert torch.equal(more["k_rest"], rests[0]) and torch.equal(more["v_rest"], rests[1])


@pytest.mark.parametrize("T", [3, 300])
def test_products_of_far_rows(T):
    """Rows and results more than 4 GB from the first to the last."""
    H, Dn, Dr, Dc = 2, 64, 16, 128
    apart = ((1 << 31) // (T - 1) // 8 + 1) * 8
    x, w = rand(1, T, H, Dn + Dr), rand(2, H, Dn, Dc, scale=0.1)
    big = torch.zeros(apart * (T - 1) + H * (Dc + Dr), dtype=BF16, device=DEV)
    ref = attn.latent_queries(x, w)
    far = big.as_strided((T, H, Dc + Dr), (apart, Dc + Dr, 1))
    attn.latent_queries(x, w, out=far)
    assert torch.equal(far, ref)
    big.zero_()
    far = big.as_strided((T, H, Dn + Dr), (apart, Dn + Dr, 1))
    far.copy_(x)
    assert torch.equal(attn.latent_queries(far, w), ref)


@pytest.mark.parametrize("latent", [False, True])
def test_shared_keys_on_far_pages(latent):
    Hq, Hkv, D, page = (16, 1, 576, 64) if latent else (8, 2, 128, 64)
    pages = (1 << 32) // (page * Hkv * D * 2) + 40
    cache = torch.empty(pages, page, Hkv, D, dtype=BF16, device=DEV)
    last = rand(1, 16, page, Hkv, D)
    cache[-16:] = last
    table = torch.tensor([[0, 1, 2, 3, 4 + b, 10 + b] for b in range(6)], dtype=torch.int32, device=DEV)
    q, cu, kv = rand(2, 6, Hq, D), ints(*range(7)), ints(300, 384, 256, 257, 320, 290)
    v = (lambda c: None if latent else c)
    more = dict(v_dim=512) if latent else {}
    ref = attn.dcp_prefix_attn(q, last, v(last), table, cu, kv, ints(0, 6), ints(256), **more)
    got = attn.dcp_prefix_attn(q, cache, v(cache), table + (pages - 16), cu, kv, ints(0, 6), ints(256), **more)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_calls_on_two_streams_at_once():
    """Two layers' calls beside each other, each with its own outputs and fresh workspaces, give what each gives alone."""
    layers = [layer(10), layer(20)]
    plans = [dict(new=ints(*[(7 * b + s) % 5 - 1 for b in range(90)]), seq=ints(*range(90)), kv=ints(*range(90))) for s in range(2)]

    def step(x, y):
        table = torch.full((90, 8), -1, dtype=torch.int32, device=DEV)
        p = attn.dcp_batch_plan(y["new"], y["seq"], y["kv"], table, torch.arange(500, dtype=torch.int32, device=DEV), ints(500), 300, 16)
        ql = attn.latent_queries(x["q"], x["w_uk"])
        ol, l1 = attn.dcp_prefix_attn(ql, x["cache"], None, x["table"], x["cu"], x["kv"], ints(0, 1), ints(16), v_dim=96)
        vals = attn.latent_values(ol[:43], x["w_uv"])
        out, l2 = expanded(x)
        return [table, *p, ql, l1[:43], vals, out[:43], l2[:43]]

    alone = [[t.clone() for t in step(*a)] for a in zip(layers, plans)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(layers[i], plans[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, alone[i]))


@pytest.mark.parametrize("mode", ["parts", "wide", "rounded"])
def test_expanded_attention_of_strided_rows(mode):
    """Strided queries and outputs, the log-sum-exp to base 2, and rows behind the last sequence, which stay as they were."""
    x = layer(30)
    H, Dk, Dv = 3, 96, 48
    more = dict(rounded=mode == "rounded", wide_weights=mode == "wide")
    ref, rl = expanded(x, **more)
    q = torch.zeros(45, H, 2, Dk, dtype=BF16, device=DEV)[:, :, 1]
    q.copy_(x["q"])
    out = torch.full((H, 45, Dv + 8), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((H, 45), 7.0, device=DEV)
    got, gl = expanded(dict(x, q=q), is_lse_base_on_e=False, out=out.transpose(0, 1)[..., :Dv], out_lse=lse.t(), **more)
    assert torch.equal(got[:43], ref[:43])
    # (one product with 1 / ln 2, or with ln 2 the other way: a rounding of 2^-24 each, and of the constants)
    assert float((gl[:43].double() * math.log(2.0) - rl[:43].double()).abs().max()) <= 4 * 2.0 ** -24 * float(rl[:43].abs().max())
    assert bool((out[:, 43:] == 7).all() and (out[..., Dv:] == 7).all() and (lse[:, 43:] == 7).all())


@pytest.mark.parametrize("mode", ["parts", "rounded"])
def test_lengths_beyond_the_buffers(mode):
    """max_keys below a cached length: the keys behind it are as keys without a page."""
    x = layer(40)
    rounded = mode == "rounded"
    out, lse = attn.dcp_latent_attn(x["q"], x["cache"], x["w_uk"], x["w_uv"], x["table"], x["cu"], x["kv"], 64, causal=False,
                                    rounded=rounded)
    ref, rl = attn.dcp_latent_attn(x["q"], x["cache"], x["w_uk"], x["w_uv"], x["table"], x["cu"], ints(64, 61), 90, causal=False,
                                   rounded=rounded)
    assert torch.equal(out[:43], ref[:43]) and torch.equal(lse[:43], rl[:43])
