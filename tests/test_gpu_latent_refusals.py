"""dcp_latent_attn writes nothing where it refuses its arguments, whichever of its two parts refuses them, and takes empty
buffers."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF).to(DEV)


def layer(Dn=64, Dr=32, Dv=48, Dc=96, H=3, most=90, parts=True):
    g = torch.Generator().manual_seed(1)
    w = rand(g, H, Dn + Dv, Dc, scale=Dc ** -0.5)
    full = lambda d: torch.full((2, most, H, d), 9.0, dtype=BF, device=DEV)         # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)                  # noqa: E731
    x = dict(q=rand(g, 45, H, Dn + Dr), kv_cache=rand(g, 12, 16, 1, Dc + Dr), w_uk=w[:, :Dn], w_uv=w[:, Dn:],
             block_table=torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6), cu_q=i32([0, 37, 43]), kv_len=i32([90, 61]),
             max_keys=most, k_out=full(Dn + Dr), v_out=full(Dv), places=torch.full((2, most), -77, dtype=torch.int32, device=DEV),
             out=torch.full((45, H, Dv), 9.0, dtype=BF, device=DEV), out_lse=torch.full((45, H), 9.0, device=DEV))
    if parts:
        x.update(k_rest=full(Dn), v_rest=full(Dv))
    else:
        x["rounded"] = True
    return x


def untouched(x):
    torch.cuda.synchronize()
    return all(bool((x[n] == 9.0).all()) for n in ("k_out", "v_out", "k_rest", "v_rest", "out", "out_lse") if n in x) and \
        bool((x["places"] == -77).all())


@pytest.mark.parametrize("parts", [True, False])
@pytest.mark.parametrize("change", [
    dict(out=lambda x: x["out"][..., :40]), dict(out=lambda x: x["out"].float()), dict(out_lse=lambda x: x["out_lse"][:3]),
    dict(out=lambda x: torch.full((45, 3, 51), 9.0, dtype=BF, device=DEV)[..., 1:49]),
    dict(workspace=lambda x: torch.empty(64, dtype=torch.uint8, device=DEV)),
    dict(cu_q=lambda x: x["cu_q"][:2]), dict(cu_q=lambda x: x["cu_q"].long()), dict(seq_len=lambda x: x["kv_len"][:1]),
    dict(scale=lambda x: -1.0), dict(k_scale=lambda x: 0.0), dict(n_ranks=lambda x: 2), dict(rank=lambda x: 1),
    dict(interleave=lambda x: 0),
], ids=lambda c: next(iter(c)))
def test_refused_arguments_of_the_attention(change, parts):
    x = layer(parts=parts)
    with pytest.raises(ValueError):
        attn.dcp_latent_attn(**dict(x, **{n: f(x) for n, f in change.items()}))
    assert untouched(x)


@pytest.mark.parametrize("parts", [True, False])
def test_refused_widths(parts):
    for dims in (dict(Dn=224, Dr=40), dict(Dv=264)):
        x = layer(**dims, parts=parts)
        with pytest.raises(attn.AttnError):
            attn.dcp_latent_attn(**x)
        assert untouched(x)


@pytest.mark.parametrize("parts", [True, False])
@pytest.mark.parametrize("dims", [(64, 32, 48), (8, 8, 48)])
def test_a_rank_without_keys(parts, dims):
    """max_keys 0: every token gets the neutral pair, also where a value has more columns than a key."""
    x = layer(*dims, most=0, parts=parts)
    out, lse = attn.dcp_latent_attn(**x)
    assert bool((out[:43] == 0).all()) and bool((lse[:43] == -float("inf")).all())
    assert bool((out[43:] == 9).all()) and bool((lse[43:] == 9).all())


@pytest.mark.parametrize("parts", [True, False])
def test_one_key_to_a_sequence(parts):
    x = layer(most=1, parts=parts)
    out, lse = attn.dcp_latent_attn(**x, causal=False)
    ref = layer(parts=parts)
    ref["kv_len"] = ref["kv_len"].clamp(max=1)
    ro, rl = attn.dcp_latent_attn(**ref, causal=False)
    assert torch.equal(out, ro) and torch.equal(lse, rl)
