"""dcp_latent_attn over caches whose scale is far from 1, against the definition in 64 bits: keys and values are of order 1
to 100 while the cached rows, or their products with the weights, are far larger or smaller.

Tolerances as in test_gpu_latent.py; what is written is a key divided by f, k_scale = f 2^p, so the half of the smallest
subnormal that it may be off by counts f times (beyond the powers that the call goes to, k_scale / 2^p times)."""
import math

import pytest
import torch

from attn_oracle import FLOOR, U
from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
H, Dn, Dr, Dv, Dc, PAGE, KV, T = 3, 64, 32, 48, 64, 16, 70, 20

# cache type, scale, size of the cached rows, of the weights (standard deviations)
SCALES = [(F8, 1e-3, 200.0, 40.0), (F8, 2.0 ** -10, 200.0, 10.0), (F8, 3e-5, 200.0, 100.0), (F8, 2.0 ** -20, 200.0, 60.0),
          (F8, 281.0, 2.0 ** -7, 0.125), (F8, 2.0 ** 12, 2.0 ** -7, 0.0625), (F8, 1.5, 1.0, 0.125), (F8, 0.3, 1.0, 0.125),
          (None, 2.0 ** -9, 900.0, 10.0), (None, 1.0, 1.0, 0.125), (None, 5.0, 1.0, 0.125)]


@pytest.mark.parametrize("mode", ["parts", "rounded"])
@pytest.mark.parametrize("dtype", [HF, BF], ids=["fp16", "bf16"])
@pytest.mark.parametrize("cache,ks,size,weight", SCALES)
def test_scales(cache, ks, size, weight, dtype, mode):
    g = torch.Generator().manual_seed(5)
    rows = (torch.randn(KV, Dc + Dr, generator=g) * size).clamp(-448, 448) if cache is F8 else torch.randn(KV, Dc + Dr, generator=g) * size
    rows = rows.to(cache or dtype)
    w = (torch.randn(H, Dn + Dv, Dc, generator=g) * weight).to(dtype)
    c, wd = rows.double() * ks, w.double()
    key = torch.cat([torch.einsum("jc,hnc->hjn", c[:, :Dc], wd[:, :Dn]), c[None, :, Dc:].expand(H, -1, -1)], 2)
    val = torch.einsum("jc,hnc->hjn", c[:, :Dc], wd[:, Dn:])
    sums = torch.einsum("jc,hnc->hjn", c[:, :Dc].abs(), wd.abs()) * (Dc + 3) * 2.0 ** -24
    # (scores near 1)
    q = (torch.randn(T, H, Dn + Dr, generator=g) / (key.std() * (Dn + Dr) ** 0.5)).to(dtype)
    pages = -(-KV // PAGE)
    cached = torch.zeros(pages + 1, PAGE, 1, Dc + Dr, dtype=cache or dtype)
    cached.view(-1, Dc + Dr)[PAGE:PAGE + KV] = rows
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)                  # noqa: E731
    buf = lambda d: torch.zeros(1, KV, H, d, dtype=dtype, device=DEV)               # noqa: E731
    k_out, v_out, more = buf(Dn + Dr), buf(Dv), {}
    if mode == "parts":
        more = dict(k_rest=buf(Dn), v_rest=buf(Dv))
    wg = w.to(DEV)
    out, lse = attn.dcp_latent_attn(q.to(DEV), cached.to(DEV), wg[:, :Dn], wg[:, Dn:], i32([list(range(1, pages + 1))]), i32([0, T]),
                                    i32([KV]), KV, scale=1.0, causal=False, k_scale=ks, k_out=k_out, v_out=v_out,
                                    rounded=mode == "rounded", **more)
    power = min(max(math.floor(math.log2(ks)), -15), 7 if cache is F8 else 0)
    f = ks / 2.0 ** power
    u = U[dtype]
    ur, floor = (u if mode == "rounded" else u * u), FLOOR[dtype] * f
    # what is written
    parts = [x.cpu().double()[0].transpose(0, 1) * f for x in (k_out, v_out)]
    if mode == "parts":
        parts[0][..., :Dn] += more["k_rest"].cpu().double()[0].transpose(0, 1) * f
        parts[1] += more["v_rest"].cpu().double()[0].transpose(0, 1) * f
    assert bool(((parts[0] - key)[..., :Dn].abs() <= ur * key[..., :Dn].abs() + sums[..., :Dn] * (1 + u) + floor).all())
    assert bool(((parts[1] - val).abs() <= ur * val.abs() + sums[..., Dn:] * (1 + u) + floor).all())
    exact = cache is F8 or dtype is BF or ks >= 1
    assert bool(((parts[0] - key)[..., Dn:].abs() <= (0.0 if exact else floor)).all())
    # the attention
    out, lse = out.cpu().double(), lse.cpu().double()
    for h in range(H):
        qd = q[:, h].double()
        s = qd @ key[h].t()
        off = torch.cat([ur * key[h, :, :Dn].abs() + sums[h, :, :Dn] + floor, torch.full((KV, Dr), 0.0 if exact else floor)], 1)
        ds = (qd.abs() @ (off + (2 * Dn + Dr + 4) * 2.0 ** -24 * key[h].abs()).t()).amax(1, keepdim=True)
        p = torch.softmax(s, 1)
        o, M = p @ val[h], p @ val[h].abs()
        tol = u * o.abs() + (u + ur) * M + p @ sums[h, :, Dn:] + 2 * floor + (2 * ds * (1 + 2 * ds) + 2.0 ** -20) * M * (1 + 2 * u) + FLOOR[dtype]
        assert bool(((out[:, h] - o).abs() <= tol).all()), h
        want = torch.logsumexp(s, 1)
        assert bool(((lse[:, h] - want).abs() <= ds[:, 0] + 2.0 ** -20 + 2.0 ** -22 * want.abs()).all()), h
