"""Weights of the expanded form where rows are few: held to 2^-16 (bf16) or 2^-22 (fp16) of themselves without being asked,
as dcp_paged_attn holds them.  Tolerances: test_gpu_latent.py, with the weights' term u M as u^2 M."""
import pytest
import torch

from attn_oracle import FLOOR, U, Problem
from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dims", [(64, 16, 48, 128), (128, 64, 128, 64), (160, 64, 200, 64)])
@pytest.mark.parametrize("seqs,more", [([(1, 500), (1, 350), (1, 7)], {}), ([(3, 200), (30, 90)], {}), ([(60, 200)], dict(wide_weights=True))])
def test_few_rows(seqs, more, dims, dtype):
    Dn, Dr, Dv, Dc = dims
    H = 3
    lat = Problem(seqs, H, 1, Dc + Dr, Dc, dtype=dtype, page=16, shared=True, seed=3)
    g = torch.Generator().manual_seed(4)
    w = (torch.randn(H, Dn + Dv, Dc, generator=g) * Dc ** -0.5).to(dtype)
    q = torch.randn(lat.T, H, Dn + Dr, generator=g).to(dtype)
    wg, scale, u = w.to(DEV), (Dn + Dr) ** -0.5, U[dtype]
    out, _ = attn.dcp_latent_attn(q.to(DEV), lat.k.to(DEV), wg[:, :Dn], wg[:, Dn:], lat.table.to(DEV), lat.cu.to(DEV), lat.kv.to(DEV),
                                  int(lat.kv.max()), scale=scale, **more)
    out = out.cpu().double()
    for b, (n, _) in enumerate(seqs):
        m, row = lat.seen(b), lat.keys(b, 0)
        at = slice(int(lat.cu[b]), int(lat.cu[b]) + n)
        for h in range(H):
            key = torch.cat([row[:, :Dc] @ w[h, :Dn].double().t(), row[:, Dc:]], 1)
            val = row[:, :Dc] @ w[h, Dn:].double().t()
            mag = row[:, :Dc].abs() @ w[h].double().abs().t() * (Dc + 3) * 2.0 ** -24
            qd = q[at, h].double()
            off = torch.cat([mag[:, :Dn] + u * u * key[:, :Dn].abs() + FLOOR[dtype], 0 * row[:, Dc:]], 1)
            ds = (scale * (qd.abs() @ (off + (2 * Dn + Dr + 4) * 2.0 ** -24 * key.abs()).t()) * m).amax(1, keepdim=True)
            p = torch.softmax((scale * qd @ key.t()).masked_fill(~m, -torch.inf), 1)
            o, M = p @ val, p @ val.abs()
            # (fp16: what a weight's second product leaves, 2^-33 of a row's largest, and a value's rest that is subnormal)
            tol = (u * o.abs() + (2 * u * u + 2 * ds * (1 + 2 * ds) + 2.0 ** -20) * M * (1 + 2 * u) + p @ mag[:, Dn:] +
                   2.0 ** -33 * m.sum(1, keepdim=True) * val.abs().amax(0) + 2 * FLOOR[dtype])
            over = (out[at, h] - o).abs() / tol
            assert bool((over <= 1.0).all()), "off by %.3g of what is allowed" % float(over.max())
