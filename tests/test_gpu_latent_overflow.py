"""Keys beyond fp16's largest number: infinite in both forms of the expansion, with a rest of 0, so that a token whose score
for such a key is -infinity goes on without it, and one whose score is +infinity is NaN, as in dcp_paged_attn."""
import math

import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rounded", [False, True])
def test_keys_beyond_the_type(rounded):
    H, Dn, Dr, Dv, Dc, KV, far = 2, 64, 16, 32, 64, 50, 17
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(H, Dn + Dv, Dc, generator=g) * Dc ** -0.5).half()
    w[:, 3, 0] = 400.0                                           # column 3 of a key: 400 times its row's first element
    rows = torch.randn(64, Dc + Dr, generator=g).half()
    rows[:, 0] *= 2.0 ** -8
    rows[far, 0] = 200.0                                         # 80000
    w[:, Dn:, 0] = 0.0                                           # (no value takes part)
    q = (torch.randn(4, H, Dn + Dr, generator=g) * 0.5).half()
    q[:2, :, 3], q[2:, :, 3] = -0.5, 0.5
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)          # noqa: E731
    buf = lambda d: torch.zeros(1, KV, H, d, dtype=torch.float16, device=DEV)       # noqa: E731
    k, v = buf(Dn + Dr), buf(Dv)
    more = {} if rounded else dict(k_rest=buf(Dn), v_rest=buf(Dv))
    wg = w.to(DEV)
    out, lse = attn.dcp_latent_attn(q.to(DEV), rows.view(4, 16, 1, -1).to(DEV), wg[:, :Dn], wg[:, Dn:], i32([[0, 1, 2, 3]]),
                                    i32([0, 4]), i32([KV]), KV, scale=0.1, causal=False, k_out=k, v_out=v, rounded=rounded, **more)
    inf = torch.zeros(KV, Dn + Dr, dtype=torch.bool)
    inf[far, 3] = True
    for h in range(H):
        assert torch.equal(torch.isinf(k[0, :, h].cpu()), inf) and not bool(torch.isnan(k).any())
        if not rounded:
            assert bool((more["k_rest"][0, far, h, 3] == 0).all()) and bool(torch.isfinite(more["k_rest"]).all())
    out, lse = out.cpu().double(), lse.cpu().double()
    assert bool(torch.isnan(out[2:]).all() and torch.isnan(lse[2:]).all())
    seen = torch.arange(KV) != far
    c, wd = rows[:KV].double()[seen], w.double()
    for h in range(H):
        key = torch.cat([c[:, :Dc] @ wd[h, :Dn].t(), c[:, Dc:]], 1)
        s = 0.1 * q[:2, h].double() @ key.t()
        val = c[:, :Dc] @ wd[h, Dn:].t()
        # every key rounded once: a score off by 2^-11 0.1 sum |q k|; weights, values and the output off by 2^-11 each
        ds = 2.0 ** -11 * 0.1 * float((q[:2, h].double().abs() @ key.abs().t()).max()) + 2.0 ** -16
        p = torch.softmax(s, 1)
        tol = (3 * 2.0 ** -11 + 2 * ds * (1 + 2 * ds)) * (p @ val.abs()) + 2.0 ** -16
        assert bool(((out[:2, h] - p @ val).abs() <= tol).all())
        assert bool(((lse[:2, h] - torch.logsumexp(s, 1)).abs() <= ds + 2.0 ** -18).all())
        assert math.isfinite(float(lse[0, h]))
