"""How exactly the attention weights go into the product with the values.

A weight x goes in as hi + lo, hi = x rounded to the payload type and lo = x -
hi rounded to it: |x - hi| <= u x, so hi + lo is off by at most u^2 x (u = eps / 2
of the type: bf16 2^-16 x, fp16 2^-22 x).  fp16's lo is subnormal below 2^-14 and
off by up to 2^-25 there, 2^-33 of a row's largest weight, which the sum over its
keys takes n times.  So of the terms in attn_oracle.py the one of the weights,
u M, becomes u^2 M + 2^-33 n max |v|, and the others stay."""
import pytest
import torch

import attn_oracle as oracle
from attn_oracle import Problem
from test_gpu_attn import call

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def exact(p):
    """(out, tolerance) in 64 bits; every row sees a key."""
    G, u = p.Hq // p.Hkv, oracle.U[p.dtype]
    out = torch.zeros(p.T, p.Hq, p.Dv, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, (n, _) in enumerate(p.seqs):
        at, seen = slice(int(p.cu[b]), int(p.cu[b]) + n), p.seen(b)
        for h in range(p.Hq):
            q, k, v = p.q[at, h].double(), p.keys(b, h // G), p.values(b, h // G)
            w = torch.softmax((p.scale * (q @ k.t())).masked_fill(~seen, -torch.inf), 1)
            ds = (p.Dk + 4) * 2.0 ** -24 * p.scale * ((q.abs() @ k.abs().t()) * seen).amax(1, keepdim=True)
            M = w @ v.abs()
            out[at, h] = w @ v
            tol[at, h] = (u * out[at, h].abs() + (u * u + 2 * ds + 2.0 ** -20) * M +
                          2.0 ** -33 * seen.sum(1, keepdim=True) * v.abs().amax(0) + oracle.FLOOR[p.dtype])
    return out, tol


def check(p, dev, **kw):
    out = call(p, dev, **kw)[0].cpu().double()
    want, tol = exact(p)
    over = (out - want).abs() / tol
    assert bool((over <= 1.0).all()), "off by %.3g of what is allowed" % float(over.max())


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,cache", [(64, None), (128, None), (256, None), (128, F8), (64, F8)])
def test_few_rows(dev, D, cache, dtype):
    check(Problem([(1, 700), (1, 33), (2, 130)], 8, 2, D, D, dtype=dtype, cache=cache, seed=D), dev)


def test_few_rows_of_split_keys(dev):
    check(Problem([(1, 6000), (1, 3)], 8, 1, 128, 128, page=64, seed=2), dev)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("cache", [None, F8], ids=["16-bit", "fp8"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (40, 64), (128, 128), (72, 128), (192, 128), (192, 192), (256, 256)])
def test_many_rows_on_request(dev, Dk, Dv, cache, dtype):
    check(Problem([(70, 150), (33, 33)], 4, 2, Dk, Dv, dtype=dtype, cache=cache, page=24, seed=Dk + Dv), dev, wide_weights=True)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("cache", [None, F8], ids=["16-bit", "fp8"])
@pytest.mark.parametrize("seqs,Hq,Dk,Dv", [([(1, 300), (1, 1)], 128, 576, 512), ([(9, 150)], 40, 576, 512), ([(3, 90)], 40, 320, 256),
                                           ([(1, 2000)], 16, 576, 512)])
def test_latent_rows_on_request(dev, seqs, Hq, Dk, Dv, cache, dtype):
    check(Problem(seqs, Hq, 1, Dk, Dv, dtype=dtype, cache=cache, shared=True, seed=Hq), dev, wide_weights=True)


@pytest.mark.parametrize("shared", [False, True], ids=["grouped", "latent"])
def test_request_changes_nothing_but_the_rounding(dev, shared):
    """Missing pages, rows without keys, several ranks and growing scores: as without it, within the looser bound."""
    from test_gpu_attn import check as as_ever

    shape = (20, 1, 576, 512) if shared else (4, 1, 128, 128)
    p = Problem([(50, 50), (20, 300), (1, 7)], *shape, N=3, rank=2, shared=shared, seed=9)
    p.table[1, 2] = -1
    as_ever(p, *call(p, dev, wide_weights=True))
    p = Problem([(40, 400)], *shape, shared=shared, seed=10)
    for j in range(400):
        page, at = p.place(0, j)
        p.k[page, at] = 0.0
        p.k[page, at, :, 0] = j / 4.0
    p.q[:, :, 0] = 8.0
    as_ever(p, *call(p, dev, wide_weights=True))
