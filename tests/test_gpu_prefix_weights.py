"""How exactly the weights of shared keys go into the product with the values: where rows are few as in dcp_paged_attn, to
2^-16 (bf16) or 2^-22 (fp16) of themselves, without being asked; elsewhere on request.  Tolerances: test_gpu_attn_weights.py,
and a part's weight in the join, one fp32 exponential and product more (2^-21 M)."""
import pytest
import torch

from attn_oracle import Problem
from test_gpu_attn_weights import exact
from test_gpu_prefix import call, share

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def check(p, groups, **kw):
    cu, same = share(p, groups)
    out = call(p, cu, same, **kw)[0].cpu().double()
    want, tol = exact(p)
    G = p.Hq // p.Hkv
    for b, (n, _) in enumerate(p.seqs):
        v = torch.stack([p.values(b, h // G).abs().amax(0) for h in range(p.Hq)])
        tol[int(p.cu[b]):int(p.cu[b]) + n] += 2.0 ** -21 * v
    over = (out - want).abs() / tol
    assert bool((over <= 1.0).all()), "off by %.3g of what is allowed" % float(over.max())


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Dk,Dv,cache", [(64, 64, None), (128, 128, None), (128, 128, F8), (96, 80, None), (192, 128, None), (256, 256, None),
                                         (64, 64, F8), (256, 256, F8)])
def test_single_tokens(Dk, Dv, cache, dtype):
    p = Problem([(1, 600 + 7 * i) for i in range(9)], 8, 2, Dk, Dv, dtype=dtype, cache=cache, seed=Dk)
    check(p, [(0, 6, 512), (6, 9, 96)])


@pytest.mark.parametrize("cache", [None, F8], ids=["bf16", "fp8"])
def test_few_tokens(cache):
    p = Problem([(4, 400), (3, 300), (4, 350), (1, 290)], 16, 2, 128, 128, cache=cache, page=32, seed=3)
    check(p, [(0, 4, 256)])


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("seqs,shape", [([(70, 300), (40, 290)], (4, 2, 128, 128, False)), ([(2, 300), (1, 290)], (40, 1, 576, 512, True)),
                                        ([(60, 300), (50, 310)], (2, 1, 192, 192, False))])
def test_on_request(seqs, shape, dtype):
    Hq, Hkv, Dk, Dv, latent = shape
    p = Problem(seqs, Hq, Hkv, Dk, Dv, dtype=dtype, shared=latent, seed=Hq)
    check(p, [(0, 2, 256)], wide_weights=True)
