"""Accumulated weights of rows that are to give nothing, against the 64-bit
oracle (tolerances: tests/attn_oracle.py)."""
import math

import pytest
import torch

from attn_oracle import Problem
from test_gpu_attn_cache import mass_call

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


FORMS = {"few": dict(seqs=[(1, 300), (1, 40), (2, 70)], Hq=8, Hkv=2, Dk=128), "many": dict(seqs=[(70, 300), (40, 40)], Hq=4, Hkv=2, Dk=128),
         "few fp8": dict(seqs=[(1, 300), (1, 40)], Hq=8, Hkv=2, Dk=64, cache=F8), "latent": dict(seqs=[(1, 200), (3, 90)], Hq=40, Hkv=1, Dk=576),
         "split rows": dict(seqs=[(400, 500)], Hq=4, Hkv=1, Dk=64)}


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_row_without_a_sum_gives_nothing_whatever_it_holds(dev, form, what):
    """lse -inf: neither a query nor a key that is not a number reaches the weights through such a row."""
    p = Problem(Dv=8, seed=7, **FORMS[form])
    lse = torch.full((p.T, p.Hq), 5.0)
    off = torch.zeros(p.T, p.Hq, dtype=torch.bool)
    off[::3, 1] = True                      # single heads
    off[-1] = True                          # the one token that sees the last key
    lse[off] = -math.inf
    before = torch.rand(p.pages, p.page, p.Hkv, generator=torch.Generator().manual_seed(1))
    want, tol = p.mass(lse, before)
    p.q[off] = what
    page, at = p.place(p.B - 1, int(p.kv[-1]) - 1)
    p.k[page, at] = what if p.k.dtype != F8 else math.nan
    got = mass_call(p, lse, before.to(dev), dev).cpu().double()
    ok = (got - want).abs() <= tol
    assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
