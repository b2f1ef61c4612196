"""One long sequence among more short ones than the chip has workgroups for, against the 64-bit oracle."""
import math

import pytest
import torch

from attn_oracle import Problem
from test_gpu_attn import call
from test_gpu_attn_cache import mass_call
from test_gpu_attn_strict import strict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("B,at,Hkv", [(130, 0, 8), (130, 129, 8), (67, 66, 8), (70, 40, 16), (300, 200, 2)])
def test_one_long_sequence(dev, B, at, Hkv):
    """Its keys are split, which shows in the workspace, and every row is right."""
    seqs = [(1, 1 + i * 7 % 60) for i in range(B)]
    seqs[at] = (2, 1500)
    p = Problem(seqs, Hkv, Hkv, 32, 32, seed=B + at)
    ws = torch.full((1 << 24,), math.nan, device=dev)
    strict(p, call(p, dev, workspace=ws))
    assert not bool(torch.isnan(ws).all()), "no range was split"
    lse = torch.full((p.T, p.Hq), 4.0)
    before = torch.zeros(p.pages, p.page, p.Hkv)
    want, tol = p.mass(lse, before)
    got = mass_call(p, lse, before.to(dev), dev).cpu().double()
    assert bool(((got - want).abs() <= tol).all())


def test_many_rows_of_many_sequences(dev):
    """The weights' kernel for many rows where sequences fill the chip: no rows are split, and no workspace is asked for."""
    seqs = [(40, 40 + i % 30) for i in range(70)]
    seqs[50] = (40, 900)
    p = Problem(seqs, 8, 8, 32, 8, seed=1)
    lse = torch.full((p.T, p.Hq), 4.0)
    before = torch.zeros(p.pages, p.page, p.Hkv)
    want, tol = p.mass(lse, before)
    got = mass_call(p, lse, before.to(dev), dev, workspace=torch.empty(0, device=dev)).cpu().double()
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("B,at,n", [(135, 134, 1), (255, 0, 1), (270, 100, 1), (140, 70, 3)])
def test_one_long_latent_sequence(dev, B, at, n):
    """The same for latent rows, where a sequence's tokens fill row tiles of their own; shared rows of few heads."""
    seqs = [(1, 1 + i * 7 % 40) for i in range(B)]
    seqs[at] = (n, 1500)
    p = Problem(seqs, 3, 1, 576, 512, shared=True, seed=B)
    ws = torch.full((1 << 25,), math.nan, device=dev)
    strict(p, call(p, dev, workspace=ws))
    assert not bool(torch.isnan(ws).all()), "no range was split"


def test_even_batches_need_no_join(dev):
    """Nothing is split: every row is written whole, and the workspace stays as it was."""
    for kw in (dict(Hq=8, Hkv=8, Dk=32, Dv=32), dict(Hq=3, Hkv=1, Dk=576, Dv=512, shared=True)):
        p = Problem([(1, 30 + i % 7) for i in range(200)], seed=3, **kw)
        ws = torch.full((1 << 25,), math.nan, device=dev)
        strict(p, call(p, dev, workspace=ws))
        assert bool(torch.isnan(ws).all())
