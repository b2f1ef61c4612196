"""Calls of dcp_prefix_attn that run every sequence by itself: the very numbers of dcp_paged_attn."""
import pytest
import torch

from attn_oracle import Problem
from test_gpu_attn import call as alone
from test_gpu_prefix import call, share

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("seqs,shape,groups", [
    ([(1, 100), (1, 90), (2, 120)], (8, 2, 128, 128, False), []), ([(1, 100), (3, 90)], (16, 1, 576, 512, True), []),
    ([(70, 300), (60, 290), (1, 260)], (8, 2, 128, 128, False), [(0, 3, 256)]), ([(16, 300), (16, 290)], (16, 1, 576, 512, True), [(0, 2, 256)]),
    ([(128, 300)], (1, 1, 64, 64, False), [(0, 1, 128)])])
def test_as_the_attention_alone(seqs, shape, groups):
    Hq, Hkv, Dk, Dv, latent = shape
    p = Problem(seqs, Hq, Hkv, Dk, Dv, shared=latent, seed=1)
    cu, same = share(p, groups)
    for more in ({}, dict(wide_weights=True)):
        got, want = call(p, cu, same, **more), alone(p, DEV, **more)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("tokens", [31, 32, 33])
def test_beside_the_border(tokens):
    """127, 128 and 129 rows to a sequence, on average, over caches where one sequence sees part of what is shared."""
    from test_gpu_attn import check

    p = Problem([(tokens - 1, 200), (tokens, 150), (tokens + 1, 60)], 4, 1, 64, 64, seed=2)
    check(p, *call(p, *share(p, [(0, 3, 96)])))
