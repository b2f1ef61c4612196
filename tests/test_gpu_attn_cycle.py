"""A cache's life across calls: lengths updated in place by the eviction."""
import pytest
import torch

import attn_oracle as oracle
from lse_weighted_merge_dcp_amd import attn
from test_gpu_attn_cache import check_evict, evict_problem

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("lens,budget,Hkv", [([5000, 64, 0, 65, 700, 63], 64, 8), ([300] * 40, 128, 16), ([0, 0], 8, 2), ([9, 3], 1, 3)])
def test_lengths_in_place(dev, lens, budget, Hkv):
    """new_len = kv_len: the heads of a sequence are cut at different times, and every one by its old length."""
    table, dst, kv, k, v, mass = evict_problem(lens, budget, Hkv, 16, 8, BF, 16, budget)
    want_new, want_kept = oracle.evict(mass, table, kv, budget, 1, 0, mass.shape[0])
    d = lambda t: t.to(dev)  # noqa: E731
    for _ in range(3):
        length = d(kv)
        new, kept = attn.dcp_cache_evict(d(mass), d(k), d(v), d(table), length, d(dst), budget, n_sink=1, new_len=length)
        assert new is length and torch.equal(length.cpu(), want_new) and torch.equal(kept.cpu(), want_kept)
    check_evict(dev, table, dst, kv, k, v, mass, budget, 1, 0)
