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


@pytest.mark.parametrize("D,pairs", [(8, False), (64, True), (128, False), (256, False), (576, True), (1024, False)])
def test_a_new_key_starts_without_weight(dev, D, pairs):
    """Weights of the rows that are written become 0, whatever lies there; all others stay."""
    g = torch.Generator().manual_seed(D)
    T, Hkv, page, pages = 37, 3, 4, 15
    q, k = torch.randn(T, 6, D, generator=g).to(BF).to(dev), torch.randn(T, Hkv, D, generator=g).to(BF).to(dev)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[5], slots[9] = -1, pages * page
    old = torch.randn(pages, page, Hkv, generator=g)
    old[0, 0], old[1, 1] = float("nan"), float("inf")
    store = torch.full((Hkv, pages, page + 3), 7.0, device=dev)     # a stride of its own for every dimension
    mass = store[:, :, 1:1 + page].permute(1, 2, 0)
    mass.copy_(old)
    kc = torch.zeros(pages, page, Hkv, D, dtype=BF, device=dev)
    cs, pos = torch.zeros(1, 0, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    for v, vc in ((None, None), (k, kc.clone())):
        attn.qk_norm_rope_append(q, k, v, None, None, pos, cs, slots.to(dev), kc, vc, interleaved=pairs, mass=mass)
        want = old.clone().view(-1, Hkv)
        want[slots[(slots >= 0) & (slots < pages * page)]] = 0.0
        assert torch.equal(torch.nan_to_num(mass.cpu(), 99.0).reshape(-1, Hkv), torch.nan_to_num(want, 99.0))
        assert bool((store[:, :, 0] == 7.0).all()) and bool((store[:, :, 1 + page:] == 7.0).all())
        mass.copy_(old)
