"""Caches without a page: every token gets the neutral pair, whatever the columns of keys and values, and what is refused
over a cache with pages is refused over one without."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def call(fn, Dk, Dv, T, B=2):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)         # noqa: E731
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)       # noqa: E731
    args = [e(T, 4, Dk).zero_(), e(0, 16, 2, Dk), e(0, 16, 2, Dv), torch.empty(B, 0, dtype=torch.int32, device=DEV),
            i32([0] * B + [T]), i32([5] * B)]
    if fn is attn.dcp_prefix_attn:
        args += [i32([0, B]), i32([16])]
    return fn(*args)


@pytest.mark.parametrize("fn", [attn.dcp_paged_attn, attn.dcp_prefix_attn])
@pytest.mark.parametrize("T", [0, 3, 200])
@pytest.mark.parametrize("Dk,Dv", [(64, 128), (128, 64), (8, 256)])
def test_neutral_pairs(fn, Dk, Dv, T):
    out, lse = call(fn, Dk, Dv, T)
    assert out.shape == (T, 4, Dv) and bool((out == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("fn", [attn.dcp_paged_attn, attn.dcp_prefix_attn])
@pytest.mark.parametrize("Dk,Dv", [(264, 64), (64, 264)])
def test_widths_that_are_refused(fn, Dk, Dv):
    with pytest.raises(attn.AttnError):
        call(fn, Dk, Dv, 3)
