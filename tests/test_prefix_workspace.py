"""Which calls of dcpa_prefix_attn need a workspace for the parts of their rows, and how large a one (no GPU)."""
import pytest

from lse_weighted_merge_dcp_amd import attn
from test_attn_host import ATTN, pack


def sizes(groups, **over):
    args = pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ATTN, N=1, rank=0, **over))
    return attn.lib().dcpa_prefix_attn_workspace(args, groups), attn.lib().dcpa_paged_attn_workspace(args)


WIDE = dict(Hq=64, Hkv=8, q_T=8192, o_T=8192, l_T=64, max_pages=1 << 16, num_pages=1 << 20)


@pytest.mark.parametrize("B,T", [(1, 1), (64, 64), (24, 48000), (3, 4000)])
def test_no_groups_as_the_attention_alone(B, T):
    prefix, paged = sizes(0, **WIDE, B=B, T=T)
    assert prefix == paged >= 0


@pytest.mark.parametrize("B,T", [(24, 48000), (1, 4096), (64, 64 * 16), (4, 400)])
def test_many_rows_as_the_attention_alone(B, T):
    for groups in (1, 3):
        prefix, paged = sizes(groups, **WIDE, B=B, T=T)
        assert prefix == paged >= 0
    assert sizes(1, **WIDE, B=24, T=48000)[0] == 0


@pytest.mark.parametrize("B,T,S", [(256, 256, 32), (64, 64, 32), (48, 192, 32), (64, 640, 128), (1000, 1000, 32)])
@pytest.mark.parametrize("groups", [1, 40])
def test_the_size_that_the_header_states(B, T, S, groups):
    prefix, _ = sizes(groups, **WIDE, B=B, T=T)
    R = T * 8
    stated = 512 * 129 * 8 * (B + groups + R / S + R / 128 + 1024 / 8)
    assert 0.9 * stated <= prefix <= 1.1 * stated
