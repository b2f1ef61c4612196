"""Further refusals of libdcpattn's host side (no GPU): see tests/test_attn_host.py."""
import pytest

from test_attn_host import A, VALUE, evict_call


@pytest.mark.parametrize("shift", [-20, -4, 4, 20])
def test_evict_refuses_lengths_that_overlap_in_part(shift):
    assert evict_call(B=6, kv_len=A, new_len=A + shift) == VALUE
