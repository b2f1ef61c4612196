"""Further refusals of libdcpattn's host side (no GPU): see tests/test_attn_host.py."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn
from test_attn_host import A, ALIGN, NULL, OK, SHAPE, STRIDE, VALUE, evict_call, rope_call


@pytest.mark.parametrize("shift", [-20, -4, 4, 20])
def test_evict_refuses_lengths_that_overlap_in_part(shift):
    assert evict_call(B=6, kv_len=A, new_len=A + shift) == VALUE


@pytest.mark.parametrize("over,want", [(dict(m_P=-1), STRIDE), (dict(m_S=1 << 57), STRIDE), (dict(T=1, mass=A + 2), ALIGN),
                                       (dict(mass=A, m_P=64, m_S=4, m_H=1), OK)])
def test_append_checks_the_weights(over, want):
    assert rope_call(**over) == want


def test_binding_checks_the_weights_of_an_append(monkeypatch):
    monkeypatch.setattr(attn, "_on_gpu", lambda *ts: 0)
    z = torch.zeros
    q, k, kc = z(3, 8, 64, dtype=torch.bfloat16), z(3, 2, 64, dtype=torch.bfloat16), z(4, 16, 2, 64, dtype=torch.bfloat16)
    for mass in (z(4, 16, 3), z(4, 16), z(4, 16, 2, dtype=torch.float64)):
        with pytest.raises(ValueError, match="mass"):
            attn.qk_norm_rope_append(q, k, None, None, None, z(3, dtype=torch.int32), z(1, 0), z(3, dtype=torch.int64), kc, None,
                                     mass=mass)


@pytest.mark.parametrize("over,want", [
    (dict(B=64, Hkv=8, budget=131072, dst_pages=8192), NULL), (dict(B=1 << 10, Hkv=1 << 10, budget=256, dst_pages=16), NULL),
    (dict(B=1 << 10, Hkv=1 << 10, budget=257, dst_pages=17), SHAPE), (dict(B=1 << 20, Hkv=4, budget=12, dst_pages=1), SHAPE),
    (dict(B=1 << 20, Hkv=3, budget=12, dst_pages=1), SHAPE), (dict(B=1 << 20, Hkv=2, budget=12, dst_pages=1), NULL), (dict(B=1, budget=(1 << 28) + 1, dst_pages=1 << 25), SHAPE),
])
def test_size_of_an_eviction(over, want):
    """2^31 work-items to a launch: rows take at most 32 and go four at a time, 2^28 of them, and 2^21 workgroups of
    1024, one to a sequence and head.  NULL: past the limits, and then refused for a pointer."""
    assert evict_call(**dict(dict(mass=0, kp_H=0, kp_B=0), **over)) == want


@pytest.mark.parametrize("over,want", [(dict(q_out=A, qo_T=2048), STRIDE), (dict(q_out=A, qo_H=256), STRIDE),
                                       (dict(q_out=A, qo_T=2048, T=1), NULL), (dict(q_out=A, qo_H=256, Hq=1, Hkv=1), NULL),
                                       (dict(q_out=A), NULL), (dict(q_out=2 * A, qo_T=2048), NULL)])
def test_append_in_place_needs_the_same_strides(over, want):
    """q_out = q of other strides would be written over queries that are still to be read.  (NULL: past this check.)"""
    assert rope_call(**dict(dict(T=3, slots=0), **over)) == want
