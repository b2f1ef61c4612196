"""cache_slots (CPU): which cache rows new tokens get."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn


def tensors(pos, seq):
    return torch.tensor(pos), torch.tensor(seq)


@pytest.mark.parametrize("N,inter", [(1, 1), (4, 1), (3, 8)])
def test_padding_gets_no_slot(N, inter):
    """Negative positions are nobody's, on the last rank too."""
    table = torch.tensor([[5, 6], [7, 8]], dtype=torch.int32)
    pos, seq = tensors([-1, -1, -5, -16, -(1 << 31), 3], [0, 1, 0, 1, 0, 1])
    for r in range(N):
        got = attn.cache_slots(pos, seq, table, 16, r, N, inter)
        assert got[:5].tolist() == [-1] * 5
        assert int(got[5]) == (7 * 16 + 3 // (N * inter) * inter + 3 % inter if 3 // inter % N == r else -1)


def test_sequences_outside_the_table_get_no_slot():
    table = torch.tensor([[5, 6], [7, 8]], dtype=torch.int32)
    pos, seq = tensors([0, 0, 0, 1], [-1, 2, 1 << 20, 1])
    assert attn.cache_slots(pos, seq, table, 16).tolist() == [-1, -1, -1, 7 * 16 + 1]
    assert attn.cache_slots(pos, seq, table[:0], 16).tolist() == [-1] * 4
    assert attn.cache_slots(pos, seq, table[:, :0], 16).tolist() == [-1] * 4
