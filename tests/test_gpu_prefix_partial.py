"""Groups of which no sequence holds all keys that the group is said to share (pages reserved ahead, say): what each holds
it sees, though the table rows name no page behind it."""
import pytest
import torch

from attn_oracle import Problem
from test_gpu_attn import check
from test_gpu_prefix import FORMS, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", [[40, 90, 60], [0, 17, 95, 95], [95, 20], [33]])
def test_no_sequence_holds_all(form, lens):
    Hq, Hkv, Dk, Dv, latent = FORMS[form]
    p = Problem([(1, max(n, 1)) for n in lens], Hq, Hkv, Dk, Dv, page=16, shared=latent, seed=7)
    longest = max(range(len(lens)), key=lambda b: lens[b])
    for b, n in enumerate(lens):
        p.kv[b] = n
        held = -(-n // 16)
        p.table[b, :held] = p.table[longest, :held]
        p.table[b, held:] = -1
    check(p, *call(p, torch.tensor([0, len(lens)], dtype=torch.int32), torch.tensor([96], dtype=torch.int32)))


def test_no_sequence_of_many_holds_all():
    """Beyond the entries that the list keeps at hand."""
    B = 1100
    p = Problem([(1, 10 + b % 80) for b in range(B)], 1, 1, 16, 16, page=16, seed=8)
    long = max(range(B), key=lambda b: int(p.kv[b]))
    for b in range(B):
        held = -(-int(p.kv[b]) // 16)
        p.table[b, :held] = p.table[long, :held]
        p.table[b, held:] = -1
    check(p, *call(p, torch.tensor([0, B], dtype=torch.int32), torch.tensor([96], dtype=torch.int32)))
