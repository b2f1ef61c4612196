"""dcp_batch_plan with the longest free list there may be, full or nearly so: pages that come back beyond its end are lost,
whatever count + pages amounts to in 32 bits, and all else is as the plain loops have it."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("room", [0, 1, 5, 4000])
def test_pages_that_come_back_to_a_list_of_nearly_2_31(room, gaps):
    most, held, need = 2 ** 31 - 1, 3000, 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)         # noqa: E731
    free = torch.full((most,), -9, dtype=torch.int32, device=DEV)
    count = most - room
    free[count - 10:count] = torch.arange(10, dtype=torch.int32, device=DEV)       # (its last pages: 0 .. 9)
    table = torch.full((2, held), -1, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(100, 100 + held, dtype=torch.int32, device=DEV)
    if gaps:
        table[0, 1::3] = -1
    back = [x for x in table[0].tolist() if x >= 0]
    kept = back[:room]
    plan = attn.dcp_batch_plan(i32([-1, need]), i32([held, 0]), i32([held, 0]), table, free, i32([count]), 8, 1)
    stack = list(range(10)) + kept                                                 # from count - 10 on
    taken = [stack[-1 - i] for i in range(need)]
    assert int(plan.free_count) == count + len(kept) - need
    assert table[1, :need + 1].tolist() == taken + [-1]
    assert plan.slots.tolist() == taken + [-1] * 6
    assert plan.seq_len.tolist() == [0, need] and plan.kv_len.tolist() == [0, need] and plan.cu_q.tolist() == [0, 0, need]
    assert free[count - 10:count + len(kept)].tolist() == stack
    assert bool((free[:count - 10] == -9).all()) and bool((free[count + len(kept):] == -9).all())
