"""Refusals of dcpa_batch_plan, by the library and by the binding (no GPU; nothing is launched)."""
import re

import pytest
import torch

import plan_oracle
from lse_weighted_merge_dcp_amd import attn
from test_attn_host import ALIGN, HEADER, NULL, SHAPE, STRIDE, VALUE

A = 0x100000
GOOD = dict(new_len=A, seq_len=A + 0x1000, kv_len=A + 0x2000, keep_pages=A + 0x3000, block_table=A + 0x4000, t_B=8,
            free_pages=A + 0x8000, free_count=A + 0x9000, free_count_out=A + 0x9000, seq_out=A + 0x1000, kv_out=A + 0x2000,
            cu_q=A + 0xa000, positions=A + 0xb000, sequence=A + 0xc000, slots=A + 0xd000, B=8, T=16, max_pages=8, page_size=16,
            free_max=64, N=4, rank=1, interleave=2)


def names():
    body = re.search(r"typedef struct \{((?:(?!typedef).)*?)\} dcpa_plan_args", open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    got = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        got += [n.strip() for n in re.sub(r"^(const )?(int32_t\*|int64_t\*|int64_t) ", "", decl).split(",")]
    return got


def call(**over):
    n = names()
    assert sorted(n) == sorted(GOOD) and set(over) <= set(n)
    return attn.lib().dcpa_batch_plan(attn.PLAN_ARGS.pack(*[dict(GOOD, **over)[k] for k in n]), None)


@pytest.mark.parametrize("over,want", [
    (dict(B=-1), SHAPE), (dict(B=(1 << 20) + 1), SHAPE), (dict(T=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 26), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=1 << 21), SHAPE),
    (dict(free_max=-1), SHAPE), (dict(free_max=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(rank=4), SHAPE),
    (dict(rank=-1), SHAPE), (dict(interleave=0), SHAPE), (dict(N=1 << 20, interleave=1 << 20), SHAPE),
    (dict(t_B=-1), STRIDE), (dict(t_B=7), STRIDE), (dict(t_B=1 << 57), STRIDE),
    (dict(new_len=0), NULL), (dict(seq_len=0), NULL), (dict(kv_len=0), NULL), (dict(block_table=0), NULL),
    (dict(free_pages=0), NULL), (dict(free_count=0), NULL), (dict(free_count_out=0), NULL), (dict(seq_out=0), NULL),
    (dict(kv_out=0), NULL), (dict(cu_q=0), NULL), (dict(positions=0), NULL), (dict(sequence=0), NULL), (dict(slots=0), NULL),
    (dict(new_len=A + 2), ALIGN), (dict(cu_q=A + 0xa001), ALIGN), (dict(slots=A + 0xd004), ALIGN),
    (dict(seq_out=A + 0x1004), VALUE), (dict(kv_out=A + 0x1ffc), VALUE), (dict(kv_out=A + 0x1000), VALUE),
    (dict(seq_out=A + 0x301c), VALUE)])
def test_refusals(over, want):
    assert call(**over) == want


def test_null_struct():
    assert attn.lib().dcpa_batch_plan(None, None) == NULL


def test_binding_checks():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)       # noqa: E731
    good = [i(4), i(4), i(4), i(4, 8), i(32), i(1), 16, 16]
    with pytest.raises(ValueError, match="device tensors"):
        attn.dcp_batch_plan(*good)
    with pytest.raises(ValueError):
        attn.dcp_batch_plan(*good[:6], -1, 16)
    with pytest.raises(ValueError):
        attn.dcp_batch_plan(*good[:7], 0)


def test_oracle_by_hand():
    """Two ranks taking turns, pages of two keys, rank 1: sequence 0 (3 tokens, 1 cached) grows by 3, sequence 1 ends,
    sequence 2 starts."""
    got = plan_oracle.plan([3, -1, 2], [3, 4, 0], [1, 2, 0], [0, 0, 0], [[5, -1, -1], [6, -1, -1], [-1, -1, -1]],
                           [7, 8, -1, -1], 2, 6, 2, 2, 1, 1)
    # page 6 comes back; positions 3 and 5 are this rank's keys 1 and 2: page 5 place 1, a new page (6) place 0;
    # sequence 2's position 1 is its key 0, page 8 place 0
    assert got == ([0, 3, 3, 5], [6, 0, 2], [3, 0, 1], 1, [3, 4, 5, 0, 1, -1], [0, 0, 0, 2, 2, -1],
                   [11, -1, 12, -1, 16, -1], [[5, 6, -1], [6, -1, -1], [8, -1, -1]], [7, 8, 6, -1])
