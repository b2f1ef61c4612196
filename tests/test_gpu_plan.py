"""dcp_batch_plan on the GPU against plain loops: every number equal."""
import random

import pytest
import torch

import plan_oracle
from attn_oracle import owned_fast
from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu


def problem(seed, B, new, seq, page, N, inter, *, ended=0.0, cut=0, short=0, width=None, rank=None, missing=0.0, spare=0):
    """Inputs as lists.  short: pages fewer on the free list than are needed; missing: table entries without a page."""
    r = random.Random(seed)
    rank = r.randrange(N) if rank is None else rank
    lens = [(-r.randint(1, 3) if r.random() < ended else r.choice([0, 1, new, r.randint(0, new)]),
             r.choice([0, r.randint(0, seq)])) for _ in range(B)]
    news, seqs = [n for n, _ in lens], [n for _, n in lens]
    kv = [max(0, owned_fast(n, rank, N, inter) - (cut if r.random() < 0.5 else 0)) for n in seqs]
    held = [-(-n // page) for n in kv]
    need = [max(0, -(-(k + owned_fast(s + max(n, 0), rank, N, inter) - owned_fast(s, rank, N, inter)) // page) - h)
            for k, s, n, h in zip(kv, seqs, news, held)]
    w = max([h + n for h, n in zip(held, need)] + [0]) + 1 if width is None else width
    total = sum(held) + sum(need) + 5
    pool = list(range(total))
    r.shuffle(pool)
    table = []
    for h in held:
        row = [pool.pop() if r.random() >= missing else -1 for _ in range(min(h, w))]
        table.append(row + [-7] * (w - len(row)))
    have = max(0, min(len(pool), sum(need) + 2 - short))
    free = pool[:have] + [-9] * (total - have + spare)
    keep = [r.randint(0, 3) for _ in range(B)]
    return dict(new=news, seq=seqs, kv=kv, keep=keep, table=table, free=free, count=have, page=page, N=N, rank=rank,
                inter=inter, width=w)


def check(p, T, *, keep=True, inplace=False, wide_table=False, repeats=1):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    B, w = len(p["new"]), p["width"]
    seq, kv, count = i32(p["seq"]), i32(p["kv"]), i32([p["count"]])
    table = torch.full((B, w + (3 if wide_table else 0)), -5, dtype=torch.int32, device="cuda")[:, :w]
    if B:
        table.copy_(torch.tensor(p["table"], dtype=torch.int32).view(B, w))
    free, new = i32(p["free"]), i32(p["new"])
    out = None
    if inplace:
        e = torch.empty
        out = attn.BatchPlan(e(B + 1, dtype=torch.int32, device="cuda"), seq, kv, count,
                             e(T, dtype=torch.int32, device="cuda"), e(T, dtype=torch.int32, device="cuda"),
                             e(T, dtype=torch.int64, device="cuda"))
    state = dict(p)
    for _ in range(repeats):
        got = attn.dcp_batch_plan(new, seq, kv, table, free, count, T, p["page"], rank=p["rank"], n_ranks=p["N"],
                                  interleave=p["inter"], keep_pages=i32(p["keep"]) if keep else None, out=out)
        want = plan_oracle.plan(state["new"], state["seq"], state["kv"], state["keep"] if keep else None, state["table"],
                                state["free"], state["count"], T, p["page"], p["N"], p["rank"], p["inter"])
        have = [got.cu_q, got.seq_len, got.kv_len, got.free_count, got.positions, got.sequence, got.slots, table, free]
        names = ["cu_q", "seq_len", "kv_len", "free_count", "positions", "sequence", "slots", "table", "free"]
        for name, x, y in zip(names, have, want):
            assert x.cpu().tolist() == (y if isinstance(y, list) else [y]), name
        if inplace:
            state.update(seq=want[1], kv=want[2], count=want[3], table=want[7], free=want[8])
    return got


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("N,inter", [(1, 1), (4, 1), (3, 5), (8, 16)])
def test_decode(page, N, inter):
    check(problem(page * N, 37, 1, 700, page, N, inter), 40)


@pytest.mark.parametrize("seed", range(6))
def test_chunks_with_ended_sequences(seed):
    check(problem(seed, 9, 300, 900, (1, 4, 16)[seed % 3], (1, 2, 8)[seed // 2], (1, 4)[seed % 2], ended=0.3), 2800)


@pytest.mark.parametrize("T", [0, 1, 100, 4096, 4097, 9000])
def test_rows_fewer_and_more_than_tokens(T):
    check(problem(T, 23, 400, 100, 16, 2, 1, ended=0.1), T)


@pytest.mark.parametrize("B", [0, 1, 64, 65, 1023, 1024, 1025, 2500])
def test_batch_sizes(B):
    check(problem(B, B, 3, 60, 4, 2, 1, ended=0.2), 3 * B + 2)


@pytest.mark.parametrize("B", [7, 1500])
def test_lists_that_run_out_and_over(B):
    check(problem(1, B, 40, 100, 4, 1, 1, short=B), 40 * B)                         # too few pages
    check(problem(2, B, 40, 100, 4, 1, 1, short=10 ** 6, ended=0.5), 40 * B)        # none but those given back
    p = problem(3, B, 5, 200, 4, 1, 1, ended=0.6)
    p["free"] = p["free"][:p["count"] + 10]                                         # no room for all that come back
    check(p, 5 * B)
    p["count"] = 10 ** 6                                                            # more than the list holds
    check(p, 5 * B)
    p["count"] = -4
    check(p, 5 * B)


def test_tables_that_are_too_narrow_and_entries_without_a_page():
    check(problem(4, 30, 50, 100, 4, 1, 1, width=20), 1500)
    check(problem(5, 30, 50, 100, 4, 2, 1, width=0), 1500)
    check(problem(6, 30, 50, 100, 4, 2, 1, missing=0.3, ended=0.3), 1500)


def test_cut_caches_and_no_kept_pages():
    check(problem(7, 30, 50, 400, 8, 2, 4, cut=37, ended=0.2), 1600)
    check(problem(8, 30, 50, 400, 8, 2, 4, cut=37, ended=0.2), 1600, keep=False)


def test_in_place_step_after_step_and_wide_tables():
    p = problem(9, 50, 1, 300, 4, 4, 1, width=200)
    check(p, 60, inplace=True, wide_table=True, repeats=12)
    check(problem(10, 1100, 2, 30, 4, 2, 1, width=60, ended=0.05), 2300, inplace=True, repeats=3)


def test_long_lengths():
    """Positions near 2^30, the longest length there is, and a page table of one wide page."""
    p = problem(11, 4, 3, 10, 16, 2, 1)
    p["seq"] = [2 ** 30 - 2, 2 ** 30 - 1, 2 ** 29, 5]
    p["kv"] = [40, 3, 2 ** 29, 5]
    p["new"] = [3, 3, 3, 2 ** 31 - 1]
    check(p, 20)


def test_a_long_prompt_takes_many_pages():
    check(problem(12, 3, 20000, 10, 1, 1, 1), 60000)


def test_slots_agree_with_cache_slots():
    p = problem(13, 20, 30, 200, 8, 4, 2)
    got = check(p, 700)
    table = torch.tensor(plan_oracle.plan(p["new"], p["seq"], p["kv"], p["keep"], p["table"], p["free"], p["count"], 700, 8, 4,
                                          p["rank"], 2)[7], dtype=torch.int32)
    want = attn.cache_slots(got.positions.cpu(), got.sequence.cpu(), table, 8, p["rank"], 4, 2)
    assert torch.equal(got.slots.cpu(), want)


def test_captured_and_replayed():
    """A step captured in place: every replay is the next step."""
    p = problem(14, 33, 1, 200, 4, 2, 1, width=120)
    p["new"] = [1] * 33
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    new, seq, kv, count, free, table = (i32(p[k]) for k in ("new", "seq", "kv", "count", "free", "table"))
    count = count.view(1)
    start = [x.clone() for x in (seq, kv, count, free, table)]
    e = torch.empty
    out = attn.BatchPlan(e(34, dtype=torch.int32, device="cuda"), seq, kv, count, e(40, dtype=torch.int32, device="cuda"),
                         e(40, dtype=torch.int32, device="cuda"), e(40, dtype=torch.int64, device="cuda"))

    def step():
        attn.dcp_batch_plan(new, seq, kv, table, free, count, 40, 4, rank=p["rank"], n_ranks=2, out=out)

    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step()
    for x, y in zip((seq, kv, count, free, table), start):
        x.copy_(y)
    state = dict(p)
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        want = plan_oracle.plan(state["new"], state["seq"], state["kv"], None, state["table"], state["free"], state["count"],
                                40, 4, 2, p["rank"], 1)
        assert out.slots.cpu().tolist() == want[6] and seq.cpu().tolist() == want[1] and table.cpu().tolist() == want[7]
        state.update(seq=want[1], kv=want[2], count=want[3], table=want[7], free=want[8])
