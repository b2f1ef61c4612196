"""Plain definition of dcpa_batch_plan: lists and loops over sequences, pages and tokens."""
from attn_oracle import owned_fast

LONGEST = 2 ** 30 - 1


def plan(new, seq, kv, keep, table, free, count, T, page, N, rank, inter):
    """All arguments are Python ints and lists; returns (cu, seq, kv, count, positions, sequence, slots, table, free)."""
    own = lambda x: owned_fast(x, rank, N, inter)      # noqa: E731
    B, table, free = len(new), [list(r) for r in table], list(free)
    width = len(table[0]) if table else 0
    pages = lambda keys: min(-(-keys // page), width)  # noqa: E731
    count = min(max(count, 0), len(free))
    for b in range(B):
        if new[b] < 0:
            for i in range(keep[b] if keep else 0, pages(kv[b])):
                if table[b][i] >= 0 and count < len(free):
                    free[count] = table[b][i]
                    count += 1
    cu, seq2, kv2 = [0], [], []
    positions, sequence, slots = [-1] * T, [-1] * T, [-1] * T
    for b in range(B):
        n = max(0, min(new[b], T - cu[-1], LONGEST - seq[b]))
        first = cu[-1]
        cu.append(first + n)
        if new[b] < 0:
            seq2.append(0)
            kv2.append(0)
            continue
        seq2.append(seq[b] + n)
        kv2.append(kv[b] + own(seq[b] + n) - own(seq[b]))
        for i in range(pages(kv[b]), pages(kv2[b])):
            count -= 1
            table[b][i] = free[count] if count >= 0 else -1
        for i in range(n):
            p = seq[b] + i
            positions[first + i], sequence[first + i] = p, b
            if p // inter % N == rank:
                j = kv[b] + own(p) - own(seq[b])
                if j // page < width and table[b][j // page] >= 0:
                    slots[first + i] = table[b][j // page] * page + j % page
    return cu, seq2, kv2, count, positions, sequence, slots, table, free
