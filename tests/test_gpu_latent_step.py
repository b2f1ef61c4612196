"""Serving steps of a latent layer over two ranks, from the plan to the values, against dense attention in 64 bits over
the rows that were cached.

A shared prompt is written once, three sequences go on behind it.  Every step: the plan (on every rank, in place), queries
into latent space, rotation and append, attention behind the shared prefix, pack, exchange and merge, values.  Then a
chunk in the expanded form, and a sequence that ends and gives its pages back.

Tolerance: outputs are means of values near 1.  On their way stand five roundings to 16 bits (latent queries, rotated
queries, weights, a rank's partial, the merged latent row, the values: 2^-8 each of rows of 64 to 256 terms near 1, whose
errors add up as roots) and the scores that the first two put off by up to 2^-7 of scores near 1: 2^-4 in all."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn, sim

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_steps_of_a_latent_layer():
    N, inter, page, H, Dn, Dr, Dv, Dc, B = 2, 2, 8, 4, 32, 16, 32, 64, 3
    dt, g = torch.bfloat16, torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g).to(dt)                   # noqa: E731
    w = (torch.randn(H, Dn + Dv, Dc, generator=g) * Dc ** -0.5).to(dt)
    wk, wv = w.to(DEV)[:, :Dn], w.to(DEV)[:, Dn:]
    angle = torch.arange(256.0)[:, None] * 0.3 ** torch.arange(Dr // 2)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    scale = (Dn + Dr) ** -0.5
    P = N * page * 2                                                        # the prompt: two whole pages on each rank
    pages, width, T = 40, 12, 80
    cache = torch.zeros(N, pages, page, 1, Dc + Dr, dtype=dt, device=DEV)
    table = torch.full((N, B, width), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(N, 1)
    count = i32([[pages]] * N)
    seq, kv = i32([[0] * B] * N), i32([[0] * B] * N)
    keep = i32([0] * B)
    history = [[] for _ in range(B)]                                        # cached rows of each sequence, rotated, on the host

    def turn(x, pos):
        """Rotation of the last Dr columns (halves), in 64 bits."""
        x = x.double().clone()
        c, s = cos_sin[pos, :Dr // 2].double(), cos_sin[pos, Dr // 2:].double()
        while c.dim() < x.dim():
            c, s = c.unsqueeze(1), s.unsqueeze(1)
        a, b = x[..., -Dr:-Dr // 2].clone(), x[..., -Dr // 2:].clone()
        x[..., -Dr:-Dr // 2], x[..., -Dr // 2:] = a * c - b * s, b * c + a * s
        return x

    def step(new, expanded=False, groups=True):
        before = [len(h) for h in history]
        n_tok = sum(max(n, 0) for n in new)
        q, k = rand(T, H, Dn + Dr), rand(T, 1, Dc + Dr)
        plans = []
        for r in range(N):
            plan = attn.dcp_batch_plan(i32(new), seq[r], kv[r], table[r], free[r], count[r], T, page, rank=r, n_ranks=N,
                                       interleave=inter, keep_pages=keep)
            seq[r].copy_(plan.seq_len)
            kv[r].copy_(plan.kv_len)
            count[r].copy_(plan.free_count)
            plans.append(plan)
        pos = plans[0].positions.cpu()
        assert pos[:n_tok].tolist() == [before[b] + i for b, n in enumerate(new) for i in range(max(n, 0))]
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                history[b] = []
            else:
                rows = turn(k[at:at + n, 0], pos[at:at + n].long()).to(dt)
                history[b] += list(rows)
                at += max(n, 0)
        out = torch.zeros(N, T, H, Dv if expanded else Dc, dtype=dt, device=DEV)
        lse = torch.zeros(N, T, H, device=DEV)
        ql = attn.latent_queries(q.to(DEV), wk)
        for r in range(N):
            p = plans[r]
            rot = attn.qk_norm_rope_append(ql, k.to(DEV), None, None, None, p.positions.clamp(min=0), cos_sin.to(DEV), p.slots,
                                           cache[r], None, rope_offset=Dc)
            args = dict(seq_len=p.seq_len, scale=scale, rank=r, n_ranks=N, interleave=inter, out=out[r], out_lse=lse[r])
            if expanded:
                qe = torch.cat([q.to(DEV)[..., :Dn], rot[..., Dc:]], -1)
                attn.dcp_latent_attn(qe, cache[r], wk, wv, table[r], p.cu_q, p.kv_len, width * page, **args)
            elif groups:
                attn.dcp_prefix_attn(rot, cache[r], None, table[r], p.cu_q, p.kv_len, i32([0, B]), i32([P // N]), v_dim=Dc, **args)
            else:
                attn.dcp_paged_attn(rot, cache[r], None, table[r], p.cu_q, p.kv_len, v_dim=Dc, **args)
        st = sim.StackedInterleaved(N, T, H, out.shape[3], dt, torch.device(DEV))
        st.pack(out, lse)
        merged, glse = st.combine(is_lse_base_on_e=True)
        merged, glse = merged.transpose(0, 1).reshape(T, H, -1), glse.transpose(0, 1).reshape(T, H)
        y = merged if expanded else attn.latent_values(merged.contiguous(), wv)
        y, glse = y.cpu().double(), glse.cpu().double()
        at, wd = 0, w.double()
        for b, n in enumerate(new):
            for i in range(max(n, 0)):
                end = before[b] + i + 1
                rows = torch.stack(history[b][:end]).double()
                qd = turn(q[at:at + 1], pos[at:at + 1].long())[0]
                for h in range(H):
                    s = scale * (rows[:, :Dc] @ wd[h, :Dn].t() @ qd[h, :Dn] + rows[:, Dc:] @ qd[h, Dn:])
                    want = torch.softmax(s, 0) @ (rows[:, :Dc] @ wd[h, Dn:].t())
                    assert float((y[at, h] - want).abs().max()) <= 2.0 ** -4, (b, i, h)
                    assert abs(float(glse[at, h] - torch.logsumexp(s, 0))) <= 2.0 ** -4
                at += 1

    step([P, 0, 0], groups=False)
    # sequences 1 and 2 go on behind the prompt's pages, which stay when they end
    for r in range(N):
        table[r, 1:, :2] = table[r, 0, :2]
        kv[r, 1:] = P // N
        seq[r, 1:] = P
    keep.copy_(i32([0, 2, 2]))
    history[1], history[2] = list(history[0]), list(history[0])
    for new in ([1, 1, 1], [1, 2, 1], [1, 1, 1], [0, 1, 1]):
        step(new)
    step([9, 20, 1], expanded=True)
    step([1, 1, 1])
    held = [-(-int(x) // page) for x in kv[:, 2]]
    left = count[:, 0].tolist()
    step([1, 1, -1])
    # its own pages came back, its part of the prompt did not; the others' new keys still fit their pages or took one
    for r in range(N):
        took = sum(-(-int(kv[r, b]) // page) - -(-(int(kv[r, b]) - 1) // page) for b in (0, 1)
                   if attn.owned_positions(len(history[b]), r, N, inter) > attn.owned_positions(len(history[b]) - 1, r, N, inter))
        assert int(count[r]) == left[r] + held[r] - 2 - took
        assert int(kv[r, 2]) == 0 and int(seq[r, 2]) == 0
    step([1, 1, 0])
