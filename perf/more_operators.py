"""Cases of the operators around a serving step of a decode-context-parallel rank.

  plan      lengths, page tables and cache slots of a step, from the numbers of
            new tokens, with pages taken from and given back to a free list
  prefix    attention of a batch whose sequences share the first pages of their
            caches, the shared keys read once for all of a group
  queries   the key half of a latent projection taken into the queries
            [nope | rope] -> [latent | rope], head by head
  values    the value half of it taken out of the attention's latent outputs
  expand    keys and values of every head from the cached latent rows
  latent    attention in the expanded form: expand, then attention of a chunk

With own = False `run` computes them with elementary torch operations in 32
bits, with own = True through the package's public calls.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
_ES = {"bf16": 2, "fp16": 2, "fp8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 256 running requests, some ending, the third of four ranks
        _plan("plan decode 256", 256, 1, 65536, 16, 4, 1, 0.05),
        # prompt chunks of 24 requests beside each other on one of eight ranks, pages of 64
        _plan("plan chunks 24x2048", 24, 2048, 131072, 64, 8, 16, 0.1),
        # the smallest call: four requests behind a short common prompt
        _prefix("prefix decode 4x1000 d64", 4, 1, 1, 1000, 200, 8, 1, 64, 64, False, "fp16", "fp16", 16, 1, 1),
        # decode of 64 requests behind one long document, grouped heads, a quarter of each cache on this rank
        _prefix("prefix decode 64", 64, 1, 1, 32768, 4096, 64, 8, 128, 128, False, "bf16", "bf16", 16, 4, 1),
        # verification of four tokens each for 48 requests in three groups, from an 8-bit cache
        _prefix("prefix verify 48x4 fp8", 48, 4, 3, 16384, 2000, 32, 4, 128, 128, False, "bf16", "fp8", 32, 2, 16),
        # decode in the latent layout with 16 heads to a rank
        _prefix("prefix latent decode 96", 96, 1, 1, 65536, 8192, 16, 1, 576, 512, True, "bf16", "bf16", 64, 8, 1),
        # queries into latent space: one decode step of 64
        _queries("queries decode 64", 64, 128, 128, 64, 512, "bf16"),
        # latent outputs to values: the same step, and a ragged prompt chunk
        _values("values decode 64", 64, 128, 128, 512, "bf16"),
        _values("values chunk 2001", 2001, 96, 128, 512, "fp16"),
        # queries of a prompt chunk
        _queries("queries chunk 4096", 4096, 128, 128, 64, 512, "bf16"),
        # keys and values of a long cached context for a chunk's attention, 128 heads
        _expand("expand 16384", 1, 16384, 128, 128, 64, 128, 512, "bf16", "bf16", 64),
        # a prompt chunk of three requests in the expanded form, half of each cache on this rank, 8-bit rows
        _latent("latent chunk 3x1500 fp8", 3, 1500, 9000, 32, 128, 64, 128, 512, "bf16", "fp8", 64, 2, 1),
    ]


def _named(c, name):
    return dict(c, name=name) if name else c


def _plan(name, B, new, seq, page, N, inter, ended):
    return _named({"op": "plan", "B": B, "new": new, "seq": seq, "page": page, "N": N, "inter": inter,
                   "rank": N // 2, "ended": ended}, name)


def _prefix(name, B, q, groups, prefix, tail, Hq, Hkv, Dk, Dv, shared, dtype, cache, page, N, inter):
    return _named({"op": "prefix", "B": B, "q": q, "groups": groups, "prefix": prefix, "tail": tail, "Hq": Hq, "Hkv": Hkv,
                   "Dk": Dk, "Dv": Dv, "shared": shared, "dtype": dtype, "cache": cache, "page": page, "N": N,
                   "inter": inter, "rank": N - 1}, name)


def _queries(name, T, H, Dn, Dr, Dc, dtype):
    return _named({"op": "queries", "T": T, "H": H, "Dn": Dn, "Dr": Dr, "Dc": Dc, "dtype": dtype}, name)


def _values(name, T, H, Dv, Dc, dtype):
    return _named({"op": "values", "T": T, "H": H, "Dv": Dv, "Dc": Dc, "dtype": dtype}, name)


def _expand(name, B, kv, H, Dn, Dr, Dv, Dc, dtype, cache, page):
    return _named({"op": "expand", "B": B, "kv": kv, "H": H, "Dn": Dn, "Dr": Dr, "Dv": Dv, "Dc": Dc, "dtype": dtype,
                   "cache": cache, "page": page}, name)


def _latent(name, B, q, seq, H, Dn, Dr, Dv, Dc, dtype, cache, page, N, inter):
    return _named({"op": "latent", "B": B, "q": q, "seq": seq, "H": H, "Dn": Dn, "Dr": Dr, "Dv": Dv, "Dc": Dc,
                   "dtype": dtype, "cache": cache, "page": page, "N": N, "inter": inter, "rank": N - 1}, name)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "prefix", "prefix", "queries", "values", "expand", "latent"])
    cost = lambda c: work(c)["bytes"] + work(c)["flops"] / 50      # noqa: E731
    most = max(cost(c) for c in listed() if c["op"] == op)
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        cache = rng.choice([dtype, dtype, "fp8"])
        page = rng.choice([1, 16, 16, 24, 32, 64, 128])
        N = rng.choice([1, 2, 3, 4, 8, 16])
        inter = rng.choice([1, 1, 8, 16])
        H = rng.choice([8, 12, 16, 32, 64, 96, 128])
        Dn, Dr, Dv, Dc = rng.choice([(128, 64, 128, 512), (128, 64, 128, 512), (64, 32, 64, 256), (96, 32, 128, 448)])
        if op == "plan":
            chunk = rng.random() < 0.5
            c = _plan(None, _log(rng, 1, 32 if chunk else 512), _log(rng, 2, 4096) if chunk else 1,
                      _log(rng, 100, 131072), page, N, inter, rng.choice([0.0, 0.05, 0.3]))
        elif op == "prefix":
            latent = rng.random() < 0.35
            B = _log(rng, 1, 96)
            Hkv = 1 if latent else rng.choice([1, 2, 4, 5, 8])
            Hq = rng.choice([16, 96, 128]) if latent else rng.choice([1, 2, 4, 7, 8, 16]) * Hkv
            D = 576 if latent else rng.choice([64, 80, 128, 128, 128, 192, 256])
            q = 1 if rng.random() < 0.6 else _log(rng, 2, 64)
            c = _prefix(None, B, q, min(B, rng.choice([1, 1, 2, 5])), _log(rng, 200, 65536), q + _log(rng, 1, 8192), Hq, Hkv,
                        D, 512 if latent else rng.choice([D, min(D, 128)]), latent, dtype, cache, page, N, inter)
            c["rank"] = rng.randrange(N)
        elif op == "queries":
            c = _queries(None, _log(rng, 1, 4096), H, Dn, Dr, Dc, dtype)
        elif op == "values":
            c = _values(None, _log(rng, 1, 4096), H, Dv, Dc, dtype)
        elif op == "expand":
            c = _expand(None, _log(rng, 1, 8), _log(rng, 50, 16384), H, Dn, Dr, Dv, Dc, dtype, cache, page)
        else:
            q = _log(rng, 16, 2048)
            c = _latent(None, _log(rng, 1, 6), q, q + _log(rng, 1, 16384), H, Dn, Dr, Dv, Dc, dtype, cache, page, N, inter)
            c["rank"] = rng.randrange(N)
        if cost(c) <= most:
            return c


# ---------------------------------------------------------------------------
# lengths: the same for every seed, so that they are the case's own
# ---------------------------------------------------------------------------
def _owned(x, c):
    """How many of the positions 0..x-1 lie on this rank."""
    block = c["N"] * c["inter"]
    return x // block * c["inter"] + min(max(x % block - c["rank"] * c["inter"], 0), c["inter"])


def _plan_lengths(c):
    """(new tokens or -1, length before) of each sequence; about a tenth of the sequences start here."""
    r = random.Random("plan %d %d %d" % (c["B"], c["new"], c["seq"]))
    got = []
    for _ in range(c["B"]):
        new = r.randint(max(1, c["new"] // 4), c["new"])
        got.append((-1 if r.random() < c["ended"] else new, 0 if r.random() < 0.1 else r.randint(1, c["seq"])))
    return got


def _prefix_lengths(c):
    """(first sequence of each group and the end, prefix of each group, (new tokens, length) of each sequence)."""
    r = random.Random("prefix %d %d %d %d" % (c["B"], c["q"], c["prefix"], c["tail"]))
    first = [g * c["B"] // c["groups"] for g in range(c["groups"] + 1)]
    prefix = [c["prefix"]] + [r.randint(max(1, c["prefix"] // 4), c["prefix"]) for _ in range(1, c["groups"])]
    seqs = []
    for g in range(c["groups"]):
        for b in range(first[g], first[g + 1]):
            n = c["q"] if b == 0 else r.randint(max(1, c["q"] // 4), c["q"])
            seqs.append((n, prefix[g] + (c["tail"] if b == 0 else r.randint(n, c["tail"]))))
    return first, prefix, seqs


def _shared_keys(c, prefix):
    """The rank's keys of a prefix that lie in whole pages."""
    return _owned(prefix, c) // c["page"] * c["page"]


def _lengths(c):
    """(new tokens, length after them) of each sequence of a chunk."""
    r = random.Random("%d %d %d" % (c["B"], c["q"], c["seq"]))
    got = [(c["q"], c["seq"])]
    for _ in range(1, c["B"]):
        n = r.randint(max(1, c["q"] // 4), c["q"])
        got.append((n, r.randint(n, c["seq"])))
    return got


def _kept(c):
    r = random.Random("%d %d" % (c["B"], c["kv"]))
    return [c["kv"]] + [r.randint(1, c["kv"]) for _ in range(1, c["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cached(shape, kind, g):
    """Cache contents: an 8-bit cache holds values divided by its scale."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16 if kind == "fp16" else torch.bfloat16)
    return x.to(_DT[kind])


def _tables(counts, page, g, before=None):
    """A page table over shuffled pages (entries behind a sequence's last page are -1) and the number of pages.
    before: pages that a sequence shares with the others of its group, in front of its own."""
    before = before or [[] for _ in counts]
    most = max(1, max(len(p) + n for p, n in zip(before, counts)))
    used = 1 + max([x for p in before for x in p], default=-1)
    order = (used + torch.randperm(sum(counts) + 2, generator=g, device="cuda")).tolist()
    rows, at = [], 0
    for p, n in zip(before, counts):
        row = p + order[at:at + n]
        rows.append(row + [-1] * (most - len(row)))
        at += n
    return _ints(rows), used + sum(counts) + 2


def _weights(c, g):
    """One projection's weights, the heads' key rows and value rows beside each other."""
    n, v = c.get("Dn", 0), c.get("Dv", 0)
    w = torch.randn((c["H"], n + v, c["Dc"]), generator=g, device="cuda", dtype=torch.float32) * c["Dc"] ** -0.5
    w = w.to(_DT[c["dtype"]])
    return w[:, :n], w[:, n:]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"c": c}
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=_DT[c["dtype"]])   # noqa: E731
    if c["op"] == "plan":
        return _prepare_plan(s, c, g, int(seed))
    if c["op"] == "prefix":
        return _prepare_prefix(s, c, g, normal)
    if c["op"] == "queries":
        s["w"] = _weights(dict(c, Dv=128), g)[0]
        s["x"] = normal(c["T"], c["H"], c["Dn"] + c["Dr"])
        s["out"] = torch.empty((c["T"], c["H"], c["Dc"] + c["Dr"]), dtype=_DT[c["dtype"]], device="cuda")
        return s
    if c["op"] == "values":
        s["w"] = _weights(dict(c, Dn=128), g)[1]
        s["x"] = normal(c["T"], c["H"], c["Dc"])
        s["out"] = torch.empty((c["T"], c["H"], c["Dv"]), dtype=_DT[c["dtype"]], device="cuda")
        return s
    s["wk"], s["wv"] = _weights(c, g)
    if c["op"] == "expand":
        kv = _kept(c)
    else:
        lens = _lengths(c)
        kv = [_owned(n, c) for _, n in lens]
        new = [n for n, _ in lens]
        s["q"] = normal(sum(new), c["H"], c["Dn"] + c["Dr"])
        s["cu"] = _ints([sum(new[:b]) for b in range(c["B"] + 1)])
        s["seq"] = _ints([n for _, n in lens])
        s["out"] = torch.empty((sum(new), c["H"], c["Dv"]), dtype=_DT[c["dtype"]], device="cuda")
        s["lse"] = torch.empty((sum(new), c["H"]), dtype=torch.float32, device="cuda")
        s["scale"] = (c["Dn"] + c["Dr"]) ** -0.5
    s["table"], pages = _tables([-(-n // c["page"]) for n in kv], c["page"], g)
    s["cache"] = _cached((pages, c["page"], 1, c["Dc"] + c["Dr"]), c["cache"], g)
    s["kv"], s["most"] = _ints(kv), max(1, max(kv))
    s["ks"] = 0.9 if c["cache"] == "fp8" else 1.0
    # the buffers that a program keeps for them; rows behind a sequence's keys stay as they are
    s["k"] = torch.zeros((c["B"], s["most"], c["H"], c["Dn"] + c["Dr"]), dtype=_DT[c["dtype"]], device="cuda")
    s["v"] = torch.zeros((c["B"], s["most"], c["H"], c["Dv"]), dtype=_DT[c["dtype"]], device="cuda")
    return s


def _prepare_plan(s, c, g, seed):
    r = random.Random(seed)
    lens = _plan_lengths(c)
    r.shuffle(lens)                                   # (the same work in another order)
    T = sum(max(n, 0) for n, _ in lens)
    s["T"] = T + 8                                    # a step's rows are padded
    page = c["page"]
    kv = [_owned(n, c) for _, n in lens]
    held = [-(-n // page) for n in kv]
    after = [-(-_owned(n + max(m, 0), c) // page) for m, n in lens]
    width = max(after + held) + 2
    pages = sum(held) + sum(after) + 16
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], width), -1, dtype=torch.int32)
    at, pool = 0, order.cpu()
    for b, n in enumerate(held):
        table[b, :n] = pool[at:at + n]
        at += n
    s["table"] = table.cuda()
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:pages - at] = order[at:]
    s["count"] = _ints([pages - at])
    s["new"], s["seq"], s["kv"] = _ints([m for m, _ in lens]), _ints([n for _, n in lens]), _ints(kv)
    s["keep"] = _ints([min(h, 2) for h in held])      # a common system prompt's pages are not given back
    return s


def _prepare_prefix(s, c, g, normal):
    first, prefix, seqs = _prefix_lengths(c)
    keys = [_shared_keys(c, p) for p in prefix]
    pages = [n // c["page"] for n in keys]
    kv = [_owned(n, c) for _, n in seqs]
    group = [max(i for i in range(c["groups"]) if first[i] <= b) for b in range(c["B"])]
    stack = torch.randperm(sum(pages), generator=g, device="cuda").tolist()
    common = [stack[sum(pages[:i]):sum(pages[:i + 1])] for i in range(c["groups"])]
    own_pages = [-(-n // c["page"]) - pages[group[b]] for b, n in enumerate(kv)]
    s["table"], total = _tables(own_pages, c["page"], g, [common[i] for i in group])
    new = [n for n, _ in seqs]
    s["q"] = normal(sum(new), c["Hq"], c["Dk"])
    s["kc"] = _cached((total, c["page"], c["Hkv"], c["Dk"]), c["cache"], g)
    s["vc"] = None if c["shared"] else _cached((total, c["page"], c["Hkv"], c["Dv"]), c["cache"], g)
    s["cu"] = _ints([sum(new[:b]) for b in range(c["B"] + 1)])
    s["kv"], s["seq"] = _ints(kv), _ints([n for _, n in seqs])
    s["cug"], s["same"] = _ints(first), _ints(keys)
    s["groups"] = [(first[i], first[i + 1], keys[i]) for i in range(c["groups"])]
    s["tail"] = max(1, max(n - keys[group[b]] for b, n in enumerate(kv)))
    s["ks"], s["vs"] = (0.9, 1.1) if c["cache"] == "fp8" else (1.0, 1.0)
    s["scale"] = c["Dk"] ** -0.5
    s["out"] = torch.empty((sum(new), c["Hq"], c["Dv"]), dtype=_DT[c["dtype"]], device="cuda")
    s["lse"] = torch.empty((sum(new), c["Hq"]), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"plan": _run_plan, "prefix": _run_prefix, "queries": _run_queries, "values": _run_values,
            "expand": _run_expand, "latent": _run_latent}[s["c"]["op"]](s)


def _run_plan(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        p = attn.dcp_batch_plan(s["new"], s["seq"], s["kv"], s["table"], s["free"], s["count"], s["T"], c["page"],
                                rank=c["rank"], n_ranks=c["N"], interleave=c["inter"], keep_pages=s["keep"])
        return {"cu_q": p.cu_q, "seq_len": p.seq_len, "kv_len": p.kv_len, "free_count": p.free_count,
                "positions": p.positions, "sequence": p.sequence, "slots": p.slots, "table": s["table"], "free": s["free"]}
    T, page, table, free = s["T"], c["page"], s["table"], s["free"]
    B, width = table.shape
    block = c["N"] * c["inter"]

    def mine(x):
        return x // block * c["inter"] + (x % block - c["rank"] * c["inter"]).clamp(0, c["inter"])

    new, L, m = s["new"].long(), s["seq"].long(), s["kv"].long()
    ended = new < 0
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.clamp(min=0).cumsum(0).clamp(max=T)])
    n = cu[1:] - cu[:-1]
    seq = torch.where(ended, 0, L + n)
    kv = torch.where(ended, 0, m + mine(L + n) - mine(L))
    i = torch.arange(width, device="cuda")
    held = ((m + page - 1) // page)[:, None]
    # the pages of ended sequences go on the free list
    back = (ended[:, None] & (i >= s["keep"][:, None]) & (i < held) & (table >= 0)).flatten()
    at = torch.where(back, s["count"].clamp(min=0) + back.long().cumsum(0) - 1, free.numel()).clamp(max=free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter_(0, at, table.flatten())[:-1]
    count = (s["count"].clamp(min=0) + back.sum()).clamp(max=free.numel())
    # new pages from its end
    need = (~ended[:, None] & (i >= held) & (i < ((kv + page - 1) // page)[:, None])).flatten()
    k = count - need.long().cumsum(0)
    got = torch.where(k >= 0, stack[k.clamp(min=0)], -1)
    grown = torch.where(need, got, table.flatten()).view(B, width)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    p = L[b] + t - cu[b]
    j = m[b] + mine(p) - mine(L[b])
    pg = grown[b, (j // page).clamp(max=width - 1)].long()
    here = real & (p // c["inter"] % c["N"] == c["rank"]) & (j // page < width) & (pg >= 0)
    free.copy_(stack)
    table.copy_(grown)
    return {"cu_q": cu.int(), "seq_len": seq.int(), "kv_len": kv.int(), "free_count": (count - need.sum()).int(),
            "positions": torch.where(real, p, -1).int(), "sequence": torch.where(real, b, -1).int(),
            "slots": torch.where(here, pg * page + j % page, -1), "table": table, "free": free}


def _paged(cache, table, scale, first, most):
    """Cached rows first .. most - 1 of each row of the table in 32 bits: [B, Hkv, most - first, D]."""
    page = cache.shape[1]
    rows = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    j = torch.arange(first, most, device="cuda")
    at = table.long().clamp(min=0)[:, (j // page).clamp(max=table.shape[1] - 1)]
    rows = rows[at, j % page]
    return rows.view(cache.dtype).float().mul_(scale).transpose(1, 2)


def _run_prefix(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.dcp_prefix_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["cug"], s["same"],
                                    seq_len=s["seq"], scale=s["scale"], v_dim=c["Dv"], rank=c["rank"], n_ranks=c["N"],
                                    interleave=c["inter"], k_scale=s["ks"], v_scale=s["vs"], out=s["out"],
                                    out_lse=s["lse"])
    B, n, Hkv, G = c["B"], c["q"], c["Hkv"], c["Hq"] // c["Hkv"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"].long()[b]
    q = torch.zeros((B, n, c["Hq"], c["Dk"]), dtype=torch.float32, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, c["Dk"]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, c["Dk"])
    out = torch.zeros((B, Hkv, n * G, c["Dv"]), dtype=torch.float32, device="cuda")
    top = torch.full((B, Hkv, n * G, 1), -math.inf, device="cuda")
    total = torch.zeros((B, Hkv, n * G, 1), device="cuda")

    # the shared keys, once for all rows of a group (they stand before every new token)
    for lo, hi, keys in s["groups"]:
        if hi == lo or keys == 0:
            continue
        k = _paged(s["kc"], s["table"][lo:lo + 1], s["ks"], 0, keys)[0]
        v = k[..., :c["Dv"]] if s["vc"] is None else _paged(s["vc"], s["table"][lo:lo + 1], s["vs"], 0, keys)[0]
        x = torch.matmul(q[lo:hi].transpose(0, 1).reshape(Hkv, -1, c["Dk"]), k.transpose(1, 2)).mul_(s["scale"])
        m = x.amax(-1, keepdim=True)
        p = x.sub_(m).exp_()
        rows = lambda y: y.view(Hkv, hi - lo, n * G, -1).transpose(0, 1)      # noqa: E731
        top[lo:hi], total[lo:hi], out[lo:hi] = rows(m), rows(p.sum(-1, keepdim=True)), rows(torch.matmul(p, v))
    # every sequence's own keys
    for lo, hi, keys in s["groups"]:
        if hi == lo:
            continue
        end = keys + s["tail"]
        k = _paged(s["kc"], s["table"][lo:hi], s["ks"], keys, end)
        v = k[..., :c["Dv"]] if s["vc"] is None else _paged(s["vc"], s["table"][lo:hi], s["vs"], keys, end)
        # local key j stands at position (j // inter * N + rank) * inter + j % inter
        j = torch.arange(keys, end, device="cuda")
        at = (j // c["inter"] * c["N"] + c["rank"]) * c["inter"] + j % c["inter"]
        here = (s["seq"] - (s["cu"][1:] - s["cu"][:-1]))[lo:hi, None] + torch.arange(n, device="cuda")
        hidden = (at > here[:, :, None]) | (j >= s["kv"][lo:hi, None, None])
        hidden = hidden[:, None, :, None, :].expand(-1, 1, -1, G, -1).reshape(hi - lo, 1, n * G, -1)
        x = torch.matmul(q[lo:hi], k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        m = torch.maximum(top[lo:hi], x.amax(-1, keepdim=True))
        ref = torch.where(m == -math.inf, 0.0, m)
        old = torch.exp(top[lo:hi] - ref)
        p = x.sub_(ref).exp_()
        total[lo:hi] = total[lo:hi] * old + p.sum(-1, keepdim=True)
        out[lo:hi] = out[lo:hi] * old + torch.matmul(p, v)
        top[lo:hi] = m
    o = out / torch.where(total > 0, total, 1.0)
    lse = top + total.log()
    o = o.view(B, Hkv, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, c["Hq"], c["Dv"])
    lse = lse.view(B, Hkv, n, G).permute(0, 2, 1, 3).reshape(B, n, c["Hq"])
    return o[b, i].to(s["q"].dtype), lse[b, i].contiguous()


def _run_queries(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.latent_queries(s["x"], s["w"], out=s["out"])
    n = c["Dn"]
    y = torch.matmul(s["x"][..., :n].float().transpose(0, 1).contiguous(), s["w"].float().contiguous())
    return torch.cat([y.transpose(0, 1).to(s["x"].dtype), s["x"][..., n:]], -1)


def _run_values(s):
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.latent_values(s["x"], s["w"], out=s["out"])
    y = torch.matmul(s["x"].float().transpose(0, 1).contiguous(), s["w"].float().transpose(1, 2).contiguous())
    return y.transpose(0, 1).to(s["x"].dtype).contiguous()


def _expanded(s):
    """Keys and values [B, most, H, .] of every head in 32 bits."""
    c = s["c"]
    row = _paged(s["cache"], s["table"], s["ks"], 0, s["most"])[:, 0]
    latent, rope = row[..., :c["Dc"]], row[..., c["Dc"]:]
    k = torch.matmul(latent, s["wk"].float().flatten(0, 1).t()).unflatten(-1, (c["H"], c["Dn"]))
    v = torch.matmul(latent, s["wv"].float().flatten(0, 1).t()).unflatten(-1, (c["H"], c["Dv"]))
    return torch.cat([k, rope[:, :, None].expand(-1, -1, c["H"], -1)], -1), v


def _run_expand(s):
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.latent_expand(s["cache"], s["wk"], s["wv"], s["table"], s["kv"], s["most"], k_scale=s["ks"],
                                  k_out=s["k"], v_out=s["v"])
    k, v = _expanded(s)
    there = (torch.arange(s["most"], device="cuda") < s["kv"][:, None])[:, :, None, None]
    s["k"].copy_(torch.where(there, k.to(s["k"].dtype), s["k"]))
    s["v"].copy_(torch.where(there, v.to(s["v"].dtype), s["v"]))
    return s["k"], s["v"]


def _run_latent(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.dcp_latent_attn(s["q"], s["cache"], s["wk"], s["wv"], s["table"], s["cu"], s["kv"], s["most"],
                                    seq_len=s["seq"], scale=s["scale"], rank=c["rank"], n_ranks=c["N"],
                                    interleave=c["inter"], k_scale=s["ks"], out=s["out"], out_lse=s["lse"],
                                    k_out=s["k"], v_out=s["v"])
    k, v = _expanded(s)
    B, n, H = c["B"], c["q"], c["H"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"].long()[b]
    q = torch.zeros((B, n, H, c["Dn"] + c["Dr"]), dtype=torch.float32, device="cuda")
    q[b, i] = s["q"].float()
    x = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)).mul_(s["scale"])          # [B, H, n, keys]
    j = torch.arange(s["most"], device="cuda")
    at = (j // c["inter"] * c["N"] + c["rank"]) * c["inter"] + j % c["inter"]
    here = (s["seq"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(n, device="cuda")
    hidden = (at > here[:, :, None]) | (j >= s["kv"][:, None, None])
    x = x.masked_fill_(hidden[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    lse = (m + total.log())[..., 0]
    return o.transpose(1, 2)[b, i].to(s["q"].dtype), lse.transpose(1, 2)[b, i].contiguous()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "plan":
        lens = _plan_lengths(c)
        T = sum(max(n, 0) for n, _ in lens) + 8
        moved = 0                                     # pages taken or given back: an entry read, an entry written
        for n, L in lens:
            held = -(-_owned(L, c) // c["page"])
            moved += held if n < 0 else -(-_owned(L + n, c) // c["page"]) - held
        return {"bytes": 16 * T + c["B"] * 4 * 7 + 8 * moved, "flops": 0}
    if c["op"] == "prefix":
        first, prefix, seqs = _prefix_lengths(c)
        keys = [_shared_keys(c, p) for p in prefix]
        own_keys = sum(_owned(seqs[b][1], c) - keys[i] for i in range(c["groups"]) for b in range(first[i], first[i + 1]))
        T = sum(n for n, _ in seqs)
        pairs = sum(_owned(p, c) for n, L in seqs for p in range(L - n + 1, L + 1))
        row = c["Dk"] + (0 if c["shared"] else c["Dv"])
        return {"bytes": T * c["Hq"] * (2 * c["Dk"] + 2 * c["Dv"] + 4) + (sum(keys) + own_keys) * c["Hkv"] * row * _ES[c["cache"]],
                "flops": 2 * pairs * c["Hq"] * (c["Dk"] + c["Dv"])}
    if c["op"] == "queries":
        return {"bytes": 2 * c["H"] * (c["T"] * (c["Dn"] + c["Dc"] + 2 * c["Dr"]) + c["Dn"] * c["Dc"]),
                "flops": 2 * c["T"] * c["H"] * c["Dn"] * c["Dc"]}
    if c["op"] == "values":
        return {"bytes": 2 * c["H"] * (c["T"] * (c["Dv"] + c["Dc"]) + c["Dv"] * c["Dc"]),
                "flops": 2 * c["T"] * c["H"] * c["Dv"] * c["Dc"]}
    weights = 2 * c["H"] * (c["Dn"] + c["Dv"]) * c["Dc"]
    row = (c["Dc"] + c["Dr"]) * _ES[c["cache"]]
    if c["op"] == "expand":
        kv = sum(_kept(c))
        return {"bytes": kv * (row + 2 * c["H"] * (c["Dn"] + c["Dr"] + c["Dv"])) + weights,
                "flops": 2 * kv * c["H"] * (c["Dn"] + c["Dv"]) * c["Dc"]}
    lens = _lengths(c)
    kv = sum(_owned(n, c) for _, n in lens)
    T = sum(m for m, _ in lens)
    pairs = sum(_owned(p, c) for m, n in lens for p in range(n - m + 1, n + 1))
    return {"bytes": kv * row + weights + T * c["H"] * (2 * (c["Dn"] + c["Dr"] + c["Dv"]) + 4),
            "flops": 2 * kv * c["H"] * (c["Dn"] + c["Dv"]) * c["Dc"] + 2 * pairs * c["H"] * (c["Dn"] + c["Dr"] + c["Dv"])}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None                                   # whole numbers
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] in ("queries", "values"):
        x, w = s["x"].double(), s["w"].double()
        heads = []
        for h in range(c["H"]):
            if c["op"] == "queries":
                heads.append(torch.cat([x[:, h, :c["Dn"]] @ w[h], x[:, h, c["Dn"]:]], 1))
            else:
                heads.append(x[:, h] @ w[h].t())
        return torch.stack(heads, 1)
    if c["op"] == "expand":
        return _exact_expand(s, c)
    if c["op"] == "latent":
        return _exact_latent(s, c)
    return _exact_prefix(s, c)


def _row(cache, table, keys, page, h, scale):
    """Cached rows 0 .. keys - 1 of one sequence and head, in 64 bits."""
    j = torch.arange(keys, device="cuda")
    bits = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    return bits[table.long()[j // page], j % page, h].view(cache.dtype).double() * scale


def _exact_expand(s, c):
    k, v = s["k"].double(), s["v"].double()
    for b, n in enumerate(_kept(c)):
        row = _row(s["cache"], s["table"][b], n, c["page"], 0, s["ks"])
        for h in range(c["H"]):
            k[b, :n, h, :c["Dn"]] = row[:, :c["Dc"]] @ s["wk"][h].double().t()
            k[b, :n, h, c["Dn"]:] = row[:, c["Dc"]:]
            v[b, :n, h] = row[:, :c["Dc"]] @ s["wv"][h].double().t()
    return k, v


def _attend(q, key, val, ends, scale):
    """One head: q [m, D], the first ends[i] keys seen by row i."""
    x = (q @ key.t()) * scale
    hidden = torch.arange(key.shape[0], device="cuda")[None] >= ends[:, None]
    x = x.masked_fill(hidden, -math.inf)
    l = torch.logsumexp(x, -1)
    return torch.where(hidden, 0.0, (x - l[:, None]).exp()) @ val, l


def _exact_latent(s, c):
    T = s["q"].shape[0]
    out = torch.zeros((T, c["H"], c["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full((T, c["H"]), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (m, n) in enumerate(_lengths(c)):
        kv = _owned(n, c)
        ends = torch.tensor([_owned(p, c) for p in range(n - m + 1, n + 1)], device="cuda")
        row = _row(s["cache"], s["table"][b], kv, c["page"], 0, s["ks"])
        for h in range(c["H"]):
            key = torch.cat([row[:, :c["Dc"]] @ s["wk"][h].double().t(), row[:, c["Dc"]:]], 1)
            val = row[:, :c["Dc"]] @ s["wv"][h].double().t()
            if kv:
                out[first:first + m, h], lse[first:first + m, h] = _attend(s["q"][first:first + m, h].double(), key, val, ends, s["scale"])
        first += m
    return out, lse


def _exact_prefix(s, c):
    G = c["Hq"] // c["Hkv"]
    T = s["q"].shape[0]
    out = torch.zeros((T, c["Hq"], c["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full((T, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (m, n) in enumerate(_prefix_lengths(c)[2]):
        kv = _owned(n, c)
        ends = torch.tensor([_owned(p, c) for p in range(n - m + 1, n + 1)], device="cuda").repeat_interleave(G)
        for h in range(c["Hkv"] if kv else 0):
            key = _row(s["kc"], s["table"][b], kv, c["page"], h, s["ks"])
            val = key[:, :c["Dv"]] if s["vc"] is None else _row(s["vc"], s["table"][b], kv, c["page"], h, s["vs"])
            q = s["q"][first:first + m, h * G:(h + 1) * G].double().reshape(m * G, -1)
            o, l = _attend(q, key, val, ends, s["scale"])
            out[first:first + m, h * G:(h + 1) * G] = torch.where(ends[:, None] > 0, o, 0.0).view(m, G, -1)
            lse[first:first + m, h * G:(h + 1) * G] = l.view(m, G)
        first += m
    return out, lse
