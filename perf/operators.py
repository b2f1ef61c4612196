"""Cases of the cached-attention operators of a decode-context-parallel rank.

A rank holds every N-th block of `inter` positions of each sequence in a paged
cache.  Four operators work on it, in the order a layer calls them:

  rope   per-head RMS norm and position rotation of new queries and keys, the
         keys and values written into the rank's cache slots
  attn   attention of new tokens (one or a chunk) over the rank's slice of the
         cache: a partial output and its log-sum-exp, as dcp_pack takes them
  mass   accumulated attention weight of every cached key, from the merged
         log-sum-exp of all ranks
  evict  the keys of highest accumulated weight kept, gathered into new pages

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
        # one decode step of 64 requests: grouped heads, 8-bit cache, an eighth of the tokens on this rank
        _rope("rope decode 64 fp8", 64, 64, 8, 128, 128, 0, "half", "bf16", "fp8", False, 8, 1),
        # a long prompt chunk in the latent layout: 512 normed + 64 rotated columns, one key head
        _rope("rope latent chunk 8192", 8192, 128, 1, 576, 64, 512, "pair", "bf16", "bf16", True, 8, 16),
        # the smallest call: one token of one request with a short cache
        _attn("attn", "attn decode 1x1000 d64", 1, 1, 1000, 8, 1, 64, 64, False, "fp16", "fp16", 16, 1, 1),
        # decode of 32 long contexts, grouped heads, a quarter of each cache on this rank
        _attn("attn", "attn decode 32 long", 32, 1, 131072, 64, 8, 128, 128, False, "bf16", "bf16", 64, 4, 1),
        # decode of many short contexts from an 8-bit cache, the last of 8 ranks (some hold no key)
        _attn("attn", "attn decode 64 fp8", 64, 1, 65536, 32, 4, 128, 128, False, "bf16", "fp8", 16, 8, 16),
        # decode in the latent layout: 128 heads share one key row whose first 512 columns are its value
        _attn("attn", "attn latent decode 64", 64, 1, 131072, 128, 1, 576, 512, True, "bf16", "bf16", 64, 8, 1),
        # ragged prompt chunks behind cached prefixes, grouped heads
        _attn("attn", "attn chunk 4x2048", 4, 2048, 16384, 32, 8, 128, 128, False, "fp16", "fp16", 32, 2, 16),
        # a cached extend in the latent layout with 96 heads
        _attn("attn", "attn latent extend 1024", 1, 1024, 16384, 96, 1, 576, 512, True, "bf16", "bf16", 64, 8, 1),
        # weights of one decode step over long caches
        _attn("mass", "mass decode 16", 16, 1, 65536, 64, 8, 128, 0, False, "bf16", "bf16", 64, 4, 1),
        # weights of a prompt chunk
        _attn("mass", "mass chunk 2x1024", 2, 1024, 16384, 32, 8, 128, 0, False, "bf16", "bf16", 16, 2, 1),
        # the caches of 8 requests cut to 4096 keys for each head
        _evict("evict 8x16384 to 4096", 8, 16384, 4096, 8, 128, 128, False, "bf16", 64, 4, 64),
        # one request's latent cache cut by half
        _evict("evict latent 1x2001 to 1000", 1, 2001, 1000, 1, 576, 512, True, "fp8", 16, 1, 7),
    ]


def _rope(name, T, Hq, Hkv, D, rot, off, style, dtype, cache, shared, N, page):
    c = {"op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "off": off, "style": style, "dtype": dtype,
         "cache": cache, "shared": shared, "N": N, "page": page, "far": 131072}
    return dict(c, name=name) if name else c


def _attn(op, name, B, q, seq, Hq, Hkv, Dk, Dv, shared, dtype, cache, page, N, inter):
    c = {"op": op, "B": B, "q": q, "seq": seq, "Hq": Hq, "Hkv": Hkv, "Dk": Dk, "Dv": Dv, "shared": shared,
         "dtype": dtype, "cache": cache, "page": page, "N": N, "inter": inter, "rank": N - 1}
    return dict(c, name=name) if name else c


def _evict(name, B, kv, budget, Hkv, Dk, Dv, shared, cache, page, sink, recent):
    c = {"op": "evict", "B": B, "kv": kv, "budget": budget, "Hkv": Hkv, "Dk": Dk, "Dv": Dv, "shared": shared,
         "cache": cache, "page": page, "sink": sink, "recent": recent}
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "attn", "attn", "mass", "evict"])
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), w["bytes"] + w["flops"] / 50)
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        cache = rng.choice([dtype, dtype, "fp8"])
        page = rng.choice([1, 16, 16, 24, 32, 64, 128])
        N = rng.choice([1, 2, 3, 4, 8, 16])
        latent = rng.random() < 0.35
        G = rng.choice([1, 2, 4, 7, 8, 16])
        Hkv = 1 if latent else rng.choice([1, 2, 4, 5, 8])
        Hq = rng.choice([16, 96, 128]) if latent else G * Hkv
        D = 576 if latent else rng.choice([64, 80, 128, 128, 128, 192, 256])
        if op == "rope":
            c = _rope(None, _log(rng, 1, 8192), Hq, Hkv, D, 64 if latent else rng.choice([D // 2, D]),
                      512 if latent else 0, rng.choice(["half", "pair"]), dtype, cache, latent, N, page)
        elif op == "evict":
            kv = _log(rng, 100, 32768)
            budget = _log(rng, 64, kv)
            c = _evict(None, _log(rng, 1, 16), kv, budget, Hkv, D, 512 if latent else D, latent, cache, page,
                       rng.randint(0, 16), rng.randint(0, 32))
        else:
            chunk = rng.random() < 0.5
            B = _log(rng, 1, 8) if chunk else _log(rng, 1, 64)
            q = _log(rng, 2, 2048) if chunk else 1
            seq = q + _log(rng, 1, 16384 if chunk else 131072)
            dv = 512 if latent else rng.choice([D, min(D, 128)])
            c = _attn(op, None, B, q, seq, Hq, Hkv, D, dv if op == "attn" else 0, latent, dtype, cache, page, N,
                      rng.choice([1, 1, 8, 16]))
            c["rank"] = rng.randrange(N)
        w = work(c)
        if w["bytes"] + w["flops"] / 50 <= most[op]:
            return c


# ---------------------------------------------------------------------------
# lengths: the same for every seed, so that they are the case's own
# ---------------------------------------------------------------------------
def _owned(x, c):
    """How many of the positions 0..x-1 lie on this rank."""
    block = c["N"] * c["inter"]
    return x // block * c["inter"] + min(max(x % block - c["rank"] * c["inter"], 0), c["inter"])


def _lengths(c):
    """(new tokens, length after them) of each sequence: ragged, the first of full length."""
    r = random.Random("%d %d %d" % (c["B"], c["q"], c["seq"]))
    got = [(c["q"], c["seq"])]
    for b in range(1, c["B"]):
        n = r.randint(max(1, c["q"] // 4), c["q"])
        got.append((n, n if b == 3 else r.randint(n, c["seq"])))
    return got


def _evict_lengths(c):
    r = random.Random("%d %d" % (c["B"], c["kv"]))
    return [c["kv"]] + [r.randint(c["kv"] // 2, c["kv"]) for _ in range(1, c["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pool(lengths, page, g):
    """A page table over shuffled pages (entries behind a sequence's last page are -1) and the number of pages."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total, order[at:]


def _cached(shape, kind, g):
    """Cache contents: an 8-bit cache holds values divided by its scale."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16 if kind == "fp16" else torch.bfloat16)
    return x.to(_DT[kind])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"c": c}
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    if c["op"] == "rope":
        T, D, dt = c["T"], c["D"], _DT[c["dtype"]]
        width = (c["Hq"] + (1 if c["shared"] else 2) * c["Hkv"]) * D
        qkv = torch.randn((T, width), generator=g, device="cuda", dtype=dt)     # one projection's rows: q | k | v
        a, b = c["Hq"] * D, (c["Hq"] + c["Hkv"]) * D
        s["q"], s["k"] = qkv[:, :a].view(T, c["Hq"], D), qkv[:, a:b].view(T, c["Hkv"], D)
        s["v"] = None if c["shared"] else qkv[:, b:].view(T, c["Hkv"], D)
        s["wq"] = None if c["shared"] else (1 + 0.1 * normal(D)).to(dt)
        s["wk"] = (1 + 0.1 * normal(c["off"] if c["shared"] else D)).to(dt)
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(c["far"], dtype=torch.float64, device="cuda")[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["pos"] = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        mine = torch.arange(T, device="cuda") % c["N"] == 0
        pages = -(-(-(-T // c["N"])) // c["page"]) + 1
        slots = torch.randperm(pages * c["page"], generator=g, device="cuda")
        s["slots"] = torch.where(mine, slots[torch.arange(T, device="cuda") // c["N"]], -1)
        s["mine"] = torch.arange(0, T, c["N"], device="cuda")       # the tokens whose keys this rank holds
        s["kc"] = _cached((pages, c["page"], c["Hkv"], D), c["cache"], g)
        s["vc"] = None if c["shared"] else _cached((pages, c["page"], c["Hkv"], D), c["cache"], g)
        s["out"] = torch.empty((T, c["Hq"], D), dtype=dt, device="cuda")
        s["ks"], s["vs"] = (0.043, 0.037) if c["cache"] == "fp8" else (1.0, 1.0)
        return s
    if c["op"] == "evict":
        lens = _evict_lengths(c)
        s["table"], pages, _ = _pool(lens, c["page"], g)
        new = -(-c["budget"] // c["page"])
        s["dst"] = (pages + torch.randperm(c["B"] * new, generator=g, device="cuda").to(torch.int32)).view(c["B"], new)
        total = pages + c["B"] * new
        s["kc"] = _cached((total, c["page"], c["Hkv"], c["Dk"]), c["cache"], g)
        s["vc"] = None if c["shared"] else _cached((total, c["page"], c["Hkv"], c["Dv"]), c["cache"], g)
        s["mass"] = torch.exp(2 * normal(total, c["page"], c["Hkv"]))
        s["kv"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return s
    lens = _lengths(c)
    kv = [_owned(n, c) for _, n in lens]
    new = [n for n, _ in lens]
    T, dt = sum(new), _DT[c["dtype"]]
    s["table"], pages, _ = _pool(kv, c["page"], g)
    s["q"] = torch.randn((T, c["Hq"], c["Dk"]), generator=g, device="cuda", dtype=dt)
    s["kc"] = _cached((pages, c["page"], c["Hkv"], c["Dk"]), c["cache"], g)
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(c["B"] + 1)], dtype=torch.int32, device="cuda")
    s["kv"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["seq"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda")
    s["ks"], s["vs"] = (0.9, 1.1) if c["cache"] == "fp8" else (1.0, 1.0)
    s["scale"] = c["Dk"] ** -0.5
    if c["op"] == "attn":
        s["vc"] = None if c["shared"] else _cached((pages, c["page"], c["Hkv"], c["Dv"]), c["cache"], g)
        s["out"] = torch.empty((T, c["Hq"], c["Dv"]), dtype=dt, device="cuda")
        s["lse"] = torch.empty((T, c["Hq"]), dtype=torch.float32, device="cuda")
    else:
        # the merged log-sum-exp of standard normal scores over all ranks' keys, with a spread
        last = torch.cat([torch.arange(n - m + 1, n + 1, device="cuda") for m, n in lens]).float()
        s["lse"] = (last.log() + 0.5)[:, None] + 0.1 * normal(T, c["Hq"])
        # what such a chunk gave each key before
        s["mass"] = normal(pages, c["page"], c["Hkv"]).square() * (c["q"] * c["Hq"] / c["Hkv"] / c["seq"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["c"]["op"]
    if op == "rope":
        return _run_rope(s)
    if op == "attn":
        return _run_attn(s)
    if op == "mass":
        return _run_mass(s)
    return _run_evict(s)


def _run_rope(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        q = attn.qk_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["pos"], s["table"], s["slots"],
                                     s["kc"], s["vc"], rope_offset=c["off"], interleaved=c["style"] == "pair",
                                     eps=1e-6, k_scale=s["ks"], v_scale=s["vs"], q_out=s["out"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    angles = s["table"][s["pos"].long()][:, None]
    q = _turn(_normed(s["q"].float(), s["wq"]), angles, c).to(s["q"].dtype)
    i = s["mine"]
    k = _turn(_normed(s["k"][i].float(), s["wk"]), angles[i], c)
    _store(s["kc"], s["slots"][i], k, s["ks"])
    if s["vc"] is not None:
        _store(s["vc"], s["slots"][i], s["v"][i].float(), s["vs"])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _normed(x, w):
    if w is None:
        return x
    a = x[..., :w.numel()]
    a = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return torch.cat([a, x[..., w.numel():]], -1)


def _turn(x, angles, c):
    half = c["rot"] // 2
    cos, sin = angles[..., :half], angles[..., half:]
    r = x[..., c["off"]:c["off"] + c["rot"]]
    if c["style"] == "pair":
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([x[..., :c["off"]], r, x[..., c["off"] + c["rot"]:]], -1)


def _store(cache, slots, x, scale):
    if cache.dtype == torch.float8_e4m3fn:
        x = (x * (1.0 / scale)).clamp(-448, 448)
    flat = cache.view(-1, *cache.shape[2:])
    if cache.dtype == torch.float8_e4m3fn:
        flat.view(torch.uint8)[slots] = x.to(cache.dtype).view(torch.uint8)
    else:
        flat[slots] = x.to(cache.dtype)


def _paged(cache, table, scale, most):
    """Each sequence's first `most` cached rows in 32 bits: [B, Hkv, most, D]."""
    rows = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    rows = rows[table.long().clamp(min=0)].flatten(1, 2)[:, :most].contiguous()
    return rows.view(cache.dtype).float().mul_(scale).transpose(1, 2)


def _scores(s):
    """Scores of all pairs [B, Hkv, q * G, L] with -inf where a query does not see a key, and the queries' places."""
    c = s["c"]
    B, n, L = c["B"], c["q"], max(1, _owned(c["seq"], c))
    G = c["Hq"] // c["Hkv"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"].long()[b]
    q = torch.zeros((B, n, c["Hq"], c["Dk"]), dtype=torch.float32, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, c["Hkv"], G, c["Dk"]).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], n * G, c["Dk"])
    k = _paged(s["kc"], s["table"], s["ks"], L)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    # local key j stands at position (j // inter * N + rank) * inter + j % inter
    j = torch.arange(L, device="cuda")
    at = (j // c["inter"] * c["N"] + c["rank"]) * c["inter"] + j % c["inter"]
    here = (s["seq"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(n, device="cuda")
    seen = (at <= here[:, :, None]) & (j < s["kv"][:, None, None])
    x.view(B, c["Hkv"], n, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    return x, b, i, k


def _run_attn(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.dcp_paged_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], seq_len=s["seq"],
                                   scale=s["scale"], v_dim=c["Dv"], rank=c["rank"], n_ranks=c["N"],
                                   interleave=c["inter"], k_scale=s["ks"], v_scale=s["vs"], out=s["out"],
                                   out_lse=s["lse"])
    x, b, i, k = _scores(s)
    v = k[..., :c["Dv"]] if s["vc"] is None else _paged(s["vc"], s["table"], s["vs"], x.shape[-1])
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = m + total.log()
    shape = (c["B"], c["Hkv"], c["q"], c["Hq"] // c["Hkv"], -1)
    o = o.view(shape).permute(0, 2, 1, 3, 4).reshape(c["B"], c["q"], c["Hq"], c["Dv"])
    lse = lse.view(shape).permute(0, 2, 1, 3, 4).reshape(c["B"], c["q"], c["Hq"])
    return o[b, i].to(s["q"].dtype), lse[b, i].contiguous()


def _run_mass(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        return attn.dcp_attn_mass(s["q"], s["kc"], s["lse"], s["mass"], s["table"], s["cu"], s["kv"],
                                  seq_len=s["seq"], scale=s["scale"], rank=c["rank"], n_ranks=c["N"],
                                  interleave=c["inter"], k_scale=s["ks"])
    x, b, i, _ = _scores(s)
    lse = torch.full((c["B"], c["q"], c["Hq"]), math.inf, device="cuda")
    lse[b, i] = s["lse"]
    lse = lse.view(c["B"], c["q"], c["Hkv"], -1).transpose(1, 2).reshape(c["B"], c["Hkv"], -1, 1)
    got = x.sub_(lse).exp_().sum(2)                                    # [B, Hkv, L]
    j = torch.arange(got.shape[2], device="cuda")
    page = s["table"].long()[:, j // c["page"]]
    inside = j < s["kv"][:, None]
    got = torch.where(inside[:, None], got, 0.0).transpose(1, 2)       # keys behind the end add nothing to page 0
    s["mass"].index_put_((page.clamp(min=0), j % c["page"]), got, accumulate=True)
    return s["mass"]


def _run_evict(s):
    c = s["c"]
    if own:
        from lse_weighted_merge_dcp_amd import attn

        n, kept = attn.dcp_cache_evict(s["mass"], s["kc"], s["vc"], s["table"], s["kv"], s["dst"], c["budget"],
                                       n_sink=c["sink"], n_recent=c["recent"])
        return {"new_len": n, "kept": kept, "k_cache": s["kc"], "v_cache": s["vc"], "mass": s["mass"]}
    B, page, budget = c["B"], c["page"], c["budget"]
    L = max(c["kv"], budget)
    j = torch.arange(L, device="cuda")
    at = s["table"].long().clamp(min=0)[:, (j // page).clamp(max=s["table"].shape[1] - 1)]
    w = s["mass"][at, j % page].transpose(1, 2)                        # [B, Hkv, L]
    kv = s["kv"].long()[:, None, None]
    w = torch.where((j < c["sink"]) | (j >= kv - c["recent"]), math.inf, w)
    w = torch.where(j < kv, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(order < kv, order, L).sort(-1).values          # by age; L: nothing more to keep
    n = s["kv"].clamp(max=budget)
    i = torch.arange(budget, device="cuda")
    real = (i < n[:, None])[:, None].expand_as(order)
    src = torch.where(real, order, 0)
    h = torch.arange(c["Hkv"], device="cuda")[None, :, None]
    source = (at.gather(1, src.flatten(1)).view_as(src), src % page, h)
    target = (s["dst"].long()[:, i // page][:, None].expand_as(src), (i % page).expand_as(src), h.expand_as(src))
    for x in (s["kc"], s["vc"], s["mass"]):
        if x is not None:
            y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            keep = real.view(real.shape + (1,) * (x.dim() - 3))
            y.index_put_(target, torch.where(keep, y[source], y[target]))
    return {"new_len": n, "kept": torch.where(real, order, -1).to(torch.int32), "k_cache": s["kc"],
            "v_cache": s["vc"], "mass": s["mass"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    ec = _ES[c["cache"]]
    if c["op"] == "rope":
        mine = -(-c["T"] // c["N"])
        heads = (1 if c["shared"] else 2) * c["Hkv"]
        return {"bytes": 2 * c["T"] * c["Hq"] * c["D"] * 2 + mine * heads * c["D"] * (2 + ec) + c["T"] * (12 + 4 * c["rot"]),
                "flops": (c["T"] * c["Hq"] + mine * c["Hkv"]) * (4 * c["D"] + 3 * c["rot"])}
    if c["op"] == "evict":
        lens = _evict_lengths(c)
        kept = sum(min(n, c["budget"]) for n in lens)
        row = c["Dk"] * ec + (0 if c["shared"] else c["Dv"] * ec) + 4
        return {"bytes": c["Hkv"] * (4 * sum(lens) + kept * (2 * row + 4)), "flops": 0}
    lens = _lengths(c)
    kv = sum(_owned(n, c) for _, n in lens)
    T = sum(m for m, _ in lens)
    pairs = sum(_owned(p, c) for m, n in lens for p in range(n - m + 1, n + 1))
    if c["op"] == "attn":
        row = c["Dk"] + (0 if c["shared"] else c["Dv"])
        return {"bytes": T * c["Hq"] * (2 * c["Dk"] + 2 * c["Dv"] + 4) + kv * c["Hkv"] * row * ec,
                "flops": 2 * pairs * c["Hq"] * (c["Dk"] + c["Dv"])}
    return {"bytes": T * c["Hq"] * (2 * c["Dk"] + 4) + kv * c["Hkv"] * (c["Dk"] * ec + 8),
            "flops": 2 * pairs * c["Hq"] * c["Dk"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rope":
        return _exact_rope(s, c)
    if c["op"] == "evict":
        return _exact_evict(s, c)
    return _exact_scores(s, c)


def _exact_rope(s, c):
    def rows(x, w, pos):
        x = x.double()
        if w is not None:
            n = w.numel()
            rms = (x[..., :n].pow(2).sum(-1, keepdim=True) / n + 1e-6).sqrt()
            x[..., :n] = x[..., :n] / rms * w.double()
        half = c["rot"] // 2
        z = torch.complex(s["table"][pos.long(), :half].double(), s["table"][pos.long(), half:].double())[:, None]
        r = x[..., c["off"]:c["off"] + c["rot"]].clone()
        r = r.unflatten(-1, (half, 2)) if c["style"] == "pair" else r.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.complex(r[..., 0].contiguous(), r[..., 1].contiguous()) * z)
        x[..., c["off"]:c["off"] + c["rot"]] = (z if c["style"] == "pair" else z.transpose(-1, -2)).flatten(-2)
        return x

    def stored(cache, x, scale):
        full = cache.double().flatten(0, 1)
        if c["cache"] == "fp8":
            x = (x / scale).clamp(-448, 448)
        full[s["slots"][s["mine"]]] = x
        return full.view(cache.shape)

    i = s["mine"]
    return {"q": rows(s["q"], s["wq"], s["pos"]), "k_cache": stored(s["kc"], rows(s["k"][i], s["wk"], s["pos"][i]), s["ks"]),
            "v_cache": None if s["vc"] is None else stored(s["vc"], s["v"][i].double(), s["vs"])}


def _exact_scores(s, c):
    """Attention or accumulated weights, one sequence and one key head at a time."""
    G = c["Hq"] // c["Hkv"]
    T = s["q"].shape[0]
    out = torch.zeros((T, c["Hq"], c["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full((T, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if c["op"] == "mass" else None
    first = 0
    for b, (m, n) in enumerate(_lengths(c)):
        kv = _owned(n, c)
        ends = torch.tensor([_owned(p, c) for p in range(n - m + 1, n + 1)], device="cuda")
        if kv:
            j = torch.arange(kv, device="cuda")
            page, place = s["table"][b].long()[j // c["page"]], j % c["page"]
            hidden = j[None, None, :] >= ends[:, None, None]
            for h in range(c["Hkv"]):
                key = s["kc"][page, place, h].double() if c["cache"] != "fp8" else s["kc"].view(torch.uint8)[page, place, h].view(torch.float8_e4m3fn).double()
                key = key * s["ks"]
                q = s["q"][first:first + m, h * G:(h + 1) * G].double()
                x = (q.reshape(m * G, -1) @ key.t()).view(m, G, kv) * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                if mass is not None:
                    mass[page, place, h] += (x - s["lse"][first:first + m, h * G:(h + 1) * G, None].double()).exp().sum((0, 1))
                    continue
                if s["vc"] is None:
                    val = key[:, :c["Dv"]]
                else:
                    val = s["vc"][page, place, h].double() if c["cache"] != "fp8" else s["vc"].view(torch.uint8)[page, place, h].view(torch.float8_e4m3fn).double()
                    val = val * s["vs"]
                l = torch.logsumexp(x, -1)
                p = torch.where(hidden, 0.0, (x - l[..., None]).exp())
                out[first:first + m, h * G:(h + 1) * G] = (p.view(m * G, kv) @ val).view(m, G, -1)
                lse[first:first + m, h * G:(h + 1) * G] = l
        first += m
    return mass if mass is not None else (out, lse)


def _exact_evict(s, c):
    page, budget = c["page"], c["budget"]
    cell = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x  # noqa: E731
    pools = [(cell(x).clone(), x.dtype) for x in (s["kc"], s["vc"], s["mass"]) if x is not None]
    for b, n in enumerate(_evict_lengths(c)):
        for h in range(c["Hkv"]):
            j = torch.arange(n, device="cuda")
            src = s["table"][b].long()[j // page]
            w = s["mass"][src, j % page, h].double()
            w[:c["sink"]] = math.inf
            w[max(0, n - c["recent"]):] = math.inf
            keep = torch.argsort(-w, stable=True)[:budget].sort().values
            i = torch.arange(len(keep), device="cuda")
            for x, _ in pools:
                x[s["dst"][b].long()[i // page], i % page, h] = x[src[keep], keep % page, h]
    got = [x.view(dt).double() for x, dt in pools]
    return {"new_len": None, "kept": None, "k_cache": got[0], "v_cache": got[1] if s["vc"] is not None else None,
            "mass": got[-1]}
