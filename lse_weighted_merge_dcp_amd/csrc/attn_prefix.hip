// attn_prefix.hip -- attention behind shared prefixes (attn_prefix.hpp): the list of
// units, the kernels of the latent layout, the join, and the calls' layout.
#include "attn_join.hpp"
#include "attn_latent.hpp"
#include "attn_prefix.hpp"

namespace dcpa {

namespace {

// ---------------------------------------------------------------------------
// prefix_list: the units of a call, by one workgroup: a thread to an entry (group
// or sequence), then a thread to a unit.
//
// The key ranges' length is chosen among 32 that cut the longest entry evenly:
// with U units of which the longest takes c keys, `share` of them at once and a
// price of kPrice keys to a unit (its start, and a part of 128 rows written and read
// again), either all run at once and take c + kPrice, or their mean load and one
// unit more.  (64 sequences behind 32768 keys on four ranks, with one product for the
// shared keys' weights: 68 us a call in ranges of 1024 keys, 75 of 704, 82 of 384.)
// Every workgroup finding its own unit from the lengths, as those of single
// sequences do, took 112 us there, a dozen dependent loads in front of 8 key tiles;
// this kernel took 8.5 and the rest 60.  Most of its time is waiting: for the lengths (two
// loads one after the other) and for code that is run once.
// More than kThreads entries do not stay in LDS and are loaded again for every length that
// is tried: 1100 sequences of one token in 4 groups take 65 us a call, 2000 in 8 115, by
// themselves 81 and 164.
// ---------------------------------------------------------------------------
constexpr int kThreads = 1024, kWaves = kThreads / 64, kTries = 32, kPrice = 1024;
constexpr int kMost = 1 << 30;
// in how many ranges: each number about a quarter above the last
struct Ways {
    uint16_t n[kTries];
};
constexpr Ways make_ways() {
    Ways w{};
    int n = 1;
    for (int k = 0; k < kTries; ++k) {
        w.n[k] = (uint16_t)n;
        n += n < 4 ? 1 : n / 4;
    }
    return w;
}
__device__ const Ways kWays = make_ways();

// In how many ranges of `len` keys `keys` are cut, one at least; inv: 1 / len.
__device__ __forceinline__ int ranges_of(int keys, int len, float inv) {
    const int q = (int)((float)keys * inv), rest = keys - q * len;      // (q off by one at most: keys / len < 2^14)
    return max(1, q + (rest > 0 ? 1 : 0) + (rest > len ? 1 : 0));
}

// Sequences of group g, and how many keys they share.
struct Group {
    int b0, b1, keys;
};
__device__ __forceinline__ Group load_group(const GroupArgs& p, int g) {
    Group x;
    x.b0 = min(max(p.cug[g], 0), p.m.B);
    x.b1 = min(max(p.cug[g + 1], x.b0), p.m.B);
    x.keys = x.b1 > x.b0 ? min(max(p.same[g], 0), p.m.max_keys) : 0;
    return x;
}
// Keys that sequence b shares with its group.
__device__ __forceinline__ int shared_of(const GroupArgs& p, int b) {
    if (p.groups == 0) return 0;
    // the last group that starts at b or before it
    int lo = 0, hi = p.groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cug[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    const Group x = load_group(p, lo);
    return b >= x.b0 && b < x.b1 ? x.keys : 0;
}

// Entry v of the list of groups and then sequences: rows, first key, keys from there on.
struct Entry {
    Seq s;
    int begin, keys, tiles;
    int b0, b1;     // (group) its sequences
    bool even;      // (sequence) its first token sees all that is shared
};
// (128 or 32 rows to a tile)
__device__ __forceinline__ int tiles_for(int each, int rows) { return (rows + each - 1) >> (each == 128 ? 7 : 5); }
// The rows of a group.
__device__ __forceinline__ void group_rows(const GroupArgs& p, Entry& x, int first, int end) {
    x.s.first = first;
    x.s.n = max(end - first, 0);
    x.tiles = x.keys > 0 ? tiles_for(p.rows, x.s.n * p.m.G) : 0;
}
// rows: also those of a group, which take one more load after the others.
__device__ __forceinline__ Entry load_entry(const GroupArgs& p, int v, bool rows) {
    Entry x{};
    x.even = true;
    if (v < p.groups) {
        const Group y = load_group(p, v);
        x.keys = x.s.kv = y.keys;
        x.b0 = y.b0;
        x.b1 = y.b1;
        if (rows) group_rows(p, x, min(max(p.m.cu[y.b0], 0), p.m.T), min(max(p.m.cu[y.b1], 0), p.m.T));
    } else if (v < p.groups + p.m.B) {
        x.s = load_seq(p.m, v - p.groups);
        x.begin = shared_of(p, v - p.groups);
        x.keys = max(x.s.kv - x.begin, 0);
        x.tiles = tiles_for(p.own_rows, x.s.n * p.m.G);
        x.even = x.s.n == 0 || visible(p.m, x.s, 0) >= x.begin;
    }
    return x;
}

__global__ __launch_bounds__(kThreads) void prefix_list(GroupArgs p) {
    __shared__ float work_s[kWaves], units_s[kTries];
    __shared__ Entry entry_s[kThreads];
    __shared__ int ends_s[kThreads], odd_s[kThreads], splits_s[kThreads], owner_s[kThreads], length_s[kTries];
    __shared__ int scan_s[2][kWaves], longest_s[kWaves], chunk_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), all = p.groups + p.m.B;
    // work and the longest entry; the first 1024 entries stay in LDS
    Entry x{};
    float work = 0.0f;
    int longest = 0;
    const bool held = all <= kThreads;       // all of them
    auto count = [&](const Entry& y) {
        work += (float)y.tiles * (float)y.keys;
        if (y.tiles > 0) longest = max(longest, y.keys);
    };
    x = load_entry(p, tid, !held);
    entry_s[tid] = x;
    if (held) {
        __syncthreads();
        if (tid < p.groups) {
            // (row b's place is the end of row b - 1; an empty group stands in its place among the others)
            auto place = [&](int b) {
                if (b == 0) return entry_s[p.groups].s.first;
                const Seq y = entry_s[p.groups + b - 1].s;
                return y.first + y.n;
            };
            group_rows(p, x, place(x.b0), place(x.b1));
        }
        __syncthreads();
        if (tid < p.groups) entry_s[tid] = x;
    }
    count(x);
    for (int v0 = kThreads; v0 < all; v0 += kThreads) count(load_entry(p, v0 + tid, true));
    auto add = [](float a, float b) { return a + b; };
    work = fold_wave(work, 0.0f, add);
    auto most_of = [](int a, int b) { return max(a, b); };
    longest = fold_wave(longest, 0, most_of);
    if (lane == 0) {
        work_s[wave] = work;
        longest_s[wave] = longest;
    }
    __syncthreads();
    // (a lane to a wave: a loop over them all is five times the code, and code that is run once waits to be fetched)
    work = fold_wave(lane < kWaves ? work_s[lane] : 0.0f, 0.0f, add);
    longest = fold_wave(lane < kWaves ? longest_s[lane] : 0, 0, most_of);
    // the ranges' lengths that are tried, and the units that each of them makes
    const int ways = kWays.n[lane % kTries];
    const int c = max(2, ((longest + ways - 1) / ways + p.step - 1) / p.step) * p.step;
    if (wave == 0 && lane < kTries) length_s[lane] = c;
    for (int k = wave; k < kTries; k += kWaves) {
        const int len = __builtin_amdgcn_readlane(c, k);
        const float inv = 1.0f / (float)len;
        float n = 0.0f;              // (exact up to 2^24, more than a launch may have)
        for (int v0 = 0; v0 < all; v0 += 64) {
            const int v = v0 + lane;
            int t, keys;
            if (v < kThreads) {
                t = entry_s[v].tiles;
                keys = entry_s[v].keys;
            } else {
                const Entry y = load_entry(p, v, true);
                t = y.tiles;
                keys = y.keys;
            }
            n += (float)t * (float)ranges_of(keys, len, inv);
        }
        n = fold_wave(n, 0.0f, add);
        if (lane == 0) units_s[k] = n;
    }
    __syncthreads();
    if (wave == 0) {
        const float n = units_s[lane % kTries];
        const float most = (float)min(c, max(longest, 1)), load = (work + n * kPrice) / (float)p.share;
        float price = n <= (float)p.share ? most + kPrice : load + most;
        if (n > (float)p.units && lane > 0) price = 3.0e38f;       // (whole entries always fit)
        const float best = fold_wave(price, 3.0e38f, [](float a, float b) { return fminf(a, b); });
        if (lane == 0) chunk_s = length_s[0];
        const uint64_t at = __ballot(price == best);
        if (at != 0 && lane == __builtin_ctzll(at)) chunk_s = c;
    }
    __syncthreads();
    const int chunk = chunk_s;

    int base = 0;
    for (int v0 = 0; v0 < all; v0 += kThreads) {
        if (v0 > 0) {
            x = load_entry(p, v0 + tid, true);
            entry_s[tid] = x;
        }
        const int v = v0 + tid, splits = ranges_of(x.keys, chunk, 1.0f / (float)chunk);
        // The shared keys are read by the table row of the first sequence of the group whose cache holds them all, of
        // the longest where none does: mostly the first one; else (padding may stand first) the wave looks for it, 64
        // sequences at a time.
        auto cached = [&](int b) { return held ? entry_s[p.groups + b].s.kv : min(max(p.m.kv[b], 0), p.m.max_keys); };
        int owner = x.b0;
        for (uint64_t todo = __ballot(x.b1 > x.b0 && x.tiles > 0 && cached(x.b0) < x.keys); todo != 0; todo &= todo - 1) {
            const int at = __builtin_ctzll(todo), keys = __builtin_amdgcn_readlane(x.keys, at);
            const int b0 = __builtin_amdgcn_readlane(x.b0, at), b1 = __builtin_amdgcn_readlane(x.b1, at);
            int found = b0, most = -1;
            for (int b = b0; b < b1 && most < keys; b += 64) {
                const int kv = b + lane < b1 ? min(cached(b + lane), keys) : -1, top = fold_wave(kv, -1, most_of);
                if (top > most) {
                    most = top;
                    found = b + __builtin_ctzll(__ballot(kv == top));
                }
            }
            if (lane == at) owner = found;
        }
        owner_s[tid] = owner;
        // units and sequences that see less than is shared, counted up to each entry
        // (lengths that contradict each other may add up to anything: no sum passes kMost)
        const int mine = (int)min((int64_t)x.tiles * splits, (int64_t)kMost);
        int ends = scan_upto(mine, kMost), odd = scan_incl(x.even ? 0 : 1);
        if (lane == 63) {
            scan_s[0][wave] = ends;
            scan_s[1][wave] = odd;
        }
        __syncthreads();
        const int e_to = scan_upto(lane < kWaves ? scan_s[0][lane] : 0, kMost), o_to = scan_incl(lane < kWaves ? scan_s[1][lane] : 0);
        if (wave > 0) {
            ends = add_to(ends, __builtin_amdgcn_readlane(e_to, wave - 1), kMost);
            odd += __builtin_amdgcn_readlane(o_to, wave - 1);
        }
        ends = add_to(base, ends, kMost);
        ends_s[tid] = ends;
        odd_s[tid] = odd;
        splits_s[tid] = splits;
        if (v < all) p.entries[v] = PrefixEntry{x.s.first, x.s.n, ends - mine, splits, x.begin, x.s.kv, x.s.len, chunk};
        __syncthreads();
        const int top = ends_s[kThreads - 1];
        for (int id = base + tid; id < min(top, p.units); id += kThreads) {
            int lo = 0, hi = min(all - v0, kThreads) - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (ends_s[mid] > id) hi = mid;
                else lo = mid + 1;
            }
            const int e = v0 + lo, s = splits_s[lo], rest = id - (lo > 0 ? ends_s[lo - 1] : base);
            const Entry y = entry_s[lo];
            int back = (int)((float)rest / (float)s);          // (off by one at most)
            back += back * s > rest ? -1 : (back + 1) * s <= rest ? 1 : 0;
            PrefixUnit u{};
            u.first = y.s.first; u.n = y.s.n; u.kv = y.s.kv; u.len = y.s.len;
            u.begin = y.begin; u.end = y.begin + y.keys;
            u.split = rest - back * s;
            u.tile = y.tiles - 1 - back;          // the last rows see most keys: they come first
            u.chunk = chunk;
            u.even = 1;
            u.b = e - p.groups;
            // (a row of a sequence that shares no keys and was not split has one part: it is written whole)
            u.splits = y.begin > 0 ? max(s, 2) : s;
            if (e < p.groups) {
                u.b = owner_s[lo];
                u.b0 = y.b0;
                u.b1 = y.b1;
                u.splits = max(s, 2);
                // (where the list is longer than the workgroup every row finds its sequence)
                u.even = all <= kThreads && odd_s[p.groups + y.b1 - 1] == odd_s[p.groups + y.b0 - 1];
            }
            // (nor do they lead outside the rows)
            if (u.tile < 0 || (int64_t)u.tile * (e < p.groups ? p.rows : p.own_rows) >= (int64_t)u.n * p.m.G) u.n = 0;
            p.list[id] = u;
        }
        base = top;
        __syncthreads();
    }
    for (int id = base + tid; id < p.units; id += kThreads) p.list[id].n = 0;
}

template <typename E, bool KV8, bool EXACT, bool WIDE> __global__ __launch_bounds__(256, 1) void prefix_latent(GroupArgs p) {
    latent_rows<E, KV8, EXACT, WIDE>(p);
}

// ---------------------------------------------------------------------------
// prefix_join: a row's parts, those against the shared keys and those against its
// sequence's own, on one scale (as attn_join).  Bound by latency: the row's place, its
// entry, its parts' sums, its parts (4096 rows of 9 to 10 parts: 10 us).
// ---------------------------------------------------------------------------
template <typename E, int NC, bool TOGETHER>
__global__ __launch_bounds__(256) void prefix_join(GroupArgs p) {
    __shared__ f32x4 share[TOGETHER ? 4 : 1][NC][64];
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    const int64_t all = (int64_t)p.m.T * p.m.G * p.m.Hkv;
    const int64_t stride = TOGETHER ? gridDim.x : (int64_t)gridDim.x * 4;
    // the last of n entries from `at` on whose rows start at t or before it: 64 at a time
    auto find = [&](int at, int n, int t) {
        int lo = 0, count = n;
        while (count > 1) {
            const int step = (count + 63) / 64, i = lo + lane * step;
            const uint64_t before = __ballot(lane * step < count && p.entries[at + min(i, n - 1)].first <= t);
            const int k = max(0, 63 - __builtin_clzll(before | 1));
            count = min(step, count - k * step);
            lo += k * step;
        }
        return at + lo;
    };
#pragma unroll 1
    for (int64_t id = TOGETHER ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave; id < all; id += stride) {
        const uint32_t at_row = fdiv((uint32_t)id, p.m.fHkv);
        const int hk = (int)((uint32_t)id - at_row * p.m.fHkv.d), t = (int)fdiv(at_row, p.m.fG), head = (int)at_row - t * p.m.G;
        // the row's group and its sequence: first slots and numbers of parts
        int slot[2] = {0, 0}, parts[2] = {0, 0}, in_tile[2] = {0, 0};
        // (both asked for before either is looked at)
        const int own = find(p.groups, p.m.B, t), group = find(0, p.groups, t);
        const PrefixEntry y = p.entries[own], g = p.entries[group];
        const bool found_seq = t >= y.first && t < y.first + y.n;
        const bool whole = y.splits == 1 && y.begin == 0;
        if (found_seq && !whole) {
            const int row = (t - y.first) * p.m.G + head, tile = row / p.own_rows;
            in_tile[1] = row - tile * p.own_rows;
            slot[1] = y.slot + (tiles_for(p.own_rows, y.n * p.m.G) - 1 - tile) * y.splits;     // (the last tile comes first)
            // the ranges that the tile's last row has keys in
            const int last = min((tile + 1) * p.own_rows, y.n * p.m.G) - 1;
            const int kend = visible(p.m, Seq{y.first, y.n, y.kv, y.len}, (int)fdiv((uint32_t)last, p.m.fG)) - y.begin;
            parts[1] = min(y.splits, max(1, (kend + y.chunk - 1) / y.chunk));
            if (y.begin > 0) {
                if (t >= g.first && t < g.first + g.n && g.kv > 0) {
                    const int grow = (t - g.first) * p.m.G + head, gtile = grow / p.rows;
                    in_tile[0] = grow - gtile * p.rows;
                    slot[0] = g.slot + (tiles_for(p.rows, g.n * p.m.G) - 1 - gtile) * g.splits;
                    parts[0] = g.splits;
                }
            }
        }
        if (!found_seq || whole) continue;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            if (slot[kind] < 0) parts[kind] = 0;
            parts[kind] = max(0, min(parts[kind], p.units - slot[kind]));
        }
        const int n = parts[0] + parts[1];
        const int64_t first0 = ((int64_t)hk * p.units + slot[0]) * p.rows + in_tile[0];
        const int64_t first1 = ((int64_t)hk * p.units + slot[1]) * p.rows + in_tile[1];
        auto part = [&](int k) { return k < parts[0] ? first0 + (int64_t)k * p.rows : first1 + (int64_t)(k - parts[0]) * p.rows; };
        join_parts<E, NC, TOGETHER>(p, share, t, hk * p.m.G + head, n, part);
    }
}

template <typename E>
hipError_t run_join(const GroupArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.m.T * a.m.G * a.m.Hkv;
    const dim3 block(256);
    if (rows <= 1024) {
        const dim3 grid((uint32_t)rows);
        return a.Dv <= 256 ? launch(prefix_join<E, 1, true>, grid, block, stream, a)
                           : launch(prefix_join<E, 2, true>, grid, block, stream, a);
    }
    const dim3 grid((uint32_t)(rows < 8192 ? (rows + 3) / 4 : 2048));
    return a.Dv <= 256 ? launch(prefix_join<E, 1, false>, grid, block, stream, a)
                       : launch(prefix_join<E, 2, false>, grid, block, stream, a);
}

template <typename E, bool KV8, bool WIDE> hipError_t run_latent(const GroupArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.units * a.m.Hkv)), block(256);
    return a.Dk == latent::DK ? launch(prefix_latent<E, KV8, true, WIDE>, grid, block, stream, a)
                              : launch(prefix_latent<E, KV8, false, WIDE>, grid, block, stream, a);
}

}  // namespace

int64_t prefix_list_bytes(int64_t units, int64_t entries) {
    return units * (int64_t)sizeof(PrefixUnit) + entries * (int64_t)sizeof(PrefixEntry);
}

AttnPlan plan_prefix(const Batch& m, int64_t groups, int Dk, int Dv, bool pieces) {
    AttnPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.latent = Dk > 256 || Dv > 256;
    // few rows a sequence: its own keys by 32 rows, as in plan_attn()
    pl.by_keys = !pl.latent && pieces && rows <= (int64_t)32 * m.B;
    pl.rows = 128;
    // row tiles, at most: of sequences, and once more of groups
    pl.tiles = (int32_t)(rows / (pl.by_keys ? 32 : 128) + m.B + rows / 128 + groups);
    // workgroups of a key head that run at once; up to twice as many key ranges beside the tiles
    const int64_t chip = pl.latent ? 256 : 512;
    pl.share = (int32_t)((chip + m.Hkv - 1) / m.Hkv);
    pl.slots = pl.tiles + 2 * pl.share;
    pl.units = pl.slots;
    pl.ws_bytes = prefix_list_bytes(pl.units, groups + m.B) + (int64_t)pl.units * m.Hkv * pl.rows * (Dv + 1) * 4;
    return pl;
}

hipError_t launch_prefix(const GroupArgs& arg, bool latent, bool bf16, bool kv8, bool wide, hipStream_t stream) {
    GroupArgs a = arg;
    a.step = latent || a.Dk > 128 || a.Dv > 128 ? 32 : 64;      // keys of a tile
    if (!latent && a.v == nullptr) {           // narrow rows: the values are read as columns of their own
        a.v = a.k;
        a.v_P = a.k_P; a.v_S = a.k_S; a.v_H = a.k_H;
    }
    hipError_t e = launch(prefix_list, dim3(1), dim3(kThreads), stream, a);
    if (e != hipSuccess) return e;
    if (!latent) e = bf16 ? launch_prefix_bf16(a, kv8, wide, stream) : launch_prefix_f16(a, kv8, wide, stream);
    else {
        auto with = [&](auto type, auto k) {
            using E = decltype(type);
            constexpr bool K8 = decltype(k)::value;
            return wide ? run_latent<E, K8, true>(a, stream) : run_latent<E, K8, false>(a, stream);
        };
        e = bf16 ? (kv8 ? with(BF16T{}, std::true_type{}) : with(BF16T{}, std::false_type{}))
                 : (kv8 ? with(F16T{}, std::true_type{}) : with(F16T{}, std::false_type{}));
    }
    if (e != hipSuccess) return e;
    return bf16 ? run_join<BF16T>(a, stream) : run_join<F16T>(a, stream);
}

}  // namespace dcpa
