// attn_prefix.hip -- attention of a batch whose sequences share the first keys
// of their caches, group by group.
//
// The rows of all sequences of a group stand together, so against the shared
// keys they are one long sequence: its row tiles take the shared keys once for
// 128 rows of whichever sequences, and every sequence's own tiles take the keys
// behind them.  Both are units of one launch of the kernels for many rows
// (attn_rows.hpp, attn_latent.hpp), which differ only in how a workgroup finds
// its share and in what a row sees; a row's parts are joined by a second kernel.
#include "attn_latent.hpp"
#include "attn_rows.hpp"

namespace dcpa {

// A workgroup's share: rows of one sequence against its own keys, or rows of a
// group against the keys that its sequences share.
struct GroupUnit : Unit {
    int begin;      // first key
    int end;        // one behind the last shared key (group)
    int b0, b1;     // the group's sequences (none: a sequence's own keys)
    bool even;      // every row of the group sees all shared keys
};

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
    // the last group that starts at b or before it
    int lo = 0, hi = p.groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cug[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    if (p.groups == 0) return 0;
    const Group x = load_group(p, lo);
    return b >= x.b0 && b < x.b1 ? x.keys : 0;
}

// Entry v of the list of groups and then sequences: rows, first key, keys from there on.
struct Entry {
    Seq s;
    int begin, keys, tiles;
};
__device__ __forceinline__ Entry load_entry(const GroupArgs& p, int v, int rows) {
    Entry x{};
    if (v < p.groups) {
        const Group y = load_group(p, v);
        if (y.keys > 0) {
            x.s.first = min(max(p.m.cu[y.b0], 0), p.m.T);
            x.s.n = min(max(p.m.cu[y.b1], x.s.first), p.m.T) - x.s.first;
            x.keys = x.s.kv = y.keys;
        }
    } else if (v < p.groups + p.m.B) {
        x.s = load_seq(p.m, v - p.groups);
        x.begin = shared_of(p, v - p.groups);
        x.keys = max(x.s.kv - x.begin, 0);
    }
    x.tiles = (x.s.n * p.m.G + rows - 1) / rows;
    return x;
}

// As key_chunk() and find_unit(), over that list.
template <int STEP> __device__ __forceinline__ int group_chunk(const GroupArgs& p, int rows) {
    if (p.slots <= 0) return kWhole;
    const int lane = threadIdx.x & 63, all = p.groups + p.m.B;
    int64_t work = 0;
    int tiles = 0;
    Entry x;
    for (int v0 = 0; v0 < all; v0 += 64) {
        x = load_entry(p, v0 + lane, rows);
        work += (int64_t)x.tiles * x.keys;
        tiles += x.tiles;
    }
    work = sum_wave(work);
    tiles = (int)sum_wave((int64_t)tiles);
    if (tiles >= p.slots) return kWhole;
    auto steps = [](int64_t x) { return (int)min((int64_t)(kWhole / STEP), max((int64_t)2, (x + STEP - 1) / STEP)); };
    int lo = steps((work + p.share - 1) / p.share), hi = max(lo, steps((work + p.slots - tiles - 1) / (p.slots - tiles)));
#pragma unroll 1
    for (int round = 0; round < 3 && lo < hi; ++round) {
        const int mid = lo + (hi - lo) / 2;
        int64_t units = 0;
        for (int v0 = 0; v0 < all; v0 += 64) {
            if (all > 64) x = load_entry(p, v0 + lane, rows);
            units += (int64_t)x.tiles * max(1, (x.keys + mid * STEP - 1) / (mid * STEP));
        }
        units = sum_wave(units);
        if (units <= p.slots) hi = mid;
        else lo = mid + 1;
    }
    return hi * STEP;
}

template <int STEP> __device__ __forceinline__ GroupUnit unit_of(const GroupArgs& p, int rows, int id) {
    GroupUnit u;
    u.ok = false;
    u.chunk = group_chunk<STEP>(p, rows);
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int v0 = 0; v0 < p.groups + p.m.B; v0 += 64) {
        const Entry x = load_entry(p, v0 + lane, rows);
        const int splits = max(1, (x.keys + u.chunk - 1) / u.chunk);
        const int incl = base + scan_incl(x.tiles * splits);
        const uint64_t past = __ballot(incl > id);
        if (past != 0) {
            const int at = __builtin_ctzll(past), v = v0 + at;
            const int t = __builtin_amdgcn_readlane(x.tiles, at), s = __builtin_amdgcn_readlane(splits, at);
            const int rest = id - (__builtin_amdgcn_readlane(incl, at) - t * s);
            u.s = seq_of(x.s, at);
            u.begin = __builtin_amdgcn_readlane(x.begin, at);
            u.end = u.begin + __builtin_amdgcn_readlane(x.keys, at);
            u.split = rest % s;
            u.tile = t - 1 - rest / s;
            u.slot = id - u.split;
            u.ok = rest >= 0 && u.tile >= 0 && (int64_t)u.tile * rows < (int64_t)u.s.n * p.m.G;
            u.b0 = u.b1 = 0;
            u.even = true;
            u.b = v - p.groups;
            // (a row of a sequence that shares no keys and was not split has one part: it is written whole)
            u.splits = u.begin > 0 ? max(s, 2) : s;
            if (v < p.groups) {
                const Group y = load_group(p, v);
                u.b = u.b0 = y.b0;
                u.b1 = y.b1;
                u.splits = max(s, 2);
                for (int b = y.b0; b < y.b1; b += 64) {
                    bool all = true;
                    if (b + lane < y.b1) {
                        const Seq q = load_seq(p.m, b + lane);
                        all = q.n == 0 || visible(p.m, q, 0) >= u.end;
                    }
                    if (__ballot(!all) != 0) u.even = false;
                }
            }
            return u;
        }
        base = __builtin_amdgcn_readlane(incl, 63);
    }
    return u;
}
__device__ __forceinline__ int first_key(const GroupUnit& u) { return u.begin; }
__device__ __forceinline__ int last_key(const GroupArgs& p, const GroupUnit& u, int last_row) {
    return u.b1 > u.b0 ? u.end : visible(p.m, u.s, (int)fdiv((uint32_t)last_row, p.m.fG));
}
__device__ __forceinline__ int sees(const GroupArgs& p, const GroupUnit& u, int token) {
    if (u.b1 == u.b0) return visible(p.m, u.s, token);
    if (u.even) return u.end;
    // the last sequence that starts at the token's row or before it
    const int t = u.s.first + token;
    int lo = u.b0, hi = u.b1 - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (min(max(p.m.cu[mid], 0), p.m.T) <= t) lo = mid;
        else hi = mid - 1;
    }
    const Seq s = load_seq(p.m, lo);
    return min(visible(p.m, s, t - s.first), u.end);
}
// (rows of several sequences are in no order)
__device__ __forceinline__ int least_seen(const GroupUnit&, int vis) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) vis = min(vis, __shfl_xor(vis, d, 64));
    return __builtin_amdgcn_readfirstlane(vis);
}
__device__ __forceinline__ int most_seen(const GroupUnit&, int vis) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) vis = max(vis, __shfl_xor(vis, d, 64));
    return __builtin_amdgcn_readfirstlane(vis);
}

namespace {

template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, bool WIDE>
__global__ __launch_bounds__(256, DK > 192 ? 1 : 2) void prefix_rows(GroupArgs p) {
    rows_of<E, KV8, EXACT, DK, DV, KT, WIDE>(p);
}
template <typename E, bool KV8, bool EXACT, bool WIDE> __global__ __launch_bounds__(256, 1) void prefix_latent(GroupArgs p) {
    latent_rows<E, KV8, EXACT, WIDE>(p);
}

// ---------------------------------------------------------------------------
// prefix_join: a row's parts, those against the shared keys and those against its
// sequence's own, on one scale (as attn_join).
// ---------------------------------------------------------------------------
template <typename E, int STEP, int NC, bool TOGETHER>
__global__ __launch_bounds__(256) void prefix_join(GroupArgs p) {
    constexpr int FLY = NC == 1 ? 8 : 4;       // parts under way at once
    __shared__ f32x4 share[TOGETHER ? 4 : 1][NC][64];
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    const int chunk = group_chunk<STEP>(p, p.rows);
    const int64_t all = (int64_t)p.m.T * p.m.G * p.m.Hkv;
    const int64_t stride = TOGETHER ? gridDim.x : (int64_t)gridDim.x * 4;
#pragma unroll 1
    for (int64_t id = TOGETHER ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave; id < all; id += stride) {
        const uint32_t at_row = fdiv((uint32_t)id, p.m.fHkv);
        const int hk = (int)((uint32_t)id - at_row * p.m.fHkv.d), t = (int)fdiv(at_row, p.m.fG), head = (int)at_row - t * p.m.G;
        // the row's group and its sequence: first slots and numbers of parts
        int slot[2] = {0, 0}, parts[2] = {0, 0}, in_tile[2] = {0, 0};
        bool whole = false, found_seq = false;
        int base = 0;
        for (int v0 = 0; v0 < p.groups + p.m.B && !found_seq; v0 += 64) {
            const Entry x = load_entry(p, v0 + lane, p.rows);
            const int splits = max(1, (x.keys + chunk - 1) / chunk);
            const int incl = base + scan_incl(x.tiles * splits);
            base = __builtin_amdgcn_readlane(incl, 63);
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                const bool mine = (v0 + lane < p.groups) == (kind == 0) && t >= x.s.first && t < x.s.first + x.s.n;
                const uint64_t found = __ballot(mine);
                if (found == 0) continue;
                const int at = __builtin_ctzll(found);
                const Seq s = seq_of(x.s, at);
                const int ns = __builtin_amdgcn_readlane(splits, at), begin = __builtin_amdgcn_readlane(x.begin, at);
                const int row = (t - s.first) * p.m.G + head, tile = row / p.rows;
                in_tile[kind] = row - tile * p.rows;
                // (the last tile comes first)
                slot[kind] = __builtin_amdgcn_readlane(incl, at) - (tile + 1) * ns;
                parts[kind] = ns;
                if (kind == 1) {
                    found_seq = true;
                    whole = ns == 1 && begin == 0;
                    // the ranges that the tile's last row has keys in
                    const int last = min((tile + 1) * p.rows, s.n * p.m.G) - 1;
                    const int kend = visible(p.m, s, (int)fdiv((uint32_t)last, p.m.fG)) - begin;
                    parts[1] = min(ns, max(1, (kend + chunk - 1) / chunk));
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
        float top = -INFINITY;
        bool bad = false;
        for (int k = lane; k < n; k += 64) {
            const float y = p.ws_l[part(k)];
            bad |= y != y;
            top = fmaxf(top, y);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        const float ref = top == -INFINITY ? 0.0f : top;
        float acc[NC * 4], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC * 4; ++i) acc[i] = 0.0f;
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += 64) {
            // a lane to a part's weight
            const int here = min(64, n - k0);
            const float f = lane < here ? exp2_fast(p.ws_l[part(k0 + lane)] - ref) : 0.0f;
            sum += f;
#pragma unroll 1
            for (int k = TOGETHER ? wave * FLY : 0; k < here; k += TOGETHER ? 4 * FLY : FLY) {
                f32x4 y[FLY][NC];
#pragma unroll
                for (int i = 0; i < FLY; ++i)
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        const int col = min(j * 256 + lane * 4, p.Dv - 4);
                        y[i][j] = *(const f32x4*)(p.ws_o + part(k0 + min(k + i, here - 1)) * p.Dv + col);
                    }
#pragma unroll
                for (int i = 0; i < FLY; ++i) {
                    const float g = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), min(k + i, 63)));
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[j * 4 + c] += k + i < here ? g * y[i][j][c] : 0.0f;
                }
            }
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (__ballot(bad) != 0) sum = NAN;
        if constexpr (TOGETHER) {
#pragma unroll
            for (int j = 0; j < NC; ++j) share[wave][j][lane] = f32x4{acc[j * 4], acc[j * 4 + 1], acc[j * 4 + 2], acc[j * 4 + 3]};
            __syncthreads();
            if (wave == 0)
#pragma unroll
                for (int j = 0; j < NC; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[j * 4 + c] = share[0][j][lane][c] + share[1][j][lane][c] + share[2][j][lane][c] + share[3][j][lane][c];
            __syncthreads();
            if (wave != 0) continue;
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        char* o = p.out + (int64_t)t * p.o_T + (int64_t)(hk * p.m.G + head) * p.o_H;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int col = j * 256 + lane * 4;
            if (col < p.Dv)
                store4<E>(o + col * 2, acc[j * 4] * inv, acc[j * 4 + 1] * inv, acc[j * 4 + 2] * inv, acc[j * 4 + 3] * inv);
        }
        if (lane == 0 && p.lse != nullptr)
            p.lse[(int64_t)t * p.l_T + (int64_t)(hk * p.m.G + head) * p.l_H] =
                (sum == 0.0f ? -INFINITY : ref + __builtin_amdgcn_logf(sum)) * p.lmul;
    }
}

template <typename E, int STEP>
hipError_t run_join(const GroupArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.m.T * a.m.G * a.m.Hkv;
    const dim3 block(256);
    if (rows <= 1024) {
        const dim3 grid((uint32_t)rows);
        return a.Dv <= 256 ? launch(prefix_join<E, STEP, 1, true>, grid, block, stream, a)
                           : launch(prefix_join<E, STEP, 2, true>, grid, block, stream, a);
    }
    const dim3 grid((uint32_t)(rows < 8192 ? (rows + 3) / 4 : 2048));
    return a.Dv <= 256 ? launch(prefix_join<E, STEP, 1, false>, grid, block, stream, a)
                       : launch(prefix_join<E, STEP, 2, false>, grid, block, stream, a);
}

template <typename E, bool KV8, bool WIDE>
hipError_t run(const GroupArgs& a, bool latent, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.units * a.m.Hkv)), block(256);
    hipError_t e;
    if (latent) {
        e = a.Dk == latent::DK ? launch(prefix_latent<E, KV8, true, WIDE>, grid, block, stream, a)
                               : launch(prefix_latent<E, KV8, false, WIDE>, grid, block, stream, a);
        return e != hipSuccess ? e : run_join<E, 32>(a, stream);
    }
    const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
    if (d <= 64) {
        e = launch(prefix_rows<E, KV8, false, 64, 64, 64, WIDE>, grid, block, stream, a);
        return e != hipSuccess ? e : run_join<E, 64>(a, stream);
    }
    if (d <= 128) {
        e = a.Dk == 128 && a.Dv == 128 ? launch(prefix_rows<E, KV8, true, 128, 128, 64, WIDE>, grid, block, stream, a)
                                       : launch(prefix_rows<E, KV8, false, 128, 128, 64, WIDE>, grid, block, stream, a);
        return e != hipSuccess ? e : run_join<E, 64>(a, stream);
    }
    e = a.Dk <= 192 && a.Dv <= 128 ? launch(prefix_rows<E, KV8, false, 192, 128, 32, WIDE>, grid, block, stream, a)
                                   : launch(prefix_rows<E, KV8, false, 256, 256, 32, WIDE>, grid, block, stream, a);
    return e != hipSuccess ? e : run_join<E, 32>(a, stream);
}

}  // namespace

AttnPlan plan_prefix(const Batch& m, int64_t groups, int Dk, int Dv) {
    AttnPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.latent = Dk > 256 || Dv > 256;
    pl.by_keys = false;
    pl.rows = 128;
    // row tiles, at most: of sequences, and once more of groups
    pl.tiles = (int32_t)(2 * (rows / pl.rows) + m.B + groups);
    const int64_t chip = pl.latent ? 256 : 512;
    pl.share = (int32_t)((chip + m.Hkv - 1) / m.Hkv);
    pl.slots = pl.tiles + pl.share;
    pl.units = pl.slots;
    pl.ws_bytes = (int64_t)pl.units * m.Hkv * pl.rows * (Dv + 1) * 4;
    return pl;
}

hipError_t launch_prefix(const GroupArgs& arg, bool latent, bool bf16, bool kv8, bool wide, hipStream_t stream) {
    GroupArgs a = arg;
    if (!latent && a.v == nullptr) {           // narrow rows: the values are read as columns of their own
        a.v = a.k;
        a.v_P = a.k_P; a.v_S = a.k_S; a.v_H = a.k_H;
    }
    auto with = [&](auto e, auto k) {
        using E = decltype(e);
        constexpr bool K8 = decltype(k)::value;
        return wide ? run<E, K8, true>(a, latent, stream) : run<E, K8, false>(a, latent, stream);
    };
    if (bf16) return kv8 ? with(BF16T{}, std::true_type{}) : with(BF16T{}, std::false_type{});
    return kv8 ? with(F16T{}, std::true_type{}) : with(F16T{}, std::false_type{});
}

}  // namespace dcpa
