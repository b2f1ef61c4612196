// attn_mass.hip -- accumulated attention weight of every cached key.
//
// For one key head and a key j, the sum over the rows that see it of
// 2^(s_j c - g), g the row's merged log-sum-exp in powers of two.  Scores are
// computed transposed as in attn_tile.hpp: a wave holds the fragments of its
// keys in registers (A operand) and walks over the query rows, 32 at a time out
// of LDS (B operand); each lane adds up the weights of its own query rows, and
// one sum over the 32 lanes at the end gives the keys' totals.  No two waves
// write the same key, so there are no atomics.
//
// Few rows (decode, mass_few) are bound by the bytes of the keys, which come
// straight into LDS, the next tile of 32 while the present one is multiplied
// (loaded into registers as fragments, 32 rows of 32 bytes to an instruction,
// the same bytes took twice as long): decode of 16 sequences of up to 16384 keys,
// 8 key heads of 128, 59 us, 4.3 TB/s (65 us with each head on an XCD of its own).  Many rows (mass_rows) are
// bound by the instructions of a weight (for 64 of them 8 clocks for the power, 4 to
// scale and 4 to add, beside 16 of matrix instructions at 128 columns; the two
// interleaved take 1.3 times the products alone) and by a barrier with a full wait
// for every 32 rows:
// 64 keys to a wave, so that a fragment of queries is read from LDS once for two
// products.  Where the batch has fewer key steps than the chip has room for, the
// rows are split, and mass_join adds the parts in order.
#include "attn_device.hpp"

namespace dcpa {

namespace {

// A batch's layout over workgroups: each takes the keys [split chunk, (split +
// 1) chunk) of a sequence, `keys` at a time, against part `part` of its rows.
// Every wave works it out from the lengths on the device, as find_unit().  Rows
// are only split where there is a workspace for the parts.
struct Share {
    Seq s;
    int b, k0, k1, slot, part, parts;
    bool ok;
};

constexpr int kOneTile = 0x3fffffff;      // rows of a tile that holds any sequence

template <int KEYS>
__device__ __forceinline__ void share_out(const Batch& m, int slots, int share, bool split_rows, int& chunk, int& parts) {
    const int lane = threadIdx.x & 63;
    int64_t steps = 0;
    int most = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64)
        if (b0 + lane < m.B) {
            const Seq s = load_seq(m, b0 + lane);
            if (s.n > 0) steps += max(1, (s.kv + KEYS - 1) / KEYS);
            most = max(most, s.n);
        }
    steps = sum_wave(steps);
    parts = 1;
    chunk = KEYS;
    if (steps >= slots) {
        chunk = key_chunk<KEYS>(m, kOneTile, slots, share);
        return;
    }
    if (!split_rows) return;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) most = max(most, __shfl_xor(most, d, 64));
    most = __builtin_amdgcn_readfirstlane(most);
    // (at least four row tiles to a part)
    const int64_t tiles = ((int64_t)most * m.G + 127) / 128;
    parts = (int)max((int64_t)1, min(slots / max((int64_t)1, steps), tiles));
}

template <int KEYS> __device__ __forceinline__ Share find_share(const Batch& m, int slots, int share, bool split_rows, int id) {
    Share u;
    u.ok = false;
    int chunk;
    share_out<KEYS>(m, slots, share, split_rows, chunk, u.parts);
    u.part = id % u.parts;
    id /= u.parts;
    u.slot = id;
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64) {
        int n = 0, kv;
        tiles_of(m, b0 + lane, kOneTile, n, kv);
        if (n > 0) n = max(1, (kv + chunk - 1) / chunk);
        const int incl = base + scan_incl(n);
        const uint64_t past = __ballot(incl > id);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            u.b = b0 + at;
            u.s = load_seq(m, u.b);
            const int split = id - (__builtin_amdgcn_readlane(incl, at) - __builtin_amdgcn_readlane(n, at));
            u.k0 = split * chunk;
            u.k1 = (int)min((int64_t)u.s.kv, (int64_t)u.k0 + chunk);
            u.ok = split >= 0 && u.k0 < u.k1 && u.s.n > 0;
            return u;
        }
        base = __builtin_amdgcn_readlane(incl, 63);
    }
    return u;
}

__device__ __forceinline__ float* mass_at(const MassArgs& p, int b, int hk, int key) {
    const uint32_t page = fdiv((uint32_t)key, p.m.fpage);
    const int id = p.m.table[(int64_t)b * p.m.t_B + page];
    if ((uint32_t)id >= (uint32_t)p.m.pages) return nullptr;
    return p.mass + (int64_t)id * p.m_P + (int64_t)(key - (int)(page * p.m.fpage.d)) * p.m_S + (int64_t)hk * p.m_H;
}

// KW keys to a wave.  The weights of one tile of rows are worked out between the
// matrix instructions of the next, whose scores go to the other of two sets of
// registers: alone, a SIMD takes 16 clocks for 64 weights (8 of them the power)
// and 16 for the products of 64 scores at 128 columns; in turn, with a barrier
// to a tile, two waves to a SIMD overlapped them by less than half (159 us for
// 2 x 4096 rows against 2 x 8192 keys of 8 heads; now 127 us, 0.7 PFLOP/s).  A
// deeper ring of tiles took more scalar registers than there are (144 us).
template <typename E, bool KV8, int DK, int KW>
__global__ __launch_bounds__(256, DK > 256 ? 1 : 2) void mass_rows(MassArgs p) {
    constexpr int KEYS = 4 * KW, NB = KW / 32, ST = DK / 16, KC = DK / 8, QROW = KC * 16, QB = 32 * QROW, NQ = 32 * KC / 256 + (32 * KC % 256 != 0);
    constexpr int PAD = NQ * 256 * 16;         // whole rounds of the workgroup
    constexpr int AHEAD = 3;                   // query fragments read ahead of their products
    __shared__ __attribute__((aligned(1024))) char qtile[2][PAD];
    static_assert(QB <= PAD, "a tile of queries fits");
    const int hk = (int)(blockIdx.x % (uint32_t)p.m.Hkv);
    const Share u = find_share<KEYS>(p.m, p.slots, p.share, p.ws != nullptr, (int)(blockIdx.x / (uint32_t)p.m.Hkv));
    if (!u.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, tiles = (nrows + 31) / 32, per_part = (tiles + u.parts - 1) / u.parts;
    const int first_tile = u.part * per_part, end_tile = min(tiles, first_tile + per_part);
    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;

    // the wave's keys from k0 on as A operands; absent ones are zeros (and masked by their place)
    auto load_keys = [&](int k0, u32x4 (&kf)[NB][ST], uint32_t (&there)[NB]) {
        const MassArgs& e = late_args<MassArgs>();
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            const int key = k0 + wave * KW + kb * 32 + r;
            const uint32_t page = fdiv((uint32_t)key, e.m.fpage);
            const int id = key < u.k1 ? table[page] : -1;
            const bool have = (uint32_t)id < (uint32_t)e.m.pages;
            there[kb] = (uint32_t)__ballot(h == 0 && have);
            const uint64_t row = have ? (uint64_t)(e.k + (int64_t)id * e.k_P +
                                                   (int64_t)(key - (int)(page * e.m.fpage.d)) * e.k_S + (int64_t)hk * e.k_H)
                                      : (uint64_t)kZeros;
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                const int c = 2 * s + h;
                const uint64_t at = at_or_zeros(c * 8 < e.Dk, row + (uint64_t)(c * (KV8 ? 8 : 16)));
                if constexpr (KV8) {
                    const u32x2 x = *(const u32x2*)at;
                    kf[kb][s].x = x.x;
                    kf[kb][s].y = x.y;
                } else {
                    kf[kb][s] = *(const u32x4*)at;
                }
            }
        }
    };
    const uint32_t lds0 = lds_addr(&qtile[0][0]);
    // Rows follow each other tile by tile, 32 on: their addresses are carried along, since the division and
    // the products of an address take 16 clocks each.
    struct Place {
        int row, sub;       // of the tile; head within the key head's
        uint64_t at;
    };
    const int G = p.m.G, next_t = (int)fdiv(32u, p.m.fG), next_g = 32 - next_t * G;
    auto place_of = [&](int t, int row, const void* base, int64_t s_T, int64_t s_H) {
        const int token = (int)fdiv((uint32_t)(t * 32 + row), p.m.fG), g = t * 32 + row - token * G;
        return Place{row, g, (uint64_t)base + (uint64_t)((u.s.first + token) * s_T + (hk * G + g) * s_H)};
    };
    auto advance = [&](Place& x, int64_t s_T, int64_t s_H) {
        x.at += (uint64_t)(next_t * s_T + next_g * s_H);
        if (next_g != 0) {
            x.sub += next_g;
            const bool wrap = x.sub >= G;
            x.sub -= wrap ? G : 0;
            x.at += wrap ? (uint64_t)(s_T - G * s_H) : 0;
        }
    };
    // the pieces of the row tile that this lane brings (columns that are not there: a row that never is), and
    // the row that it weighs
    Place piece[NQ], mine;
    auto start_at = [&](int t) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int ch = i * 256 + tid, row = min(ch / KC, 31), c = (ch % KC) ^ swz<KC>(row);
            piece[i] = place_of(t, row, p.q + c * 16, p.q_T, p.q_H);
            if (c * 8 >= p.Dk) piece[i].row = 32;
        }
        mine = place_of(t, r, p.lse, p.l_T * 4, p.l_H * 4);
    };
    // row tile t, whose turn it is, into buffer b, and this lane's log-sum-exp in powers of two
    auto fetch = [&](int t, int b, float& g) {
        const int left = min(nrows - t * 32, 32);
        g = *(const __attribute__((address_space(1))) float*)at_or_zeros(mine.row < left, mine.at);
        advance(mine, p.l_T * 4, p.l_H * 4);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            dma16((const char*)at_or_zeros(piece[i].row < left, piece[i].at), lds0 + (uint32_t)(b * PAD + (i * 256 + wave * 64) * 16));
            advance(piece[i], p.q_T, p.q_H);
        }
    };

    // rows that see none of the range come first: skip their tiles
    int lo = first_tile, hi = end_tile;
    while (lo < hi) {
        const int mid = (lo + hi) / 2, last = min(mid * 32 + 31, nrows - 1);
        if (visible(p.m, u.s, (int)fdiv((uint32_t)last, p.m.fG)) > u.k0) hi = mid;
        else lo = mid + 1;
    }
    const int begin = lo;
    const bool single = end_tile - begin <= 1;     // one tile of rows for all the keys: it stays in LDS
    u32x4 kf[NB][ST];
    uint32_t there[NB] = {};
    float g_next = 0.0f;
#pragma unroll 1
    for (int k0 = u.k0; k0 < u.k1; k0 += KEYS) {
        const bool fresh = !single || k0 == u.k0;
        if (begin < end_tile) {
            if (fresh) {
                meet();       // (other waves may still read the last keys' tiles)
                start_at(begin);
                fetch(begin, 0, g_next);
            }
            load_keys(k0, kf, there);
        }
        const int key0 = k0 + wave * KW;
        float acc[NB][16];
        f32x16 s0[NB], s1[NB];
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[kb][i] = s0[kb][i] = s1[kb][i] = 0.0f;
        if constexpr (KV8) {
#pragma unroll
            for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                for (int s = 0; s < ST; ++s) kf[kb][s] = widen8<E>(u32x2{kf[kb][s].x, kf[kb][s].y});
        }
        // (the keys are there from here on: else the wait for them would stand in the loop, and wait for tiles)
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int s = 0; s < ST; ++s) asm volatile("" : "+v"(kf[kb][s]));
        float g_old = INFINITY;       // (the first time there is nothing to weigh)
        auto weigh = [&](const f32x16 (&s)[NB], int j) {
            acc[j / 16][j % 16] += exp2_fast(__builtin_fmaf(s[j / 16][j % 16], p.c, -g_old));
            asm volatile("" : "+v"(acc[j / 16][j % 16]));     // (here, not where the sum is next used)
        };
        auto step = [&](int t, int buf, f32x16 (&now)[NB], const f32x16 (&old)[NB]) {
            if (fresh) {
                dma_wait();
                meet();       // tile t is there, and the other buffer is free
            }
            const float g = g_next;
            const bool some = __ballot(g == -INFINITY) != 0;     // rows that saw nothing anywhere, whatever stands in them
            const uint32_t qrow = lds0 + (uint32_t)(buf * PAD + r * QROW);
            if (t + 1 < end_tile) fetch(t + 1, buf ^ 1, g_next);
            u32x4 b[ST];
#pragma unroll
            for (int k = 0; k < AHEAD && k < ST; ++k) b[k] = lds_read16(qrow + (uint32_t)(((2 * k + h) ^ swz<KC>(r)) * 16));
#pragma unroll
            for (int k = 0; k < ST; ++k) {
                if (k + AHEAD < ST) b[k + AHEAD] = lds_read16(qrow + (uint32_t)(((2 * (k + AHEAD) + h) ^ swz<KC>(r)) * 16));
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) {
                    now[kb] = k == 0 ? Mat<E>::mma(kf[kb][k], b[k], f32x16{}) : Mat<E>::mma(kf[kb][k], b[k], now[kb]);
                    const int part = k * NB + kb, all = NB * 16;
#pragma unroll
                    for (int j = part * all / (ST * NB); j < (part + 1) * all / (ST * NB); ++j) weigh(old, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            const bool none = g == -INFINITY;
            g_old = none ? INFINITY : g * p.lmul;
            // rows are in the order of their tokens: where the first sees all of the wave's keys, so do the
            // others, but for those behind the last and those without a sum, which see nothing
            if (t * 32 + 31 >= nrows || some || visible(p.m, u.s, (int)fdiv((uint32_t)(t * 32), p.m.fG)) < key0 + KW) {
                const int row = t * 32 + r;
                const int lim = row < nrows && !none ? visible(p.m, u.s, (int)fdiv((uint32_t)row, p.m.fG)) - key0 - 4 * h : 0;
                // (a row whose sum is NaN gives NaN to what it sees and nothing to the rest)
                const bool bad = g_old != g_old;
                if (bad) g_old = 0.0f;
#pragma unroll
                for (int j = 0; j < NB * 16; ++j) {
                    const float seen = bad ? NAN : now[j / 16][j % 16];
                    now[j / 16][j % 16] = j / 16 * 32 + 8 * (j % 16 / 4) + j % 4 < lim ? seen : -INFINITY;
                }
            }
        };
        auto finish = [&](const f32x16 (&s)[NB]) {
#pragma unroll
            for (int j = 0; j < NB * 16; ++j) weigh(s, j);
        };
#pragma unroll 1
        for (int t = begin; t < end_tile; t += 2) {
            step(t, 0, s0, s1);
            if (t + 1 == end_tile) break;
            step(t + 1, 1, s1, s0);
        }
        if ((end_tile - begin) % 2 != 0) finish(s0);
        else finish(s1);
        const MassArgs& e = late_args<MassArgs>();
        // totals over the 32 query lanes; lane i of each half takes register i
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x = acc[kb][i];
                x += dcp::dpp_f<0x128>(x);
                x += dcp::dpp_f<0x124>(x);
                x += dcp::dpp_f<0x122>(x);
                x += dcp::dpp_f<0x121>(x);
                total = (lane & 15) == i ? x : total;
            }
            total += __shfl_xor(total, 16, 64);
            if (r < 16) {
                const int place = kb * 32 + 8 * (r / 4) + r % 4 + 4 * h, k = k0 + wave * KW + place;
                if (u.parts > 1) {
                    e.ws[(((int64_t)u.slot * e.m.Hkv + hk) * u.parts + u.part) * KEYS + wave * KW + place] = total;
                } else if (k < u.k1 && (there[kb] >> (place & 31) & 1u) != 0) {
                    *mass_at(e, u.b, hk, k) += total;
                }
            }
        }
    }
}

// Few rows: a wave takes a quarter of the range, tile after tile (see attn_keys).
template <typename E, bool KV8, int DK>
__global__ __launch_bounds__(256, DK > 128 ? 1 : 2) void mass_few(MassArgs p) {
    constexpr int KT = 32, ES = KV8 ? 1 : 2, KROW = DK * ES, KB = KT * KROW, NK = KB / 1024, ST = DK / 16;
    constexpr int GROUP = 8;                   // tiles whose page numbers and sums are held at once
    __shared__ __attribute__((aligned(1024))) char tile[4][2][KB];
    __shared__ int32_t page_of[4][2][GROUP * KT];
    __shared__ uint64_t row_at[4][KT];
    __shared__ float sum_of[4][GROUP * KT];
    int hk, unit;
    heads_together(p.m, hk, unit);
    if (unit >= p.units) return;
    const Share u = find_share<128>(p.m, p.slots, p.share, false, unit);
    if (!u.ok) return;
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, row_tiles = (nrows + 31) / 32;
    const int all_tiles = (u.k1 - u.k0 + KT - 1) / KT, quarter = (all_tiles + 3) / 4, first = min(wave * quarter, all_tiles);
    const int tiles = min(quarter, all_tiles - first), base_key = u.k0 + first * KT;
    if (tiles <= 0) return;                    // (the waves of this kernel never meet)

    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;
    int32_t pages[GROUP * KT / 64];
    auto load_pages = [&](int group) {
#pragma unroll
        for (int k = 0; k < GROUP * KT / 64; ++k) {
            const int key = base_key + group * GROUP * KT + k * 64 + lane;
            pages[k] = key < u.k1 ? table[fdiv((uint32_t)key, p.m.fpage)] : -1;
        }
    };
    auto keep_pages = [&](int group) {
#pragma unroll
        for (int k = 0; k < GROUP * KT / 64; ++k) page_of[wave][group & 1][k * 64 + lane] = pages[k];
    };
    const uint32_t kbuf = lds_addr(&tile[wave][0][0]);
    auto turn = [](int row) { return KV8 ? (KROW >= 128 ? row >> 1 & 7 : row >> 1 & 3) : swz<KROW / 16>(row); };
    auto fetch = [&](int t) {
        if (h == 0) {
            const int page = page_of[wave][t / GROUP & 1][t % GROUP * KT + r];
            const uint32_t key = (uint32_t)(base_key + t * KT + r);
            const uint32_t place = key - fdiv(key, p.m.fpage) * p.m.fpage.d;
            row_at[wave][r] = (uint32_t)page < (uint32_t)p.m.pages
                                  ? (uint64_t)(p.k + (int64_t)page * p.k_P + (int64_t)place * p.k_S + (int64_t)hk * p.k_H)
                                  : (uint64_t)kZeros;
        }
        constexpr int cols = KROW / 16;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int ch = i * 64 + lane, from = ch / cols, c = (ch % cols) ^ turn(from);
            dma16((const char*)at_or_zeros(c * 16 < p.Dk * ES, row_at[wave][from] + (uint64_t)(c * 16)),
                  __builtin_amdgcn_readfirstlane(kbuf + (uint32_t)((t & 1) * KB + i * 1024)));
        }
    };
    // the lane's query row of row tile rt
    u32x4 q[ST];
    int vis = 0;
    float g = 0.0f;
    auto load_rows = [&](int rt) {
        const int row = min(rt * 32 + r, nrows - 1), token = (int)fdiv((uint32_t)row, p.m.fG), head = hk * p.m.G + row - token * p.m.G;
        vis = rt * 32 + r < nrows ? visible(p.m, u.s, token) - base_key : 0;
        const float x = p.lse[(int64_t)(u.s.first + token) * p.l_T + (int64_t)head * p.l_H];
        g = x == -INFINITY ? INFINITY : x * p.lmul;
        const char* from = p.q + (int64_t)(u.s.first + token) * p.q_T + (int64_t)head * p.q_H;
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            const int c = 2 * s + h;
            const u32x4 y = *(const u32x4*)(from + min(c, p.Dk / 8 - 1) * 16);
            q[s] = c * 8 < p.Dk ? y : u32x4{0, 0, 0, 0};
        }
    };
    load_pages(0);
    load_rows(0);
    keep_pages(0);
    fetch(0);
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        if (t % GROUP == 0 && t + GROUP < tiles) {
            load_pages(t / GROUP + 1);
            keep_pages(t / GROUP + 1);
        }
        if (t + 1 < tiles) {
            fetch(t + 1);
            asm volatile("s_waitcnt vmcnt(%0)" :: "n"(NK) : "memory");
        } else {
            dma_wait();
        }
        const uint32_t buf = kbuf + (uint32_t)((t & 1) * KB);
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll 1
        for (int rt = 0; rt < row_tiles; ++rt) {
            if (row_tiles > 1) load_rows(rt);
            f32x16 s;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
            for (int st = 0; st < ST; ++st) {
                u32x4 a;
                if constexpr (KV8)
                    a = widen8<E>(*(const DCPA_LDS u32x2*)(uintptr_t)(buf + (uint32_t)(r * KROW + (st ^ turn(r)) * 16 + h * 8)));
                else
                    a = lds_read16(buf + (uint32_t)(r * KROW + ((2 * st + h) ^ turn(r)) * 16));
                s = Mat<E>::mma(a, q[st], s);
            }
            // (a row that saw nothing anywhere gives nothing, whatever stands in it)
            const int lim = (g == INFINITY ? 0 : vis) - t * KT - 4 * h;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = exp2_fast(__builtin_fmaf(s[i], p.c, -g));
                acc[i] += 8 * (i / 4) + i % 4 < lim ? x : 0.0f;
            }
        }
        // (the next load into this buffer does not wait for these reads)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        // totals over the 32 query lanes; lane i of each half takes register i
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = acc[i];
            x += dcp::dpp_f<0x128>(x);
            x += dcp::dpp_f<0x124>(x);
            x += dcp::dpp_f<0x122>(x);
            x += dcp::dpp_f<0x121>(x);
            mine = (lane & 15) == i ? x : mine;
        }
        mine += __shfl_xor(mine, 16, 64);
        if (r < 16) sum_of[wave][t % GROUP * KT + 8 * (r / 4) + r % 4 + 4 * h] = mine;
        if (t % GROUP == GROUP - 1 || t + 1 == tiles) {
            // the sums of the group's keys join their weights
            const int from = t / GROUP * GROUP * KT;
            float* at[GROUP * KT / 64];
            float old[GROUP * KT / 64];
#pragma unroll
            for (int k = 0; k < GROUP * KT / 64; ++k) {
                const uint32_t key = (uint32_t)(base_key + from + k * 64 + lane);
                const int page = from + k * 64 + lane < tiles * KT ? page_of[wave][t / GROUP & 1][k * 64 + lane] : -1;
                const uint32_t place = key - fdiv(key, p.m.fpage) * p.m.fpage.d;
                at[k] = (uint32_t)page < (uint32_t)p.m.pages
                            ? p.mass + (int64_t)page * p.m_P + (int64_t)place * p.m_S + (int64_t)hk * p.m_H : nullptr;
                old[k] = 0.0f;
                if (at[k] != nullptr) old[k] = *at[k];
            }
#pragma unroll
            for (int k = 0; k < GROUP * KT / 64; ++k)
                if (at[k] != nullptr) *at[k] = old[k] + sum_of[wave][k * 64 + lane];
        }
    }
}

// The parts of split rows, added in order: a thread to a key.
template <int KEYS> __global__ __launch_bounds__(KEYS) void mass_join(MassArgs p) {
    int chunk, parts;
    share_out<KEYS>(p.m, p.slots, p.share, p.ws != nullptr, chunk, parts);
    if (parts == 1) return;
    const int hk = (int)(blockIdx.x % (uint32_t)p.m.Hkv);
    const Share u = find_share<KEYS>(p.m, p.slots, p.share, p.ws != nullptr, (int)(blockIdx.x / (uint32_t)p.m.Hkv) * parts);
    const int key = u.k0 + (int)threadIdx.x;
    if (!u.ok || key >= u.k1) return;
    float* m = mass_at(p, u.b, hk, key);
    if (m == nullptr) return;
    const float* w = p.ws + ((int64_t)u.slot * p.m.Hkv + hk) * parts * KEYS + threadIdx.x;
    float sum = 0.0f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) sum += w[(int64_t)i * KEYS];
    *m += sum;
}

// Keys of a workgroup's step.
int keys_of(bool few, int Dk) { return few || Dk > 128 ? 128 : 256; }

}  // namespace

MassPlan plan_mass(const Batch& m, int Dk, bool pieces) {
    MassPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.few = pieces && Dk <= 256 && rows <= (int64_t)32 * m.B;
    // two workgroups to a CU (four with few rows, whose ranges are then shorter); every sequence
    // needs one at least
    const int64_t want = pl.few ? 1024 : 512;
    const int64_t seqs = m.T < m.B ? m.T : m.B;
    pl.slots = pl.share = (int32_t)((want + m.Hkv - 1) / m.Hkv);
    // rows are split only where sequences are few: parts > 1 only while steps * parts <= slots
    pl.ws_bytes = pl.few || 2 * seqs > pl.slots ? 0 : (int64_t)pl.slots * m.Hkv * keys_of(pl.few, Dk) * 4;
    fill_slots((int32_t)seqs, pl.slots, pl.share);
    // a sequence without keys or with one step takes a unit all the same
    pl.units = pl.slots;
    if (seqs * m.Hkv >= 4 * want) {
        // more sequences than that: each is one unit, whole
        pl.slots = 0;
        pl.units = (int32_t)seqs;
    }
    return pl;
}

namespace {
template <typename E, bool KV8> hipError_t run(const MassArgs& a, bool few, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.units * a.m.Hkv)), block(256);
    if (few) {
        const dim3 near((uint32_t)((int64_t)(a.units + 7) / 8 * 8 * a.m.Hkv));      // (see heads_together())
        return a.Dk <= 64    ? launch(mass_few<E, KV8, 64>, near, block, stream, a)
               : a.Dk <= 128 ? launch(mass_few<E, KV8, 128>, near, block, stream, a)
                             : launch(mass_few<E, KV8, 256>, near, block, stream, a);
    }
    const hipError_t e = a.Dk <= 64    ? launch(mass_rows<E, KV8, 64, 64>, grid, block, stream, a)
                         : a.Dk <= 128 ? launch(mass_rows<E, KV8, 128, 64>, grid, block, stream, a)
                         : a.Dk <= 256 ? launch(mass_rows<E, KV8, 256, 32>, grid, block, stream, a)
                                       : launch(mass_rows<E, KV8, 576, 32>, grid, block, stream, a);
    if (e != hipSuccess || a.ws == nullptr) return e;
    return keys_of(false, a.Dk) == 128 ? launch(mass_join<128>, grid, dim3(128), stream, a)
                                       : launch(mass_join<256>, grid, dim3(256), stream, a);
}
}  // namespace

hipError_t launch_mass(const MassArgs& a, bool few, bool bf16, bool kv8, hipStream_t stream) {
    if (bf16) return kv8 ? run<BF16T, true>(a, few, stream) : run<BF16T, false>(a, few, stream);
    return kv8 ? run<F16T, true>(a, few, stream) : run<F16T, false>(a, few, stream);
}

}  // namespace dcpa
