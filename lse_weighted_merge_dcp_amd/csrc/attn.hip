// attn.hip -- attention of new tokens over a rank's paged cache, with the
// partial output and log-sum-exp that the merge takes.
//
// attn_rows: 128 query rows of a key head to a workgroup (attn_rows.hpp).
// attn_keys: up to 32 rows (decode of grouped heads); each wave takes its own
// tiles of keys, and the four are joined in LDS at the end.
// attn_join: joins the key ranges of one row tile that went to different
// workgroups.
#include "attn_rows.hpp"

namespace dcpa {

namespace {

template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, bool WIDE>
__global__ __launch_bounds__(256, DK > 192 ? 1 : 2) void attn_rows(AttnArgs p) {
    rows_of<E, KV8, EXACT, DK, DV, KT, WIDE>(p);
}

// ---------------------------------------------------------------------------
// attn_keys
//
// Bound by the cache's bytes: 32 keys of 128 columns are 16 KB and 512 clocks of
// matrix instructions.  A wave keeps one tile of keys and one of values in LDS and
// asks for the next keys as soon as its products have read the present ones,
// for the next values likewise, so one of the two is always on its way; the
// other waves of the CU (two workgroups) fill the gaps.  8-bit rows lie in LDS
// as in the cache and are widened as fragments: no two waves read the same.  The
// matrix instructions have time to spare, so the weights take two products, their
// remainders the second (see weights()).  32 contexts of up to 32768 keys, 64 / 8
// heads: 369 us, 5.1 TB/s, with one product too; 64 8-bit ones of up to 8192: 72.9 us,
// 3.6 TB/s, 71.5 with one (149 us when widened on the way into LDS).
// ---------------------------------------------------------------------------
template <typename E, bool KV8, int DK, int DV>
__global__ __launch_bounds__(256, DK > 128 ? 1 : 2) void attn_keys(AttnArgs p) {
    constexpr int KT = 32, ES = KV8 ? 1 : 2, KROW = DK * ES, VROW = DV * ES;
    constexpr int KB = KT * KROW, VB = KT * VROW, NK = KB / 1024, NV = VB / 1024;
    constexpr int GROUP = 8;                   // tiles whose page numbers are held at once, twice
    __shared__ __attribute__((aligned(1024))) char tile[4][KB + VB];
    __shared__ int32_t page_of[4][2][GROUP * KT];
    __shared__ uint64_t row_at[4][2][KT];      // where the next tile's key and value rows lie
    __shared__ float part_mc[4][32], part_l[4][32];
    __shared__ int part_odd[4];

    int hk, unit;
    heads_together(p.m, hk, unit);
    if (unit >= p.units) return;
    const Unit u = find_unit<128>(p.m, 32, p.slots, p.share, unit);
    if (!u.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, row0 = u.tile * 32;
    const int last_row = min(row0 + 32, nrows) - 1;
    const int kend = visible(p.m, u.s, (int)fdiv((uint32_t)last_row, p.m.fG));
    const int k0 = u.split * u.chunk, k1 = (int)min((int64_t)kend, (int64_t)k0 + u.chunk);
    if (u.split > 0 && k0 >= k1) return;
    // the wave's tiles are its own quarter of the range, one after the other
    const int all_tiles = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;
    const int quarter = (all_tiles + 3) / 4, first = min(wave * quarter, all_tiles);
    const int tiles = min(quarter, all_tiles - first), base_key = k0 + first * KT;

    Rows<DK, DV, 1> w;
    const int row = min(row0 + r, last_row), token = (int)fdiv((uint32_t)row, p.m.fG);
    const int vis = visible(p.m, u.s, token) - base_key;
    const int vmin = __builtin_amdgcn_readlane(vis, 0);
    load_query<DK>(w.q[0], p.q + (int64_t)(u.s.first + token) * p.q_T +
                               (int64_t)(hk * p.m.G + row - token * p.m.G) * p.q_H, p.Dk, h);
    clear_rows(w);
    bool odd = false;

    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;
    auto load_pages = [&](int group, int32_t (&x)[GROUP * KT / 64]) {
#pragma unroll
        for (int k = 0; k < GROUP * KT / 64; ++k) {
            const int key = base_key + group * GROUP * KT + k * 64 + lane;
            x[k] = key < k1 ? table[fdiv((uint32_t)key, p.m.fpage)] : -1;
        }
    };
    auto keep_pages = [&](int group, const int32_t (&x)[GROUP * KT / 64]) {
#pragma unroll
        for (int k = 0; k < GROUP * KT / 64; ++k) page_of[wave][group & 1][k * 64 + lane] = x[k];
    };
    // lanes 0 .. 31 place the key rows of tile t, the others its value rows
    const char* my_base = h == 0 ? p.k + (int64_t)hk * p.k_H : p.v + (int64_t)hk * p.v_H;
    const int64_t my_P = h == 0 ? p.k_P : p.v_P, my_S = h == 0 ? p.k_S : p.v_S;
    auto place_rows = [&](int t) {
        const int page = page_of[wave][t / GROUP & 1][t % GROUP * KT + r];
        const uint32_t key = (uint32_t)(base_key + t * KT + r);
        const uint32_t place = key - fdiv(key, p.m.fpage) * p.m.fpage.d;
        row_at[wave][h][r] = page_row(page, p.m, my_base, my_P, my_S, 0, place);
        return (uint32_t)__ballot(h == 0 && (uint32_t)page < (uint32_t)p.m.pages);
    };
    const uint32_t kbuf = lds_addr(&tile[wave][0]), vbuf = kbuf + KB;
    // a row's chunk c of 16 bytes lies at c ^ turn(row)
    auto turn = [](bool val, int row) {
        if constexpr (KV8) return DK >= 128 ? row >> 1 & 7 : row >> 1 & 3;
        else return val ? swz_v<VROW / 16>(row) : swz<KROW / 16>(row);
    };
    auto fetch = [&](bool val, uint32_t buf) {
        constexpr int NMAX = NK > NV ? NK : NV;
        const int cols = (val ? VROW : KROW) / 16, n = val ? NV : NK, width = (val ? p.Dv : p.Dk) * ES;
#pragma unroll
        for (int i = 0; i < NMAX; ++i) {
            if (i >= n) break;
            const int ch = i * 64 + lane, from = ch / cols, c = (ch % cols) ^ turn(val, from);
            const uint64_t a = at_or_zeros(c * 16 < width, row_at[wave][val][from] + (uint64_t)(c * 16));
            dma16((const char*)a, __builtin_amdgcn_readfirstlane(buf + (uint32_t)(i * 1024)));
        }
    };

    int32_t pages[GROUP * KT / 64];
    uint32_t there = 0;
    if (tiles > 0) {
        load_pages(0, pages);
        keep_pages(0, pages);
        there = place_rows(0);
        fetch(false, kbuf);
        fetch(true, vbuf);
    }
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        // keys of t are there; its values may still be on their way
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"(NV) : "memory");
        f32x16 s[1][1];
        uint32_t pr[1][1][8], rest[1][1][8];
        if constexpr (KV8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[0][0][i] = 0.0f;
#pragma unroll
            for (int st = 0; st < DK / 16; ++st) {
                const u32x2 x = *(const DCPA_LDS u32x2*)(uintptr_t)(kbuf + (uint32_t)(r * KROW + ((st ^ turn(false, r)) * 16) + h * 8));
                s[0][0] = Mat<E>::mma(widen8<E>(x), w.q[0][st], s[0][0]);
            }
        } else {
            scores<E, DK, 1, KT, KROW>(s, w.q, kbuf);
        }
        const uint32_t now = there;
        const bool next = t + 1 < tiles;
        if (next) {
            // (loads into LDS do not wait for this wave's reads)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            there = place_rows(t + 1);
            fetch(false, kbuf);
        }
        const int lim[1] = {vis - t * KT};
        const bool full = now == 0xffffffffu && vmin >= (t + 1) * KT;
        weights<E>(w, s, pr, rest, now, lim, full, p.c);
        // values of t
        if (next) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(NK) : "memory");
        else dma_wait();
        if constexpr (KV8) {
            const int g = (lane >> 4) & 1, li = lane & 15, j = li >> 1, key = 4 * h + (j & 3) + 8 * (j >> 2);
            outputs<E, DK, DV, 1, KT>(w, pr, rest, [&](int cb, int ks) {
                const uint32_t a = vbuf + (uint32_t)((ks * 16 + key) * VROW + ((2 * cb + g) ^ turn(true, ks * 16 + key)) * 16 + (li & 1) * 8);
                return widen8<E>(lds_read_tr8(a));
            });
        } else {
            ValuePlace<VROW> vp;
            vp.set(vbuf, lane);
            outputs<E, DK, DV, 1, KT>(w, pr, rest, [&](int cb, int ks) { return vp.read(cb, ks); });
        }
        if (!full) odd |= odd_values<E, KV8>(vbuf, VB);
        if (t % GROUP == 0 && t + GROUP < tiles) {
            load_pages(t / GROUP + 1, pages);
            keep_pages(t / GROUP + 1, pages);
        }
        if (next) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            fetch(true, vbuf);
        }
    }

    // the four waves' sums and outputs on one scale, through LDS
    const float l = half_sum(w.l[0]);
    if (h == 0) {
        part_mc[wave][r] = w.mc[0];
        part_l[wave][r] = l;
    }
    if (lane == 0) part_odd[wave] = odd;
    meet();
    if ((part_odd[0] | part_odd[1] | part_odd[2] | part_odd[3]) != 0) {
        slow_rows<E, KV8, DK, DV>(late_args<AttnArgs>(), u, hk, unit, 32, row0, row0 + wave * 8, min(row0 + wave * 8 + 8, nrows), k0, k1);
        return;
    }
    float mc = kNoMax;
#pragma unroll
    for (int k = 0; k < 4; ++k) mc = fmaxf(mc, part_mc[k][r]);
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) total += part_l[k][r] * exp2_fast(part_mc[k][r] - mc);
    // (mc +infinity, a row that met a score of +infinity: its sums are NaN already)
    const float f = w.mc[0] == mc ? 1.0f : exp2_fast(w.mc[0] - mc);
    // each wave adds up its quarter of the output registers
    constexpr int PART = DV / 32 * 16 / 4;
    float* all = (float*)&tile[0][0];
    constexpr int ROUNDS = (4 * DV / 32 * 16 * 64 * 4 + (int)sizeof(tile) - 1) / (int)sizeof(tile);
    constexpr int PER = PART / ROUNDS;         // registers of each quarter that one round exchanges
    static_assert(PART % ROUNDS == 0, "rounds of equal size");
    float mine[PART];
#pragma unroll
    for (int round = 0; round < ROUNDS; ++round) {
        meet();
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = k * PART + round * PER + i;
                all[((k * 4 + wave) * PER + i) * 64 + lane] = w.o[0][at / 16][at % 16] * f;
            }
        meet();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            mine[round * PER + i] = (all[((wave * 4 + 0) * PER + i) * 64 + lane] + all[((wave * 4 + 1) * PER + i) * 64 + lane]) +
                                    (all[((wave * 4 + 2) * PER + i) * 64 + lane] + all[((wave * 4 + 3) * PER + i) * 64 + lane]);
    }
    const int my_row = row0 + r;
    if (my_row >= nrows) return;
    float scale, lse2;
    finish(total, mc, p.vs, scale, lse2);
    const int head = hk * p.m.G + row - token * p.m.G;
    const int64_t at = ((int64_t)hk * p.units + unit) * 32 + r;
    const bool split = u.splits > 1;
    if (h == 0 && wave == 0) {
        if (split) p.ws_l[at] = lse2;
        else if (p.lse != nullptr) p.lse[(int64_t)(u.s.first + token) * p.l_T + (int64_t)head * p.l_H] = lse2 * p.lmul;
    }
    char* o = p.out + (int64_t)(u.s.first + token) * p.o_T + (int64_t)head * p.o_H;
#pragma unroll
    for (int i = 0; i < PART; i += 4) {
        const int reg = wave * PART + i, col = reg / 16 * 32 + (reg % 16) * 2 + h * 4;
        if (col >= p.Dv) continue;
        f32x4 x;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = total == 0.0f ? 0.0f : mine[i + k] * scale;
        if (split) *(f32x4*)(p.ws_o + at * p.Dv + col) = x;
        else store4<E>(o + col * 2, x[0], x[1], x[2], x[3]);
    }
}

// ---------------------------------------------------------------------------
// attn_join: the rows of sequences whose keys were split; each lane holds four
// columns (eight where the rows are wide).  Few rows have many parts: the four
// waves of a workgroup share a row's (TOGETHER).  Many rows have few: a wave goes
// from row to row, and works out the lengths once.  Bound by latency: eight parts
// under way at once (7 rows of 155 parts: 9 us, 54 us one part after the other by
// one wave; 2048 rows by a wave each 8 us, by a workgroup each 14 us).  Where the
// lengths turn out even nothing was split, and nothing is joined.
// ---------------------------------------------------------------------------
template <typename E, int STEP, int NC, bool TOGETHER>
__global__ __launch_bounds__(256) void attn_join(AttnArgs p) {
    constexpr int FLY = NC == 1 ? 8 : 4;       // parts under way at once
    __shared__ f32x4 share[TOGETHER ? 4 : 1][NC][64];
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    int longest;
    const int chunk = key_chunk<STEP>(p.m, p.rows, p.slots, p.share, longest);
    if (__ballot(longest > chunk) == 0) return;       // nothing was split
    // lengths and units of sequences b0 .. b0 + 63, a lane to each
    struct Line {
        Seq s;
        int splits, incl;
    };
    auto line_at = [&](int b0, int base) {
        Line x{};
        int tiles = 0;
        if (b0 + lane < p.m.B) {
            x.s = load_seq(p.m, b0 + lane);
            tiles = (x.s.n * p.m.G + p.rows - 1) / p.rows;
        }
        x.splits = max(1, (x.s.kv + chunk - 1) / chunk);
        x.incl = base + scan_incl(tiles * x.splits);
        return x;
    };
    const Line start = line_at(0, 0);
    const int64_t all = (int64_t)p.m.T * p.m.G * p.m.Hkv;
    const int64_t stride = TOGETHER ? gridDim.x : (int64_t)gridDim.x * 4;
#pragma unroll 1
    for (int64_t id = TOGETHER ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave; id < all; id += stride) {
        const uint32_t at_row = fdiv((uint32_t)id, p.m.fHkv);
        const int hk = (int)((uint32_t)id - at_row * p.m.fHkv.d), t = (int)fdiv(at_row, p.m.fG), head = (int)at_row - t * p.m.G;
        Line x = start;
        uint64_t found = 0;
        for (int b0 = 0;; b0 += 64, x = line_at(b0, __builtin_amdgcn_readlane(x.incl, 63))) {
            found = __ballot(t >= x.s.first && t < x.s.first + x.s.n);
            if (found != 0 || b0 + 64 >= p.m.B) break;
        }
        if (found == 0) continue;
        const int at = __builtin_ctzll(found);
        const Seq s = seq_of(x.s, at);
        const int ns = __builtin_amdgcn_readlane(x.splits, at);
        if (ns == 1) continue;                // written whole
        const int row = (t - s.first) * p.m.G + head, tile = row / p.rows, in_tile = row - tile * p.rows;
        // (a sequence's last tile comes first)
        const int slot = __builtin_amdgcn_readlane(x.incl, at) - (tile + 1) * ns;
        if (slot < 0) continue;
        // the ranges that the tile's last row has keys in
        const int last = min((tile + 1) * p.rows, s.n * p.m.G) - 1;
        const int kend = visible(p.m, s, (int)fdiv((uint32_t)last, p.m.fG));
        const int parts = min(max(1, (kend + chunk - 1) / chunk), p.units - slot);
        const int64_t first = ((int64_t)hk * p.units + slot) * p.rows + in_tile;
        float top = -INFINITY;
        bool bad = false;
        for (int k = lane; k < parts; k += 64) {
            const float y = p.ws_l[first + (int64_t)k * p.rows];
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
        for (int k0 = 0; k0 < parts; k0 += 64) {
            // a lane to a part's weight
            const int here = min(64, parts - k0);
            const float f = lane < here ? exp2_fast(p.ws_l[first + (int64_t)(k0 + lane) * p.rows] - ref) : 0.0f;
            sum += f;
#pragma unroll 1
            for (int k = TOGETHER ? wave * FLY : 0; k < here; k += TOGETHER ? 4 * FLY : FLY) {
                f32x4 y[FLY][NC];
#pragma unroll
                for (int i = 0; i < FLY; ++i)
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        const int col = min(j * 256 + lane * 4, p.Dv - 4);
                        y[i][j] = *(const f32x4*)(p.ws_o + (first + (int64_t)(k0 + min(k + i, here - 1)) * p.rows) * p.Dv + col);
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

}  // namespace

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
AttnPlan plan_attn(const Batch& m, int Dk, int Dv, bool pieces) {
    AttnPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.latent = Dk > 256 || Dv > 256;
    // few rows a sequence: 32-row tiles whose waves share out the keys
    pl.by_keys = !pl.latent && pieces && rows <= (int64_t)32 * m.B;
    pl.rows = pl.by_keys ? 32 : 128;
    // row tiles, at most: a tile holds rows of one sequence
    const int64_t most = rows / pl.rows + m.B, each = (int64_t)m.T * ((m.G + pl.rows - 1) / pl.rows);
    pl.tiles = (int32_t)(most < each ? most : each);
    // Workgroups that run at once: one latent workgroup to a CU, two of the others.  Fewer row
    // tiles than that: the keys are split so that the units fill the chip once; decode of ragged
    // batches (few rows, a few tokens to a sequence of latent ones) up to four times over (see
    // fill_slots()).
    const int64_t busy = (int64_t)pl.tiles * m.Hkv;
    const int64_t chip = pl.latent ? 256 : pl.by_keys ? 1024 : 512;
    pl.slots = pl.share = (int32_t)((chip + m.Hkv - 1) / m.Hkv);
    const bool decode = pl.by_keys || (pl.latent && m.T <= (int64_t)8 * m.B);
    if (decode) fill_slots(pl.tiles, pl.slots, pl.share);
    if (busy >= (decode ? 4 * chip : chip)) pl.slots = 0;
    pl.units = pl.slots > pl.tiles ? pl.slots : pl.tiles;
    pl.ws_bytes = pl.slots == 0 ? 0 : (int64_t)pl.units * m.Hkv * pl.rows * (Dv + 1) * 4;
    return pl;
}

namespace {

template <typename E, int STEP>
hipError_t run_join(const AttnArgs& a, hipStream_t stream) {
    // a workgroup to a row up to what the chip holds at once, then a wave, and no more waves than that
    const int64_t rows = (int64_t)a.m.T * a.m.G * a.m.Hkv;
    const dim3 block(256);
    if (rows <= 1024) {
        const dim3 grid((uint32_t)rows);
        return a.Dv <= 256 ? launch(attn_join<E, STEP, 1, true>, grid, block, stream, a)
                           : launch(attn_join<E, STEP, 2, true>, grid, block, stream, a);
    }
    const dim3 grid((uint32_t)(rows < 8192 ? (rows + 3) / 4 : 2048));
    return a.Dv <= 256 ? launch(attn_join<E, STEP, 1, false>, grid, block, stream, a)
                       : launch(attn_join<E, STEP, 2, false>, grid, block, stream, a);
}

template <typename E, bool KV8, bool WIDE>
hipError_t run_rows(const AttnArgs& a, const AttnPlan& pl, dim3 grid, dim3 block, hipStream_t stream) {
    // (whole rows need no test of columns)
    const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
    hipError_t e;
    if (d <= 64)
        e = a.Dk == 64 && a.Dv == 64 ? launch(attn_rows<E, KV8, true, 64, 64, 64, WIDE>, grid, block, stream, a)
                                     : launch(attn_rows<E, KV8, false, 64, 64, 64, WIDE>, grid, block, stream, a);
    else if (d <= 128)
        e = a.Dk == 128 && a.Dv == 128 ? launch(attn_rows<E, KV8, true, 128, 128, 64, WIDE>, grid, block, stream, a)
                                       : launch(attn_rows<E, KV8, false, 128, 128, 64, WIDE>, grid, block, stream, a);
    else {
        e = a.Dk <= 192 && a.Dv <= 128   ? launch(attn_rows<E, KV8, false, 192, 128, 32, WIDE>, grid, block, stream, a)
            : a.Dk <= 192 && a.Dv <= 192 ? launch(attn_rows<E, KV8, false, 192, 192, 32, WIDE>, grid, block, stream, a)
                                         : launch(attn_rows<E, KV8, false, 256, 256, 32, WIDE>, grid, block, stream, a);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 32>(a, stream);
    }
    if (e != hipSuccess || pl.slots == 0) return e;
    return run_join<E, 64>(a, stream);
}

template <typename E, bool KV8>
hipError_t run(const AttnArgs& a, const AttnPlan& pl, bool wide, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)pl.units * a.m.Hkv)), block(256);
    hipError_t e;
    if (pl.by_keys) {
        const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
        const dim3 near((uint32_t)((int64_t)(pl.units + 7) / 8 * 8 * a.m.Hkv));      // (see heads_together())
        e = d <= 64    ? launch(attn_keys<E, KV8, 64, 64>, near, block, stream, a)
            : d <= 128 ? launch(attn_keys<E, KV8, 128, 128>, near, block, stream, a)
                       : launch(attn_keys<E, KV8, 256, 256>, near, block, stream, a);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 128>(a, stream);
    }
    if (pl.latent) {
        e = launch_latent(a, grid, std::is_same_v<E, BF16T>, KV8, wide, stream);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 32>(a, stream);
    }
    return wide ? run_rows<E, KV8, true>(a, pl, grid, block, stream) : run_rows<E, KV8, false>(a, pl, grid, block, stream);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& arg, const AttnPlan& pl, bool bf16, bool kv8, bool wide, hipStream_t stream) {
    AttnArgs a = arg;
    if (!pl.latent && a.v == nullptr) {        // narrow rows: the values are read as columns of their own
        a.v = a.k;
        a.v_P = a.k_P; a.v_S = a.k_S; a.v_H = a.k_H;
    }
    if (bf16) return kv8 ? run<BF16T, true>(a, pl, wide, stream) : run<BF16T, false>(a, pl, wide, stream);
    return kv8 ? run<F16T, true>(a, pl, wide, stream) : run<F16T, false>(a, pl, wide, stream);
}

}  // namespace dcpa
