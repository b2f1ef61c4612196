// attn_keys.hpp -- attention of up to 32 rows (decode of grouped heads): each wave
// takes its own tiles of keys, and the four are joined in LDS at the end.  Shared
// by attn.hip and attn_prefix.hip, as attn_rows.hpp.
#pragma once
#include "attn_common.hpp"

namespace dcpa {

// ---------------------------------------------------------------------------
// keys_of
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
template <bool KV8, int DK, int DV> struct KeysLds {
    static constexpr int KT = 32, GROUP = 8;   // GROUP: tiles whose page numbers are held at once, twice
    __attribute__((aligned(1024))) char tile[4][KT * (DK + DV) * (KV8 ? 1 : 2)];
    int32_t page_of[4][2][GROUP * KT];
    uint64_t row_at[4][2][KT];                 // where the next tile's key and value rows lie
    float part_mc[4][32], part_l[4][32];
    int part_odd[4];
};

template <typename E, bool KV8, int DK, int DV, typename A, typename U>
__device__ __forceinline__ void keys_of(const A& p, KeysLds<KV8, DK, DV>& lds, const U& u, int hk, int unit) {
    constexpr int KT = 32, ES = KV8 ? 1 : 2, KROW = DK * ES, VROW = DV * ES;
    constexpr int KB = KT * KROW, VB = KT * VROW, NK = KB / 1024, NV = VB / 1024;
    constexpr int GROUP = KeysLds<KV8, DK, DV>::GROUP;
    auto& tile = lds.tile;
    auto& page_of = lds.page_of;
    auto& row_at = lds.row_at;
    auto& part_mc = lds.part_mc;
    auto& part_l = lds.part_l;
    auto& part_odd = lds.part_odd;
    if (!u.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, row0 = u.tile * 32;
    const int last_row = min(row0 + 32, nrows) - 1;
    const int kend = last_key(p, u, last_row);
    const int k0 = first_key(u) + u.split * u.chunk, k1 = (int)min((int64_t)kend, (int64_t)k0 + u.chunk);
    if (u.split > 0 && k0 >= k1) return;
    // the wave's tiles are its own quarter of the range, one after the other
    const int all_tiles = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;
    const int quarter = (all_tiles + 3) / 4, first = min(wave * quarter, all_tiles);
    const int tiles = min(quarter, all_tiles - first), base_key = k0 + first * KT;

    Rows<DK, DV, 1> w;
    const int row = min(row0 + r, last_row), token = (int)fdiv((uint32_t)row, p.m.fG);
    const int vis = sees(p, u, token) - base_key;
    const int vmin = least_seen(u, vis);
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
        slow_rows<E, KV8, DK, DV>(late_args<A>(), u, hk, unit, p.rows, row0, row0 + wave * 8, min(row0 + wave * 8 + 8, nrows), k0, k1);
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
    const int64_t at = ((int64_t)hk * p.units + unit) * p.rows + r;
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

}  // namespace dcpa
