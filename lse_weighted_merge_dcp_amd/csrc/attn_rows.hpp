// attn_rows.hpp -- attention of many rows: 128 query rows of a key head to a
// workgroup, 32 to a wave, tiles of keys and values in LDS shared by the four
// waves.  Shared by the batch of single sequences (attn.hip) and the one whose
// sequences share first keys (attn_prefix.hip), which find their units each in
// its own way: unit_of(), first_key(), last_key() and sees() go by the arguments.
#pragma once
#include "attn_common.hpp"

namespace dcpa {

// ---------------------------------------------------------------------------
// rows_of
//
// Bound by the matrix instructions (32 clocks for 64 scores of 128 columns and
// their share of the outputs), with 20 clocks of vector work for the same
// scores beside them.  So the next tile's scores are computed while this one's
// powers are taken, and its maximum while this one's values are multiplied: a
// tile's keys are fetched one turn before its values.  (One after the other, two
// waves to a SIMD filled each other's gaps by half: 4 ragged sequences of up to
// 2048 tokens over 16384, 32 / 8 heads of 128, took 533 us; now 477 us, 0.87
// PFLOP/s.)  Wider rows take 32 keys to a tile, and where the registers hold 192
// columns two workgroups to a CU still fit: 1511 tokens of 192 / 128 columns take
// 60 us, 133 us in tiles of 256.
// The weights are rounded to the payload type for the product with the values,
// whose error is then that of the output's own rounding once more.  WIDE: what the
// rounding left takes a second product, half as many matrix instructions again:
// the chunk above takes 631 us with it, 473 without.
// ---------------------------------------------------------------------------
template <int DK, int DV, int KT> struct RowsLds {
    __attribute__((aligned(1024))) char ktile[2][KT * DK * 2], vtile[2][KT * DV * 2];
    uint64_t krow_at[4][KT], vrow_at[4][KT];     // of tile t at t % 4
    uint64_t there_at[4];
};
// Keys and values in two parts, the second what the rounding of the first left (DR columns of a key have one).
template <int DK, int DV, int KT, int DR> struct PairLds : RowsLds<DK, DV, KT> {
    __attribute__((aligned(1024))) char krest[2][KT * DR * 2], vrest[2][KT * DV * 2];
    uint64_t krest_at[4][KT], vrest_at[4][KT];
};

template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, bool WIDE, int DR = 0, typename A, typename L>
__device__ __forceinline__ void rows_of(const A& p, L& lds) {
    constexpr bool PAIRS = DR > 0;
    constexpr int RC = DR / 8, SR = DR / 16, RROW = DR * 2, RB = KT * RROW, NR = KT * RC / 256;
    static_assert(!(PAIRS && KV8) && KT * RC % 256 == 0 && DR <= DK, "parts of 16 bits");
    constexpr int R = 128, KC = DK / 8, VC = DV / 8, NB = KT / 32, ST = DK / 16, CB = DV / 32, KS = KT / 16;
    constexpr int KROW = KC * 16, VROW = VC * 16;
    constexpr int KB = KT * KROW, VB = KT * VROW;
    constexpr int NK = KT * KC / 256, NV = KT * VC / 256;   // 16-byte chunks of a thread
    constexpr int AHEAD = 2;                                // fragments read ahead of their products
    static_assert(KT * KC % 256 == 0 && KT * VC % 256 == 0, "a tile is whole rounds of the workgroup");
    auto& krow_at = lds.krow_at;
    auto& vrow_at = lds.vrow_at;
    auto& there_at = lds.there_at;

    const int hk = (int)(blockIdx.x % (uint32_t)p.m.Hkv), unit = (int)(blockIdx.x / (uint32_t)p.m.Hkv);
    const auto u = unit_of<KT>(p, R, unit);
    if (!u.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, row0 = u.tile * R, wave_row = wave * 32;
    const int Dk = EXACT ? DK : p.Dk, Dv = EXACT ? DV : p.Dv;

    // the key range of this unit: what the tile's last row sees, cut to the split
    const int last_row = min(row0 + R, nrows) - 1;
    const int kend = last_key(p, u, last_row);
    const int k0 = first_key(u) + u.split * u.chunk, k1 = (int)min((int64_t)kend, (int64_t)k0 + u.chunk);
    if (u.split > 0 && k0 >= k1) return;      // (the join counts the ranges by itself)
    const int tiles = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;

    Rows<DK, DV, 1> w;
    int vis;
    {
        const int row = min(row0 + wave_row + r, last_row), token = (int)fdiv((uint32_t)row, p.m.fG);
        vis = sees(p, u, token) - k0;
        load_query<DK>(w.q[0], p.q + (int64_t)(u.s.first + token) * p.q_T +
                                   (int64_t)(hk * p.m.G + row - token * p.m.G) * p.q_H, Dk, h);
    }
    const int vmin = least_seen(u, vis);
    // (waves behind the last row only help to fetch)
    const int mine = row0 + wave_row < nrows ? max(0, min(tiles, (most_seen(u, vis) + KT - 1) / KT)) : 0;
    clear_rows(w);
    bool odd = false;

    const int64_t koff = (int64_t)hk * p.k_H, voff = (int64_t)hk * p.v_H;
    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;
    // where the rows of tile t lie, by the first wave
    auto page_of = [&](int t) {
        const int key = k0 + t * KT + lane;
        return lane < KT && key < k1 ? table[fdiv((uint32_t)key, p.m.fpage)] : -1;
    };
    auto place_rows = [&](int t, int page) {
        const uint32_t key = (uint32_t)(k0 + t * KT + lane);
        const uint32_t place = key - fdiv(key, p.m.fpage) * p.m.fpage.d;
        const uint64_t ka = page_row(page, p.m, p.k, p.k_P, p.k_S, koff, place);
        if (lane < KT) {
            krow_at[t & 3][lane] = ka;
            vrow_at[t & 3][lane] = page_row(page, p.m, p.v, p.v_P, p.v_S, voff, place);
            if constexpr (PAIRS) {
                lds.krest_at[t & 3][lane] = page_row(page, p.m, p.kr, p.kr_P, p.kr_S, (int64_t)hk * p.kr_H, place);
                lds.vrest_at[t & 3][lane] = page_row(page, p.m, p.vr, p.vr_P, p.vr_S, (int64_t)hk * p.vr_H, place);
            }
        }
        const uint64_t bits = __ballot(lane < KT && (uint32_t)page < (uint32_t)p.m.pages);
        if (lane == 0) there_at[t & 3] = bits;
    };
    const uint32_t kbuf = lds_addr(&lds.ktile[0][0]), vbuf = lds_addr(&lds.vtile[0][0]);
    u32x2 reg8[KV8 ? NK + NV : 1];
    // the keys or values of tile t: straight into LDS, or into registers to be widened
    auto fetch = [&](auto val, int t) {
        constexpr bool V = decltype(val)::value;
        constexpr int cols = V ? VC : KC;
#pragma unroll
        for (int i = 0; i < (V ? NV : NK); ++i) {
            const int ch = i * 256 + tid, row = ch / cols, c = (ch % cols) ^ (V ? swz_v<VC>(row) : swz<KC>(row));
            const uint64_t base = V ? vrow_at[t & 3][row] : krow_at[t & 3][row];
            uint64_t at = base + (uint64_t)(c * (KV8 ? 8 : 16));
            if constexpr (!EXACT) at = at_or_zeros(c * 8 < (V ? Dv : Dk), at);
            if constexpr (KV8)
                reg8[(V ? NK : 0) + i] = *(const u32x2*)at;
            else
                dma16((const char*)at, (V ? vbuf + (uint32_t)((t & 1) * VB) : kbuf + (uint32_t)((t & 1) * KB)) +
                                           (uint32_t)((i * 256 + wave * 64) * 16));
        }
        if constexpr (PAIRS) {
            constexpr int rcols = V ? VC : RC;
#pragma unroll
            for (int i = 0; i < (V ? NV : NR); ++i) {
                const int ch = i * 256 + tid, row = ch / rcols, c = (ch % rcols) ^ (V ? swz_v<VC>(row) : swz<RC>(row));
                uint64_t at = (V ? lds.vrest_at[t & 3][row] : lds.krest_at[t & 3][row]) + (uint64_t)(c * 16);
                if constexpr (!EXACT) at = at_or_zeros(c * 8 < (V ? Dv : p.Dr), at);
                dma16((const char*)at, (V ? lds_addr(&lds.vrest[0][0]) + (uint32_t)((t & 1) * VB)
                                          : lds_addr(&lds.krest[0][0]) + (uint32_t)((t & 1) * RB)) +
                                           (uint32_t)((i * 256 + wave * 64) * 16));
            }
        }
    };
    auto widen = [&](auto val, int t) {
        constexpr bool V = decltype(val)::value;
        if constexpr (KV8)
#pragma unroll
            for (int i = 0; i < (V ? NV : NK); ++i)
                lds_write16((V ? vbuf + (uint32_t)((t & 1) * VB) : kbuf + (uint32_t)((t & 1) * KB)) + (uint32_t)((i * 256 + tid) * 16),
                            widen8<E>(reg8[(V ? NK : 0) + i]));
    };
    constexpr std::true_type values{};
    constexpr std::false_type keys{};

    // scores of tile t; `beside(n)`: what is done beside matrix instruction n of NB (ST + SR)
    auto multiply_keys = [&](int t, f32x16 (&s)[1][NB], auto beside) {
        constexpr int N = ST * NB, ALL = N + SR * NB;
        KeyPlace<KROW> place;
        place.set(kbuf + (uint32_t)((t & 1) * KB), r, h);
        KeyPlace<PAIRS ? RROW : KROW> more;
        if constexpr (PAIRS) more.set(lds_addr(&lds.krest[0][0]) + (uint32_t)((t & 1) * RB), r, h);
        u32x4 a[ALL];
        auto read = [&](int n) {
            if (n < N) a[n] = lds_read16(place.at[n / NB % place.N] + (uint32_t)(n / NB / place.N * place.N * 32 + n % NB * 32 * KROW));
            else a[n] = lds_read16(more.at[(n - N) / NB % more.N] + (uint32_t)((n - N) / NB / more.N * more.N * 32 + n % NB * 32 * RROW));
        };
#pragma unroll
        for (int n = 0; n < AHEAD && n < ALL; ++n) read(n);
#pragma unroll
        for (int n = 0; n < ALL; ++n) {
            if (n + AHEAD < ALL) read(n + AHEAD);
            f32x16& x = s[0][n % NB];
            x = n < NB ? Mat<E>::mma(a[n], w.q[0][n / NB], f32x16{}) : Mat<E>::mma(a[n], w.q[0][(n < N ? n : n - N) / NB], x);
            beside(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // masks of tile t's scores; whether there was nothing to mask
    auto mask = [&](int t, f32x16 (&s)[1][NB]) {
        const uint64_t there = there_at[t & 3];
        const uint64_t whole = KT == 64 ? ~0ull : (1ull << (KT & 63)) - 1;
        const uint64_t have = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(there >> 32)) << 32 |
                              (uint32_t)__builtin_amdgcn_readfirstlane((int)there);
        if (have == whole && vmin >= (t + 1) * KT) return true;
        const int lim[1] = {vis - t * KT};
        mask_scores(s, have, lim);
        return false;
    };

    // keys of tile 0 and 1 and the values of tile 0 are on their way before the first turn
    if (wave == 0) {
        int page[3];
#pragma unroll
        for (int t = 0; t < 3; ++t) page[t] = page_of(t);
#pragma unroll
        for (int t = 0; t < 3; ++t) place_rows(t, page[t]);
    }
    // (the query is there from here on: else the waits for it would stand in the loop, and wait for tiles)
#pragma unroll
    for (int st = 0; st < ST; ++st) asm volatile("" : "+v"(w.q[0][st]));
    meet();
    f32x16 s0[1][NB], s1[1][NB];
    float top = -INFINITY;
    bool full = true;
    if (tiles > 0) {
        fetch(keys, 0);
        widen(keys, 0);
        if constexpr (!KV8) dma_wait();
        meet();
        if (tiles > 1) fetch(keys, 1);
        fetch(values, 0);
        if (mine > 0) {
            multiply_keys(0, s0, [](int) {});
            full = mask(0, s0);
#pragma unroll
            for (int j = 0; j < 16 * NB; ++j) top = fmaxf(top, s0[0][j / 16][j % 16]);
        }
        if (tiles > 1) widen(keys, 1);
        widen(values, 0);
    }
    // the turn of tile t, whose scores are there: powers, values, and the scores of the next
    auto turn = [&](int t, f32x16 (&now)[1][NB], f32x16 (&next)[1][NB]) {
        if constexpr (!KV8) dma_wait();
        meet();       // keys t + 1 and values t are there; every wave is done with keys t and values t - 1
        int page = -1;
        if (wave == 0) page = page_of(t + 3);
        if (t + 2 < tiles) fetch(keys, t + 2);
        if (t + 1 < tiles) fetch(values, t + 1);
        if (t < mine) {
            raise_top<E>(w, top, p.c);
            float mc = w.mc[0];
            uint32_t pr[1][NB][8], rest[NB][8];
            float sum = 0.0f;
            // pairs of weights, as B operands
            auto power = [&](int j) {
                const float x = exp2_fast(__builtin_fmaf(now[0][j / 8][j % 8 * 2], p.c, -mc));
                const float y = exp2_fast(__builtin_fmaf(now[0][j / 8][j % 8 * 2 + 1], p.c, -mc));
                sum += x + y;
                pr[0][j / 8][j % 8] = Mat<E>::pack2(x, y);
                asm volatile("" : "+v"(pr[0][j / 8][j % 8]), "+v"(sum));     // (here, not where it is used)
                if constexpr (WIDE) {
                    uint32_t& left = rest[j / 8][j % 8];
                    left = Mat<E>::pack2(x - Mat<E>::low(pr[0][j / 8][j % 8]), y - Mat<E>::high(pr[0][j / 8][j % 8]));
                    asm volatile("" : "+v"(left));
                }
            };
            const bool more = t + 1 < mine, all = full;
            if (more) {
                multiply_keys(t + 1, next, [&](int n) {
#pragma unroll
                    for (int j = n * 8 / (ST + SR); j < (n + 1) * 8 / (ST + SR); ++j) power(j);
                });
                full = mask(t + 1, next);
            } else {
                asm volatile("" : "+v"(mc));      // (or both branches' powers were taken ahead of them)
#pragma unroll
                for (int j = 0; j < 8 * NB; ++j) power(j);
            }
            w.l[0] += sum;
            top = -INFINITY;
            ValuePlace<VROW> vp, vq;
            vp.set(vbuf + (uint32_t)((t & 1) * VB), lane);
            if constexpr (PAIRS) vq.set(lds_addr(&lds.vrest[0][0]) + (uint32_t)((t & 1) * VB), lane);
            constexpr int N = CB * KS, P = PAIRS ? 2 : 1;         // products of a fragment and of its rest
            u32x4 a[N * P];
            auto read = [&](int n) { a[n] = n % P == 0 ? vp.read(n / P % CB, n / P / CB) : vq.read(n / P % CB, n / P / CB); };
#pragma unroll
            for (int n = 0; n < AHEAD && n < N * P; ++n) read(n);
#pragma unroll
            for (int n = 0; n < N; ++n) {
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    if (n * P + q + AHEAD < N * P) read(n * P + q + AHEAD);
                    const uint32_t* pp = &pr[0][n / CB / 2][(n / CB & 1) * 4];
                    w.o[0][n % CB] = Mat<E>::mma(a[n * P + q], u32x4{pp[0], pp[1], pp[2], pp[3]}, w.o[0][n % CB]);
                }
                if constexpr (WIDE) {
                    const uint32_t* pl = &rest[n / CB / 2][(n / CB & 1) * 4];
                    w.o[0][n % CB] = Mat<E>::mma(a[n * P], u32x4{pl[0], pl[1], pl[2], pl[3]}, w.o[0][n % CB]);
                }
#pragma unroll
                for (int j = n * 16 * NB / N; j < (n + 1) * 16 * NB / N; ++j)
                    top = fmaxf(top, next[0][j / 16][j % 16]);       // (of no use behind the last)
                asm volatile("" : "+v"(top));
                __builtin_amdgcn_sched_barrier(0);
            }
            if (!all) {
                odd |= odd_values<E, false>(vbuf + (uint32_t)((t & 1) * VB), VB);
                if constexpr (PAIRS) odd |= odd_values<E, false>(lds_addr(&lds.vrest[0][0]) + (uint32_t)((t & 1) * VB), VB);
            }
        }
        if (wave == 0 && t + 3 < tiles) place_rows(t + 3, page);
        if (t + 2 < tiles) widen(keys, t + 2);
        if (t + 1 < tiles) widen(values, t + 1);
    };
#pragma unroll 1
    for (int t = 0; t < tiles; t += 2) {
        turn(t, s0, s1);
        if (t + 1 < tiles) turn(t + 1, s1, s0);
    }
    if (odd)
        slow_rows<E, KV8, DK, DV>(late_args<A>(), u, hk, unit, R, row0, row0 + wave_row, min(row0 + wave_row + 32, nrows), k0, k1);
    else
        write_rows<E>(late_args<A>(), u, w, hk, unit, R, row0, wave_row, nrows);
}

}  // namespace dcpa
