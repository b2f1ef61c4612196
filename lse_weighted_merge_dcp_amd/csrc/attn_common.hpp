// attn_common.hpp -- what the attention kernels share beside the tile: cache
// addresses, the writing of finished rows, and the row-by-row path.
#pragma once
#include "attn_tile.hpp"

namespace dcpa {

// The address of a cached token's row for one key head, or of a row of zeros
// where the table names no page.
__device__ __forceinline__ uint64_t page_row(int page, const Batch& m, const char* base, int64_t P, int64_t S,
                                             int64_t off, uint32_t place) {
    return at_or_zeros((uint32_t)page < (uint32_t)m.pages,
                       (uint64_t)(base + off) + times64((uint32_t)page, P) + times64(place, S));
}

// Writes a wave's finished rows: to the outputs, or as a part for the join.
template <typename E, int DK, int DV, int RB>
__device__ __forceinline__ void write_rows(const AttnArgs& p, const Unit& u, const Rows<DK, DV, RB>& w, int hk,
                                           int unit, int tile_rows, int row0, int wave_row, int nrows) {
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int in_tile = wave_row + rb * 32 + r, row = row0 + in_tile;
        const float l = half_sum(w.l[rb]);
        float f, lse2;
        finish(l, w.mc[rb], p.vs, f, lse2);
        if (row >= nrows) continue;
        if (u.splits > 1) {
            const int64_t at = ((int64_t)hk * p.units + unit) * tile_rows + in_tile;
            float* o = p.ws_o + at * p.Dv;
            if (h == 0) p.ws_l[at] = lse2;
#pragma unroll
            for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = cb * 32 + i * 8 + h * 4;
                    if (col < p.Dv) {
                        f32x4 x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = l == 0.0f ? 0.0f : w.o[rb][cb][i * 4 + k] * f;
                        *(f32x4*)(o + col) = x;
                    }
                }
        } else {
            const int token = (int)fdiv((uint32_t)row, p.m.fG), head = hk * p.m.G + row - token * p.m.G;
            char* o = p.out + (int64_t)(u.s.first + token) * p.o_T + (int64_t)head * p.o_H;
            if (h == 0 && p.lse != nullptr)
                p.lse[(int64_t)(u.s.first + token) * p.l_T + (int64_t)head * p.l_H] = lse2 * p.lmul;
#pragma unroll
            for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = cb * 32 + i * 8 + h * 4;
                    if (col < p.Dv) {
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = l == 0.0f ? 0.0f : w.o[rb][cb][i * 4 + k] * f;
                        store4<E>(o + col * 2, x[0], x[1], x[2], x[3]);
                    }
                }
        }
    }
}

// Rows [first, end) of the unit one by one, without matrix products: a wave to
// a row, the columns over its lanes, one key after the other, so that a key is
// either seen by the row or never touched.  Taken only where attend() asks for
// it (values that are not finite in a masked tile).  A call of its own, with
// its own copies of the arguments: a reference to the kernel's would move them
// from scalar registers to memory for the whole kernel.
template <typename E, bool KV8, int DK, int DV, typename A, typename U>
__device__ __noinline__ void slow_rows(A p, U u, int hk, int unit, int tile_rows, int row0,
                                       int first, int end, int k0, int k1) {
    const int lane = threadIdx.x & 63;
    constexpr int NQ = (DK + 63) / 64, NO = (DV + 63) / 64, ES = KV8 ? 1 : 2;
    using C = std::conditional_t<KV8, dcp::FP8T, E>;
    auto one = [](const char* at) {
        float f;
        if constexpr (KV8) dcp::Cvt<C, 1>::unpack(dcp::vload<1>(at), &f);
        else dcp::Cvt<C, 2>::unpack(dcp::vload<2>(at), &f);
        return f;
    };
    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;
#pragma unroll 1
    for (int row = first; row < end; ++row) {
        const int token = (int)fdiv((uint32_t)row, p.m.fG), head = hk * p.m.G + row - token * p.m.G;
        const int stop = min(k1, sees(p, u, token));
        const char* q = p.q + (int64_t)(u.s.first + token) * p.q_T + (int64_t)head * p.q_H;
        float x[NQ], acc[NO], mc = kNoMax, l = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            x[i] = 0.0f;
            if (lane + 64 * i < p.Dk) dcp::Cvt<E, 2>::unpack(dcp::vload<2>(q + (lane + 64 * i) * 2), &x[i]);
        }
#pragma unroll
        for (int i = 0; i < NO; ++i) acc[i] = 0.0f;
#pragma unroll 1
        for (int key = k0; key < stop; ++key) {
            const uint32_t page = fdiv((uint32_t)key, p.m.fpage);
            const int id = table[page];
            if ((uint32_t)id >= (uint32_t)p.m.pages) continue;
            const int64_t place = key - (int64_t)page * p.m.page_size;
            const char* kr = p.k + (int64_t)id * p.k_P + place * p.k_S + (int64_t)hk * p.k_H;
            const char* vr = p.v == nullptr ? kr : p.v + (int64_t)id * p.v_P + place * p.v_S + (int64_t)hk * p.v_H;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (lane + 64 * i < p.Dk) s += x[i] * one(kr + (lane + 64 * i) * ES);
            const char* rest = nullptr;
            if constexpr (std::is_same_v<A, PairArgs>) {
                const char* more = p.kr + (int64_t)id * p.kr_P + place * p.kr_S + (int64_t)hk * p.kr_H;
                rest = p.vr + (int64_t)id * p.vr_P + place * p.vr_S + (int64_t)hk * p.vr_H;
#pragma unroll
                for (int i = 0; i < NQ; ++i)
                    if (lane + 64 * i < p.Dr) s += x[i] * one(more + (lane + 64 * i) * ES);
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
            s *= p.c;
            const float next = fmaxf(mc, s), f = exp2_fast(mc - next), w = exp2_fast(s - next);
            mc = next;
            l = l * f + w;
#pragma unroll
            for (int i = 0; i < NO; ++i)
                if (lane + 64 * i < p.Dv)
                    acc[i] = acc[i] * f + w * (one(vr + (lane + 64 * i) * ES) + (rest != nullptr ? one(rest + (lane + 64 * i) * ES) : 0.0f));
        }
        float f, lse2;
        finish(l, mc, p.vs, f, lse2);
        const int64_t at = ((int64_t)hk * p.units + unit) * tile_rows + (row - row0);
        if (lane == 0) {
            if (u.splits > 1) p.ws_l[at] = lse2;
            else if (p.lse != nullptr) p.lse[(int64_t)(u.s.first + token) * p.l_T + (int64_t)head * p.l_H] = lse2 * p.lmul;
        }
#pragma unroll
        for (int i = 0; i < NO; ++i) {
            const int col = lane + 64 * i;
            if (col >= p.Dv) continue;
            const float o = l == 0.0f ? 0.0f : acc[i] * f;
            if (u.splits > 1) p.ws_o[at * p.Dv + col] = o;
            else dcp::vstore<2>(p.out + (int64_t)(u.s.first + token) * p.o_T + (int64_t)head * p.o_H + col * 2,
                                dcp::Cvt<E, 2>::pack(&o));
        }
    }
}

}  // namespace dcpa
