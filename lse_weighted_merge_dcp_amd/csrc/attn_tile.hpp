// attn_tile.hpp -- one tile of keys against the query rows of a wave: scores,
// online softmax and the product with the values.  Shared by the two
// attention kernels.
//
// Scores are computed transposed, S^T = K Q^T (A = keys, B = queries): lane l
// then holds, for query row l % 32 alone, the keys 8(i/4) + i%4 + 4h of every
// 32.  A row's maximum and sum need one exchange between the half-waves, its
// rescaling is a per-lane factor, and since the order of keys within a matrix
// product is free, the weights are already the B operand of O^T = V^T P^T:
// lane half h supplies keys {0..3, 8..11} + 4h of each 16, and the transposing
// LDS read fetches the values of just those keys.
#pragma once
#include "attn_device.hpp"

namespace dcpa {

// Wave state of RB blocks of 32 query rows.
template <int DK, int DV, int RB> struct Rows {
    u32x4 q[RB][DK / 16];
    f32x16 o[RB][DV / 32];
    float mc[RB];    // reference exponent (powers of two), already times c
    float l[RB];     // sum of this half-wave's weights
};

template <int DK, int DV, int RB>
__device__ __forceinline__ void clear_rows(Rows<DK, DV, RB>& w) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) w.o[rb][cb][i] = 0.0f;
        w.mc[rb] = kNoMax;
        w.l[rb] = 0.0f;
    }
}

// Query row `row` (clamped by the caller) of one head as B operand.
template <int DK, int N>
__device__ __forceinline__ void load_query(u32x4 (&q)[N], const char* row, int Dk, int h) {
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        // (one address for all columns, no branch around a load)
        const int c = 2 * s + h;
        const u32x4 x = *(const u32x4*)(row + min(c, Dk / 8 - 1) * 16);
        q[s] = c * 8 < Dk ? x : u32x4{0, 0, 0, 0};
    }
}

// One tile of KT keys.  kbase / vbase: LDS addresses of the key and value
// rows (KROW, VROW bytes apart).  `there`: bit j set where key j of the tile
// exists.  vis[rb]: how many keys from the tile's first on the lane's row sees
// (any value; compared with the key's place).  full: no masking needed.
template <typename E, int DK, int DV, int RB, int KT, int KROW, int VROW>
__device__ __forceinline__ bool attend(Rows<DK, DV, RB>& w, uint32_t kbase, uint32_t vbase, uint64_t there,
                                       const int (&vis)[RB], bool full, float c) {
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    constexpr int NB = KT / 32;
    f32x16 s[RB][NB];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[rb][kb][i] = 0.0f;
        const uint32_t krow = kbase + (uint32_t)((kb * 32 + r) * KROW);
        uint32_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = krow + (uint32_t)(((2 * j + h) ^ swz(r)) * 16);
#pragma unroll
        for (int st = 0; st < DK / 16; ++st) {
            const u32x4 a = lds_read16(at[st & 3] + (uint32_t)((st >> 2) * 128));
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) s[rb][kb] = Mat<E>::mma(a, w.q[rb][st], s[rb][kb]);
        }
    }
    uint32_t p[RB][NB][8];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        if (!full) {
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint32_t bits = (uint32_t)(there >> (32 * kb)) >> (4 * h);
                const int lim = vis[rb] - kb * 32 - 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = 8 * (i / 4) + i % 4;
                    s[rb][kb][i] = (bits >> j & 1u) != 0 && j < lim ? s[rb][kb][i] : -INFINITY;
                }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[rb][kb][i]);
        top = half_max(top) * c;
        // (kTop: the scale on which the type's weights keep their precision)
        if (__ballot(top > w.mc[rb] + Mat<E>::kTop + kLazy) != 0) {
            const float next = top > w.mc[rb] + Mat<E>::kTop ? top - Mat<E>::kTop : w.mc[rb];
            const float f = exp2_fast(w.mc[rb] - next);
            w.mc[rb] = next;
            w.l[rb] *= f;
#pragma unroll
            for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
                for (int i = 0; i < 16; ++i) w.o[rb][cb][i] *= f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = exp2_fast(__builtin_fmaf(s[rb][kb][2 * i], c, -w.mc[rb]));
                const float y = exp2_fast(__builtin_fmaf(s[rb][kb][2 * i + 1], c, -w.mc[rb]));
                sum += x + y;
                p[rb][kb][i] = Mat<E>::pack2(x, y);
            }
        w.l[rb] += sum;
    }
    // value fragments: 16 lanes read four rows of 32 bytes, transposed
    const int g = (lane >> 4) & 1, li = lane & 15;
    const uint32_t vrow = vbase + (uint32_t)((4 * h + li / 4) * VROW) + (uint32_t)((li & 1) * 8);
    uint32_t va[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) va[j] = vrow + (uint32_t)(((4 * j + 2 * g + (li & 3) / 2) ^ swz(4 * h + li / 4)) * 16);
    auto fragment = [&](int cb, int ks) {
        const uint32_t a = va[cb & 1] + (uint32_t)((cb >> 1) * 128 + ks * 16 * VROW);
        const u32x2 x = lds_read_tr(a), y = lds_read_tr(a + 8 * VROW);
        return u32x4{x.x, x.y, y.x, y.y};
    };
#pragma unroll
    for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
            const u32x4 a = fragment(cb, ks);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const uint32_t* pp = &p[rb][ks / 2][(ks & 1) * 4];
                w.o[rb][cb] = Mat<E>::mma(a, u32x4{pp[0], pp[1], pp[2], pp[3]}, w.o[rb][cb]);
            }
        }
    if (full) return false;
    uint32_t hit = 0;
#pragma unroll 1
    for (int i = lane; i < KT * (DV / 8); i += 64) {
        const u32x4 x = lds_read16(vbase + (uint32_t)((i / (DV / 8)) * VROW + (i % (DV / 8)) * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            hit |= (x[k] & Mat<E>::kExp & 0xffffu) == (Mat<E>::kExp & 0xffffu) ||
                   (x[k] & Mat<E>::kExp & 0xffff0000u) == (Mat<E>::kExp & 0xffff0000u);
    }
    return __ballot(hit != 0) != 0;
}

// A finished row: factor of its outputs and its log-sum-exp in powers of two.
__device__ __forceinline__ void finish(float l, float mc, float vs, float& f, float& lse2) {
    f = l == 0.0f ? 0.0f : vs / l;
    lse2 = l == 0.0f ? -INFINITY : mc + __builtin_amdgcn_logf(l);
}

// Lane's four neighbouring columns of 16-bit outputs (rows are 4-byte aligned).
template <typename E> __device__ __forceinline__ void store4(char* at, float a, float b, float c, float d) {
    dcp::Vec<8> v;
    v.w[0] = Mat<E>::pack2(a, b);
    v.w[1] = Mat<E>::pack2(c, d);
    dcp::vstore<8>(at, v);
}

}  // namespace dcpa
