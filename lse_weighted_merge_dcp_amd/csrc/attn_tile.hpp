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

// Fragment addresses within a tile of 16-bit rows (see swz()).
template <int KROW> struct KeyPlace {      // key r of 32, columns 16 st + 8 h .. + 7
    static constexpr int N = KROW % 256 == 0 ? 8 : 4;
    uint32_t at[N];
    __device__ __forceinline__ void set(uint32_t base, int r, int h) {
#pragma unroll
        for (int j = 0; j < N; ++j) at[j] = base + (uint32_t)(r * KROW + ((2 * j + h) ^ swz<KROW / 16>(r)) * 16);
    }
    __device__ __forceinline__ u32x4 read(int st) const { return lds_read16(at[st % N] + (uint32_t)(st / N * N * 32)); }
};
template <int VROW> struct ValuePlace {    // 32 columns of block cb, the keys {0..3, 8..11} + 4 h of 16 ks ..
    static constexpr int N = VROW % 256 == 0 ? 4 : 2;
    uint32_t at[N];
    __device__ __forceinline__ void set(uint32_t base, int lane) {
        // 16 lanes read four rows of 32 bytes, transposed
        const int h = lane >> 5, g = (lane >> 4) & 1, li = lane & 15, row = 4 * h + li / 4;
#pragma unroll
        for (int j = 0; j < N; ++j)
            at[j] = base + (uint32_t)(row * VROW + (li & 1) * 8 + ((4 * j + 2 * g + (li & 3) / 2) ^ swz_v<VROW / 16>(row)) * 16);
    }
    __device__ __forceinline__ u32x4 read(int cb, int ks) const {
        const uint32_t a = at[cb % N] + (uint32_t)(cb / N * N * 64 + ks * 16 * VROW);
        const u32x2 x = lds_read_tr(a), y = lds_read_tr(a + 8 * VROW);
        return u32x4{x.x, x.y, y.x, y.y};
    }
};

// Scores of KT keys.
template <typename E, int DK, int RB, int KT, int KROW>
__device__ __forceinline__ void scores(f32x16 (&s)[RB][KT / 32], const u32x4 (&q)[RB][DK / 16], uint32_t kbase) {
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int kb = 0; kb < KT / 32; ++kb) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[rb][kb][i] = 0.0f;
        KeyPlace<KROW> place;
        place.set(kbase + (uint32_t)(kb * 32 * KROW), r, h);
#pragma unroll
        for (int st = 0; st < DK / 16; ++st) {
            const u32x4 a = place.read(st);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) s[rb][kb] = Mat<E>::mma(a, q[rb][st], s[rb][kb]);
        }
    }
}

// Masks a tile's scores.  `there`: bit j set where key j of the tile exists.
// vis[rb]: how many keys from the tile's first on the lane's row sees (any
// value; compared with the key's place).
template <int RB, int NB>
__device__ __forceinline__ void mask_scores(f32x16 (&s)[RB][NB], uint64_t there, const int (&vis)[RB]) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
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

// The reference exponent for a tile whose scores reach `best` (of this half-wave's
// keys); rescales sum and outputs where it moves.
template <typename E, int DK, int DV, int RB>
__device__ __forceinline__ void raise_top(Rows<DK, DV, RB>& w, float best, float c, int rb = 0) {
    const float top = half_max(best) * c;
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
}

// Weights of a tile's scores, as B operands: p, rounded to the payload type, and
// in `rest` what the rounding left, so that the two together hold a weight to
// 2^-17 (bf16) or 2^-22 (fp16) of itself.  Updates maximum, sum and, where the
// maximum moved, the outputs.  full: no masking needed.
template <typename E, int DK, int DV, int RB, int NB>
__device__ __forceinline__ void weights(Rows<DK, DV, RB>& w, f32x16 (&s)[RB][NB], uint32_t (&p)[RB][NB][8],
                                        uint32_t (&rest)[RB][NB][8], uint64_t there, const int (&vis)[RB], bool full,
                                        float c) {
    if (!full) mask_scores(s, there, vis);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        float top = -INFINITY;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[rb][kb][i]);
        raise_top<E>(w, top, c, rb);
        float sum = 0.0f;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = exp2_fast(__builtin_fmaf(s[rb][kb][2 * i], c, -w.mc[rb]));
                const float y = exp2_fast(__builtin_fmaf(s[rb][kb][2 * i + 1], c, -w.mc[rb]));
                sum += x + y;
                p[rb][kb][i] = Mat<E>::pack2(x, y);
                rest[rb][kb][i] = Mat<E>::pack2(x - Mat<E>::low(p[rb][kb][i]), y - Mat<E>::high(p[rb][kb][i]));
            }
        w.l[rb] += sum;
    }
}

// Outputs += weights x values of KT keys, the weights in two products (see weights()); `fragment` as ValuePlace::read.
template <typename E, int DK, int DV, int RB, int KT, typename F>
__device__ __forceinline__ void outputs(Rows<DK, DV, RB>& w, const uint32_t (&p)[RB][KT / 32][8],
                                        const uint32_t (&rest)[RB][KT / 32][8], F&& fragment) {
#pragma unroll
    for (int cb = 0; cb < DV / 32; ++cb)
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
            const u32x4 a = fragment(cb, ks);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const uint32_t *pp = &p[rb][ks / 2][(ks & 1) * 4], *pr = &rest[rb][ks / 2][(ks & 1) * 4];
                w.o[rb][cb] = Mat<E>::mma(a, u32x4{pp[0], pp[1], pp[2], pp[3]}, w.o[rb][cb]);
                w.o[rb][cb] = Mat<E>::mma(a, u32x4{pr[0], pr[1], pr[2], pr[3]}, w.o[rb][cb]);
            }
        }
}

// A value that one row sees and another does not must not reach the other as
// 0 * infinity, which a matrix product cannot avoid.  Where a masked tile
// holds anything not finite the wave's rows are computed again by slow_rows().
// Whether the `bytes` bytes at `base` hold such a value; CODE: 8-bit NaN codes.
template <typename E, bool CODE>
__device__ __forceinline__ bool odd_values(uint32_t base, int bytes) {
    uint32_t hit = 0;
#pragma unroll 1
    for (int i = (threadIdx.x & 63) * 16; i < bytes; i += 1024) {
        const u32x4 x = lds_read16(base + (uint32_t)i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (CODE) {
#pragma unroll
                for (int j = 0; j < 4; ++j) hit |= (x[k] >> (8 * j) & 0x7fu) == 0x7fu;
            } else {
                hit |= (x[k] & Mat<E>::kExp & 0xffffu) == (Mat<E>::kExp & 0xffffu) ||
                       (x[k] & Mat<E>::kExp & 0xffff0000u) == (Mat<E>::kExp & 0xffff0000u);
            }
        }
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
