// attn_product.hpp -- a workgroup's tile of Y[m][n] = sum_k X[m][k] W[n][k]:
// both operands in LDS, K in steps of 64, products in matrix instructions.
//
// The product is computed transposed (A = weights, B = rows), so that a lane
// holds, of one row m, four neighbouring columns n in a register group; an
// exchange between the half-waves makes them eight, and the rows go out in
// pieces of 16 bytes without passing through LDS again.
#pragma once
#include "attn_device.hpp"

namespace dcpa {

// MT x NT: the tile; WM x WN: the waves' places in it; ST: steps of K in LDS at once (ST - 1 of them on
// their way).  TURNED: the weights lie with n innermost ([k][n]) and are transposed as they are read from
// LDS.  X8: rows of 8-bit values, widened on their way into LDS.
template <typename E, int MT_, int NT_, int WM, int WN, int ST, bool TURNED, bool X8> struct Product {
    static constexpr int MT = MT_, NT = NT_, KT = 64, THREADS = WM * WN * 64;
    static constexpr int BM = MT / WM / 32, BN = NT / WN / 32;
    static constexpr int XB = MT * 128, WB = NT * 128;                 // bytes of a step
    static constexpr int NX = XB / 16 / THREADS, NW = WB / 16 / THREADS;
    static constexpr int WC = TURNED ? NT / 8 : 8;                     // 16-byte pieces of a row of weights in LDS
    static_assert(XB % (16 * THREADS) == 0 && WB % (16 * THREADS) == 0, "a step is whole rounds of the workgroup");
    static_assert(THREADS / WC % 16 == 0, "the pieces of a thread lie at one place of their rows");
    static constexpr int LDS = ST * (XB + WB);

    uint32_t xs, ws;                     // LDS addresses
    int tid, lane, wave, wm, wn;
    f32x16 acc[BN][BM];
    u32x2 raw[X8 ? NX : 1];
    uint64_t xat[NX], wat[NW];           // the thread's pieces of step 0 (without the column)
    int xc, wc;                          // their piece within the row: of k, of n where turned

    __device__ __forceinline__ Product(char* lds) {
        tid = threadIdx.x;
        lane = tid & 63;
        wave = (int)dcp::wave_id();
        wm = wave % WM;
        wn = wave / WM;
        xs = lds_addr(lds);
        ws = xs + ST * XB;
        xc = (tid & 7) ^ swz<8>(tid / 8);
        wc = (tid % WC) ^ swz<WC>(tid / WC);
    }
    // row of the tile that piece i of this thread belongs to (a row of k where the weights are turned)
    __device__ __forceinline__ int x_row(int i) const { return i * (THREADS / 8) + tid / 8; }
    __device__ __forceinline__ int w_row(int i) const { return i * (THREADS / WC) + tid / WC; }

    // Step kt asked for.  K: columns (rows of turned weights) that there are; w_K: bytes between rows of turned
    // weights; n_here: whether the thread's columns of turned weights exist.
    __device__ __forceinline__ void fetch(int kt, int K, int64_t w_K, bool n_here) {
        const int s = kt % ST, k0 = kt * KT;
        const bool whole = k0 + KT <= K;
        const bool x_in = whole || k0 + xc * 8 < K;
        const uint32_t xto = xs + (uint32_t)(s * XB + wave * 1024), wto = ws + (uint32_t)(s * WB + wave * 1024);
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const uint64_t at = at_or_zeros(x_in, xat[i] + (uint64_t)((k0 + xc * 8) * (X8 ? 1 : 2)));
            if constexpr (X8) raw[i] = *(const u32x2*)at;
            else dma16((const char*)at, xto + (uint32_t)(i * THREADS * 16));
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            uint64_t at;
            if constexpr (TURNED)
                at = at_or_zeros(n_here && (whole || k0 + w_row(i) < K), wat[i] + (uint64_t)((int64_t)k0 * w_K));
            else
                at = at_or_zeros(whole || k0 + wc * 8 < K, wat[i] + (uint64_t)((k0 + wc * 8) * 2));
            dma16((const char*)at, wto + (uint32_t)(i * THREADS * 16));
        }
    }
    // 8-bit rows of step kt, which have been asked for last, into LDS
    __device__ __forceinline__ void widen(int kt) {
        if constexpr (X8)
#pragma unroll
            for (int i = 0; i < NX; ++i)
                lds_write16(xs + (uint32_t)(kt % ST * XB + (i * THREADS + tid) * 16), widen8<E>(raw[i]));
    }
    __device__ __forceinline__ void multiply(int kt) {
        const uint32_t xb = xs + (uint32_t)(kt % ST * XB + wm * BM * 32 * 128), wb = ws + (uint32_t)(kt % ST * WB);
        const int r = lane & 31, h = lane >> 5, g = (lane >> 4) & 1, li = lane & 15;
#pragma unroll
        for (int st = 0; st < KT / 16; ++st) {
            u32x4 a[BN], b[BM];
            const uint32_t at = (uint32_t)(r * 128 + ((2 * st + h) ^ swz<8>(r)) * 16);
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                const int nb = wn * BN + i;                  // block of 32 columns
                if constexpr (TURNED) {
                    const int k = st * 16 + 8 * h + li / 4, c = nb * 4 + 2 * g + (li & 3) / 2;
                    const u32x2 lo = lds_read_tr(wb + (uint32_t)(k * NT * 2 + (c ^ swz<WC>(k)) * 16 + (li & 1) * 8));
                    const u32x2 hi = lds_read_tr(wb + (uint32_t)((k + 4) * NT * 2 + (c ^ swz<WC>(k + 4)) * 16 + (li & 1) * 8));
                    a[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
                } else {
                    a[i] = lds_read16(wb + (uint32_t)(nb * 32 * 128) + at);
                }
            }
#pragma unroll
            for (int i = 0; i < BM; ++i) b[i] = lds_read16(xb + (uint32_t)(i * 32 * 128) + at);
#pragma unroll
            for (int i = 0; i < BN; ++i)
#pragma unroll
                for (int j = 0; j < BM; ++j) acc[i][j] = Mat<E>::mma(a[i], b[j], acc[i][j]);
        }
    }
    __device__ __forceinline__ void run(int K, int64_t w_K, bool n_here) {
        static_assert(!X8 || ST == 2, "8-bit rows stay in registers for one step");
#pragma unroll
        for (int i = 0; i < BN; ++i)
#pragma unroll
            for (int j = 0; j < BM; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
        const int steps = (K + KT - 1) / KT;
#pragma unroll
        for (int t = 0; t < ST - 1; ++t)
            if (t < steps) {
                fetch(t, K, w_K, n_here);
                widen(t);
            }
#pragma unroll 1
        for (int t = 0; t < steps; ++t) {
            // step t is there (later ones may still be on their way)
            if (t + ST - 2 < steps) asm volatile("s_waitcnt vmcnt(%0)" :: "n"((ST - 2) * (NX + NW)) : "memory");
            else dma_wait();
            meet();
            const bool more = t + ST - 1 < steps;
            if (more) fetch(t + ST - 1, K, w_K, n_here);
            multiply(t);
            if (more) widen(t + ST - 1);
        }
    }
    // The wave's results times `scale`, rounded, in pieces of eight columns: put(row of the tile, column of the
    // tile, piece, what the rounding left where REST).
    template <bool REST, typename F> __device__ __forceinline__ void store(float scale, F&& put) {
        const int r = lane & 31, h = lane >> 5;
        // (the upper half-wave's part of the first group of four against the lower one's of the second)
        auto join = [](const uint32_t (&v)[2][2]) {
            const auto x = __builtin_amdgcn_permlane32_swap(v[0][0], v[1][0], false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(v[0][1], v[1][1], false, false);
            return u32x4{x[0], y[0], x[1], y[1]};
        };
#pragma unroll
        for (int j = 0; j < BM; ++j)
#pragma unroll
            for (int i = 0; i < BN; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t v[2][2], rest[2][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            const int k = q * 8 + e * 4 + d * 2;
                            float x = acc[i][j][k] * scale, y = acc[i][j][k + 1] * scale;
                            // (one value each: the compiler would take the product into the conversion, which then
                            // rounds it once, and round it twice for the rest)
                            if constexpr (REST) asm("" : "+v"(x), "+v"(y));
                            v[e][d] = Mat<E>::pack2(x, y);
                            if constexpr (REST) rest[e][d] = Mat<E>::pack2(x - Mat<E>::low(v[e][d]), y - Mat<E>::high(v[e][d]));
                        }
                    const u32x4 whole = join(v);
                    u32x4 left = {};
                    if constexpr (REST) left = join(rest);
                    put((wm * BM + j) * 32 + r, (wn * BN + i) * 32 + q * 16 + h * 8, whole, left);
                }
    }
};

}  // namespace dcpa
