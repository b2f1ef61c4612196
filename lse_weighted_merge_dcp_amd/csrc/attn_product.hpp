// attn_product.hpp -- a workgroup's tiles of Y[m][n] = sum_k X[m][k] W[n][k],
// one after the other: both operands in LDS, K in steps, products in matrix
// instructions.
//
// The steps of all tiles make one row, so that the first operands of a tile are on
// their way while the last one's products are taken and its results go out (4096
// tokens' queries by a workgroup to each tile of 128 x 128: 349 us, 229 so).  The
// product is computed transposed (A = weights, B = rows), so that a lane holds, of
// one row m, four neighbouring columns n in a register group; an exchange between
// the half-waves makes them eight, and through 4 KB of LDS of its own a wave turns
// them into whole lines of 128 bytes of a row.  (Stored from the registers in pieces
// of 32 bytes, lines left the L2 half written: 1.9 GB for 1.3.)
#pragma once
#include "attn_device.hpp"

namespace dcpa {

// MT x NT: the tile, KT: columns of a step; WM x WN: the waves' places in the tile; ST: steps in LDS at once
// (ST - 1 of them on their way).  TURNED: the weights lie with n innermost ([k][n]) and are transposed as they
// are read from LDS.  X8: rows of 8-bit values, widened on their way into LDS.
template <typename E, int MT_, int NT_, int KT_, int WM, int WN, int ST, bool TURNED, bool X8> struct Product {
    static constexpr int MT = MT_, NT = NT_, KT = KT_, THREADS = WM * WN * 64;
    static constexpr int BM = MT / WM / 32, BN = NT / WN / 32;
    static constexpr int ROW = KT * 2, KC = KT / 8;                    // bytes and pieces of a row of KT columns (see swz())
    static constexpr int XB = MT * ROW, WB = NT * ROW;                 // bytes of a step
    static constexpr int NX = XB / 16 / THREADS, NW = WB / 16 / THREADS;
    static constexpr int WC = TURNED ? NT / 8 : KC;                    // 16-byte pieces of a row of weights in LDS
    static constexpr int OC = BN * 4;                                  // pieces of a wave's part of a row of results
    static constexpr int OB = 32 * OC * 16;                            // bytes of 32 such rows
    static constexpr int STORES = BM * OC / 2;                         // a wave's stores of a tile
    static_assert(XB % (16 * THREADS) == 0 && WB % (16 * THREADS) == 0, "a step is whole rounds of the workgroup");
    static_assert(THREADS / WC % 16 == 0 && THREADS / KC % 16 == 0, "the pieces of a thread lie at one place of their rows");
    static constexpr int LDS = ST * (XB + WB) + WM * WN * OB;

    uint32_t xs, ws, os;                 // LDS addresses
    int tid, lane, wave, wm, wn;
    f32x16 acc[BN][BM];
    u32x2 raw[X8 ? NX : 1];
    uint64_t xat[NX], wat[NW];           // the thread's pieces of the tile that is fetched, without the step
    int xc, wc;                          // their piece within the row: of k, of n where turned
    bool n_here;                         // (turned) whether the thread's columns exist

    __device__ __forceinline__ Product(char* lds) {
        tid = threadIdx.x;
        lane = tid & 63;
        wave = (int)dcp::wave_id();
        wm = wave % WM;
        wn = wave / WM;
        xs = lds_addr(lds);
        ws = xs + ST * XB;
        os = ws + ST * WB + (uint32_t)(wave * OB);
        xc = (tid % KC) ^ swz<KC>(tid / KC);
        wc = (tid % WC) ^ swz<WC>(tid / WC);
        n_here = true;
    }
    // row of the tile that piece i of this thread belongs to (a row of k where the weights are turned)
    __device__ __forceinline__ int x_row(int i) const { return i * (THREADS / KC) + tid / KC; }
    __device__ __forceinline__ int w_row(int i) const { return i * (THREADS / WC) + tid / WC; }

    // Step k0 .. k0 + KT - 1 of the tile asked for, into place s.  K: columns (rows of turned weights) that there are;
    // w_K: bytes between rows of turned weights.
    __device__ __forceinline__ void fetch(int s, int k0, int K, int64_t w_K) {
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
    // 8-bit rows of the step that has been asked for last, into place s
    __device__ __forceinline__ void widen(int s) {
        if constexpr (X8)
#pragma unroll
            for (int i = 0; i < NX; ++i) lds_write16(xs + (uint32_t)(s * XB + (i * THREADS + tid) * 16), widen8<E>(raw[i]));
    }
    __device__ __forceinline__ void multiply(int s) {
        const uint32_t xb = xs + (uint32_t)(s * XB + wm * BM * 32 * ROW), wb = ws + (uint32_t)(s * WB);
        const int r = lane & 31, h = lane >> 5, g = (lane >> 4) & 1, li = lane & 15;
#pragma unroll
        for (int st = 0; st < KT / 16; ++st) {
            u32x4 a[BN], b[BM];
            const uint32_t at = (uint32_t)(r * ROW + ((2 * st + h) ^ swz<KC>(r)) * 16);
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                const int nb = wn * BN + i;                  // block of 32 columns
                if constexpr (TURNED) {
                    const int k = st * 16 + 8 * h + li / 4, c = nb * 4 + 2 * g + (li & 3) / 2;
                    const u32x2 lo = lds_read_tr(wb + (uint32_t)(k * NT * 2 + (c ^ swz<WC>(k)) * 16 + (li & 1) * 8));
                    const u32x2 hi = lds_read_tr(wb + (uint32_t)((k + 4) * NT * 2 + (c ^ swz<WC>(k + 4)) * 16 + (li & 1) * 8));
                    a[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
                } else {
                    a[i] = lds_read16(wb + (uint32_t)(nb * 32 * ROW) + at);
                }
            }
#pragma unroll
            for (int i = 0; i < BM; ++i) b[i] = lds_read16(xb + (uint32_t)(i * 32 * ROW) + at);
#pragma unroll
            for (int i = 0; i < BN; ++i)
#pragma unroll
                for (int j = 0; j < BM; ++j) acc[i][j] = Mat<E>::mma(a[i], b[j], acc[i][j]);
        }
    }
    // `tiles` tiles: aim(t) sets the addresses (xat, wat, n_here) of tile t, finish(t) takes its results and returns
    // whether it made exactly MADE vector memory operations (if it did, they need not be waited for with the
    // operands that were asked for before them).
    template <int MADE, typename F, typename G>
    __device__ __forceinline__ void run(int tiles, int K, int64_t w_K, F&& aim, G&& finish) {
        const int steps = (K + KT - 1) / KT;
        int ft = 0, fk = 0, fs = 0;          // the next step to ask for: tile, step, place
        auto ask = [&] {
            if (ft == tiles) return;
            if (fk == 0) aim(ft);
            fetch(fs, fk * KT, K, w_K);
        };
        auto asked = [&] {
            if (ft == tiles) return;
            widen(fs);
            fs = fs + 1 == ST ? 0 : fs + 1;
            if (++fk == steps) {
                fk = 0;
                ++ft;
            }
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            ask();
            asked();
        }
        int s = 0;
        bool made = false;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
#pragma unroll
            for (int i = 0; i < BN; ++i)
#pragma unroll
                for (int j = 0; j < BM; ++j)
#pragma unroll
                    for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
                // this step is there (later ones may still be on their way)
                if (ST > 2 && ft < tiles) asm volatile("s_waitcnt vmcnt(%0)" :: "n"((ST - 2) * (NX + NW)) : "memory");
                else if (made && ST == 2) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(MADE) : "memory");
                else dma_wait();
                made = false;
                meet();
                ask();
                multiply(s);
                asked();
                s = s + 1 == ST ? 0 : s + 1;
            }
            made = finish(t);
        }
    }
    // The wave's results times `scale`, rounded, to the rows of the tile, `at` being where the columns out_col() .. + 7
    // of its first row lie and `bytes` a row's distance from the next; ok(row): whether they are written.  REST:
    // what the rounding left as well, likewise.  FAR: results that no cache will hold until they are read.
    __device__ __forceinline__ int out_col() const { return wn * BN * 32 + lane % OC * 8; }
    template <bool REST, bool FAR, typename F>
    __device__ __forceinline__ void store(float scale, char* at, int64_t bytes, char* rest, int64_t rest_bytes, F&& ok) {
        at += (wm * BM * 32 + lane / OC) * bytes;
        rest += (wm * BM * 32 + lane / OC) * rest_bytes;
        const int r = lane & 31, h = lane >> 5;
        // (rows of 128 bytes: two of them share 256)
        auto place = [](int row, int c) { return (uint32_t)(row * OC * 16 + (c ^ (OC == 8 ? row >> 1 & 7 : row >> 2 & 3)) * 16); };
        static_assert(OC == 4 || OC == 8, "rows of one or two blocks");
        // (a result that the type cannot hold is infinite and leaves nothing: their difference would make its row NaN)
        auto left = [](float x, float rounded) { return __builtin_isinf(rounded) ? 0.0f : x - rounded; };
#pragma unroll
        for (int j = 0; j < BM; ++j)
#pragma unroll
            for (int pass = 0; pass < (REST ? 2 : 1); ++pass) {
#pragma unroll
                for (int i = 0; i < BN; ++i)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[2][2];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int d = 0; d < 2; ++d) {
                                const int k = q * 8 + e * 4 + d * 2;
                                float x = acc[i][j][k] * scale, y = acc[i][j][k + 1] * scale;
                                // (one value each: the compiler would take the product into the conversion, which
                                // then rounds it once, and round it twice for the rest)
                                if constexpr (REST) asm("" : "+v"(x), "+v"(y));
                                v[e][d] = Mat<E>::pack2(x, y);
                                if (pass == 1) v[e][d] = Mat<E>::pack2(left(x, Mat<E>::low(v[e][d])), left(y, Mat<E>::high(v[e][d])));
                            }
                        // (the upper half-wave's part of the first group of four against the lower one's of the second)
                        const auto x = __builtin_amdgcn_permlane32_swap(v[0][0], v[1][0], false, false);
                        const auto y = __builtin_amdgcn_permlane32_swap(v[0][1], v[1][1], false, false);
                        lds_write16(os + place(r, i * 4 + q * 2 + h), u32x4{x[0], y[0], x[1], y[1]});
                    }
                // (a wave's LDS accesses stay in order)
                asm volatile("" ::: "memory");
#pragma unroll
                for (int k = 0; k < OC / 2; ++k) {
                    const int row = k * (64 / OC) + lane / OC;
                    const u32x4 v = lds_read16(os + place(row, lane % OC));
                    if (ok((wm * BM + j) * 32 + row)) {
                        u32x4* to = (u32x4*)(pass == 0 ? at : rest);
                        if constexpr (FAR) __builtin_nontemporal_store(v, to);
                        else *to = v;
                    }
                    // (from one row to the next, not all the addresses at once)
                    if (pass == 0) {
                        at += 64 / OC * bytes;
                        asm volatile("" : "+v"(at));
                    } else {
                        rest += 64 / OC * rest_bytes;
                        asm volatile("" : "+v"(rest));
                    }
                }
                asm volatile("" ::: "memory");
            }
    }
};

}  // namespace dcpa
