// attn_rope.hip -- per-head RMS norm and position rotation of new queries and
// keys in one pass, the keys and values written into the cache.
//
// A stream: each row (one head of one token) is read once and written once.
// A group of LPR lanes holds a row, eight elements (16 bytes) to a lane and
// slot; the mean of squares is one reduction over the group, and the partner of
// a rotated column in the "halves" layout comes from another lane of the group.
#include "attn_device.hpp"

namespace dcpa {

namespace {

template <int LPR> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// One row: x[s] holds elements 8 (s LPR + lane) .. + 7.
template <typename E, int LPR, int SLOTS>
__device__ __forceinline__ void norm_turn(float (&x)[SLOTS][8], int lane, const char* row, const char* w, int nw, float eps,
                                          const float* cs, int off, int rot, bool pairs) {
    float f = 1.0f;
    if (nw > 0) {
        float sq = 0.0f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (8 * (s * LPR + lane) < nw)
#pragma unroll
                for (int i = 0; i < 8; ++i) sq += x[s][i] * x[s][i];
        f = 1.0f / __builtin_sqrtf(group_sum<LPR>(sq) / (float)nw + eps);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e0 = 8 * (s * LPR + lane);
            if (e0 < nw) {
                float g[8];
                dcp::Cvt<E, 16>::unpack(dcp::vload<16>(w + e0 * 2), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[s][i] = x[s][i] * f * g[i];
            }
        }
    }
    if (rot == 0) return;
    const int half = rot / 2;
    if (pairs) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e0 = 8 * (s * LPR + lane) - off;
            if (e0 >= 0 && e0 < rot) {
                const f32x4 c = *(const f32x4*)(cs + e0 / 2), n = *(const f32x4*)(cs + half + e0 / 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[s][2 * i], b = x[s][2 * i + 1];
                    x[s][2 * i] = a * c[i] - b * n[i];
                    x[s][2 * i + 1] = b * c[i] + a * n[i];
                }
            }
        }
    } else {
        // the partner stands half a range away: the same place of another chunk
        const int step = half / 8;
        float y[SLOTS][8];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int chunk = s * LPR + lane, e0 = 8 * chunk - off;
            const int partner = e0 < half ? chunk + step : chunk - step;
            if constexpr (SLOTS == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[s][i] = __shfl(x[s][i], partner & (LPR - 1), LPR);
            } else if (e0 >= 0 && e0 < rot) {
                // (read again, out of the cache, and normed alike: which slot holds it differs from lane to lane)
                dcp::Cvt<E, 16>::unpack(dcp::vload<16>(row + partner * 16), y[s]);
                if (partner * 8 < nw) {
                    float g[8];
                    dcp::Cvt<E, 16>::unpack(dcp::vload<16>(w + partner * 16), g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[s][i] = y[s][i] * f * g[i];
                }
            }
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e0 = 8 * (s * LPR + lane) - off;
            if (e0 >= 0 && e0 < rot) {
                const bool low = e0 < half;
                const int j = low ? e0 : e0 - half;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = cs[j + i], n = cs[half + j + i];
                    x[s][i] = low ? x[s][i] * c - y[s][i] * n : x[s][i] * c + y[s][i] * n;
                }
            }
        }
    }
}

template <typename E, bool KV8, int LPR, int SLOTS>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p) {
    constexpr int RPB = 256 / LPR;       // rows of a workgroup
    const int lane = (int)(threadIdx.x % LPR);
    const uint32_t row = blockIdx.x * RPB + threadIdx.x / LPR;
    const int token = (int)fdiv(row, p.fheads), which = (int)(row - (uint32_t)token * p.fheads.d);
    if (token >= p.T) return;
    const int pos = min(max(p.pos[token], 0), p.positions - 1);
    const float* cs = p.cs + (int64_t)pos * p.cs_P;
    const bool query = which < p.Hq, value = which >= p.Hq + p.Hkv;
    char* to;
    const char* from;
    int D = p.D;
    bool narrow = false;
    float scale = 1.0f;
    if (query) {
        from = p.q + (int64_t)token * p.q_T + (int64_t)which * p.q_H;
        to = p.qo + (int64_t)token * p.qo_T + (int64_t)which * p.qo_H;
    } else {
        const int64_t slot = p.slots[token];
        if (slot < 0 || slot >= p.slots_max) return;
        const int64_t page = slot / p.page_size, place = slot - page * p.page_size;
        const int hk = which - p.Hq - (value ? p.Hkv : 0);
        from = value ? p.v + (int64_t)token * p.v_T + (int64_t)hk * p.v_H : p.k + (int64_t)token * p.k_T + (int64_t)hk * p.k_H;
        to = value ? p.vc + page * p.vc_P + place * p.vc_S + (int64_t)hk * p.vc_H
                   : p.kc + page * p.kc_P + place * p.kc_S + (int64_t)hk * p.kc_H;
        if (value) D = p.Dv;
        narrow = KV8;
        scale = value ? p.iv : p.ik;
    }
    float x[SLOTS][8];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e0 = 8 * (s * LPR + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[s][i] = 0.0f;
        if (e0 < D) dcp::Cvt<E, 16>::unpack(dcp::vload<16>(from + e0 * 2), x[s]);
    }
    if (!value)
        norm_turn<E, LPR, SLOTS>(x, lane, from, query ? p.wq : p.wk, query ? p.nq : p.nk, p.eps, cs, p.off, p.rot, p.pairs != 0);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e0 = 8 * (s * LPR + lane);
        if (e0 >= D) continue;
        if (KV8 && narrow) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[s][i] *= scale;
            dcp::vstore<8>(to + e0, dcp::Cvt<dcp::FP8T, 8>::pack(x[s]));
        } else {
            dcp::vstore<16>(to + e0 * 2, dcp::Cvt<E, 16>::pack(x[s]));
        }
    }
}

template <typename E, bool KV8> hipError_t run(const RopeArgs& a, hipStream_t stream) {
    const int D = a.v != nullptr && a.Dv > a.D ? a.Dv : a.D;
    const int64_t rows = (int64_t)a.T * (a.Hq + a.Hkv * (a.v != nullptr ? 2 : 1));
    auto grid = [&](int lpr) { return dim3((uint32_t)((rows * lpr + 255) / 256)); };
    const dim3 block(256);
    if (D <= 64) return launch(rope_kernel<E, KV8, 8, 1>, grid(8), block, stream, a);
    if (D <= 128) return launch(rope_kernel<E, KV8, 16, 1>, grid(16), block, stream, a);
    if (D <= 256) return launch(rope_kernel<E, KV8, 16, 2>, grid(16), block, stream, a);
    if (D <= 512) return launch(rope_kernel<E, KV8, 16, 4>, grid(16), block, stream, a);
    if (D <= 640) return launch(rope_kernel<E, KV8, 16, 5>, grid(16), block, stream, a);
    return launch(rope_kernel<E, KV8, 16, 8>, grid(16), block, stream, a);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool bf16, bool kv8, hipStream_t stream) {
    if (bf16) return kv8 ? run<BF16T, true>(a, stream) : run<BF16T, false>(a, stream);
    return kv8 ? run<F16T, true>(a, stream) : run<F16T, false>(a, stream);
}

}  // namespace dcpa
