// attn_rope.hip -- per-head RMS norm and position rotation of new queries and
// keys in one pass, the keys and values written into the cache.
//
// A stream: each row (one head of one token) is read once and written once.
// A group of LPR lanes holds a row, eight elements (16 bytes) to a lane and
// slot; the mean of squares is one reduction over the group.  Sixteen lanes to a
// row of 576 (a 64-lane row left most of its second slot idle: 552 us for 8192 x
// 129 rows against 424 with 16 lanes, 5.7 TB/s; with eight lanes and nine slots
// the registers leave two waves to a SIMD: 651 us).  Rows turned by halves ask for
// cosines and sines too, and for a partner: 4000 x (64 + 8 + 8) heads of 128, all
// cached, take 56 us, 49 turned by pairs, where HBM alone would take 27.
#include "attn_device.hpp"

namespace dcpa {

namespace {

template <int LPR> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// Eight elements from column e0 on, times the row's factor and the weights.
template <typename E>
__device__ __forceinline__ void norm8(const dcp::Vec<16>& raw, int e0, const char* w, int nw, float f, float (&x)[8]) {
    dcp::Cvt<E, 16>::unpack(raw, x);
    if (e0 < nw) {
        float g[8];
        dcp::Cvt<E, 16>::unpack(dcp::vload<16>(w + e0 * 2), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g[i];
    }
}

template <typename E, bool KV8, bool PAIRS, int LPR, int SLOTS>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p) {
    constexpr int RPB = 256 / LPR;       // rows of a workgroup
    const int lane = (int)(threadIdx.x % LPR);
    const uint32_t row = blockIdx.x * RPB + threadIdx.x / LPR;
    const int token = (int)fdiv(row, p.fheads), which = (int)(row - (uint32_t)token * p.fheads.d);
    if (token >= p.T) return;
    // (without rotation there may be no positions)
    const int pos = p.rot > 0 ? min(max(p.pos[token], 0), p.positions - 1) : 0;
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
        // (slots may be past 32 bits)
        const int64_t page = slot / p.page_size, place = slot - page * p.page_size;
        const int hk = which - p.Hq - (value ? p.Hkv : 0);
        from = value ? p.v + (int64_t)token * p.v_T + (int64_t)hk * p.v_H : p.k + (int64_t)token * p.k_T + (int64_t)hk * p.k_H;
        to = value ? p.vc + page * p.vc_P + place * p.vc_S + (int64_t)hk * p.vc_H
                   : p.kc + page * p.kc_P + place * p.kc_S + (int64_t)hk * p.kc_H;
        if (value) D = p.Dv;
        else if (p.mass != nullptr && lane == 0) p.mass[page * p.m_P + place * p.m_S + hk * p.m_H] = 0.0f;
        narrow = KV8;
        scale = value ? p.iv : p.ik;
    }
    // the row as it was read; its pieces are widened one at a time, so that more rows are under way
    dcp::Vec<16> raw[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e0 = 8 * (s * LPR + lane);
        if (e0 < D) raw[s] = dcp::vload<16>(from + e0 * 2);
        else raw[s].w[0] = raw[s].w[1] = raw[s].w[2] = raw[s].w[3] = 0;
    }
    const char* w = query ? p.wq : p.wk;
    const int nw = value ? 0 : query ? p.nq : p.nk, rot = value ? 0 : p.rot, half = rot / 2;
    // Halves: the partners of four columns are the four that stand half a range (a multiple of four) away.  With a
    // piece to a lane they come from another lane; else they are read again, out of the cache, and before any store
    // (the row may be written in place).
    auto partner = [&](int s, int g) {
        const int col = 8 * (s * LPR + lane) + 4 * g;
        return col - p.off < half ? col + half : col - half;
    };
    dcp::Vec<16> other[SLOTS];
    if constexpr (!PAIRS && SLOTS > 1)
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int at = 8 * (s * LPR + lane) - p.off;
            if (at >= 0 && at < rot)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const dcp::Vec<8> y = dcp::vload<8>(from + partner(s, g) * 2);
                    other[s].w[2 * g] = y.w[0];
                    other[s].w[2 * g + 1] = y.w[1];
                }
        }
    float f = 1.0f;
    if (nw > 0) {
        float sq = 0.0f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (8 * (s * LPR + lane) < nw) {
                float x[8];
                dcp::Cvt<E, 16>::unpack(raw[s], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sq += x[i] * x[i];
            }
        f = 1.0f / __builtin_sqrtf(group_sum<LPR>(sq) / (float)nw + p.eps);
    }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        if constexpr (SLOTS > 1) asm volatile("" : "+v"(raw[s].w[0]), "+v"(raw[s].w[1]), "+v"(raw[s].w[2]), "+v"(raw[s].w[3]));
        const int e0 = 8 * (s * LPR + lane), at = e0 - p.off;
        float x[8];
        norm8<E>(raw[s], e0, w, nw, f, x);
        const bool turned = at >= 0 && at < rot;
        if constexpr (PAIRS) {
            if (turned) {
                const f32x4 c = *(const f32x4*)(cs + at / 2), n = *(const f32x4*)(cs + half + at / 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * c[i] - b * n[i];
                    x[2 * i + 1] = b * c[i] + a * n[i];
                }
            }
        } else {
            float y[8];
            if constexpr (SLOTS == 1) {
                const bool other_four = half % 8 != 0;        // (of the piece)
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[4 * g + i] = __shfl(other_four ? x[4 * (1 - g) + i] : x[4 * g + i], partner(s, g) / 8 & (LPR - 1), LPR);
            } else if (turned) {
                dcp::Cvt<E, 16>::unpack(other[s], y);
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    if (partner(s, g) < nw) {
                        float t[4];
                        dcp::Cvt<E, 8>::unpack(dcp::vload<8>(w + partner(s, g) * 2), t);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[4 * g + i] = y[4 * g + i] * f * t[i];
                    }
            }
            if (turned) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const bool low = at + 4 * g < half;
                    const int j = low ? at + 4 * g : at + 4 * g - half;
                    const f32x4 c = *(const f32x4*)(cs + j), n = *(const f32x4*)(cs + half + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& v = x[4 * g + i];
                        v = low ? v * c[i] - y[4 * g + i] * n[i] : v * c[i] + y[4 * g + i] * n[i];
                    }
                }
            }
        }
        if (e0 >= D) continue;
        if (KV8 && narrow) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= scale;
            dcp::vstore<8>(to + e0, dcp::Cvt<dcp::FP8T, 8>::pack(x));
        } else {
            dcp::vstore<16>(to + e0 * 2, dcp::Cvt<E, 16>::pack(x));
        }
    }
}

template <typename E, bool KV8, bool PAIRS> hipError_t run(const RopeArgs& a, hipStream_t stream) {
    const int D = a.v != nullptr && a.Dv > a.D ? a.Dv : a.D;
    const int64_t heads = a.Hq + a.Hkv * (a.v != nullptr ? 2 : 1);
    // at most 2^23 workgroups to a launch: as many tokens at a time
    auto go = [&](void (*kernel)(RopeArgs), int lpr) {
        const int64_t rows = 256 / lpr, most = (rows << 23) / heads;
        RopeArgs b = a;
        for (int64_t t = 0; t < a.T; t += most) {
            b.T = (int32_t)(a.T - t < most ? a.T - t : most);
            b.q = a.q + t * a.q_T;
            b.k = a.k + t * a.k_T;
            if (a.v != nullptr) b.v = a.v + t * a.v_T;
            b.qo = a.qo + t * a.qo_T;
            if (a.pos != nullptr) b.pos = a.pos + t;
            b.slots = a.slots + t;
            const hipError_t e = launch(kernel, dim3((uint32_t)((b.T * heads + rows - 1) / rows)), dim3(256), stream, b);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    if (D <= 64) return go(rope_kernel<E, KV8, PAIRS, 8, 1>, 8);
    if (D <= 128) return go(rope_kernel<E, KV8, PAIRS, 16, 1>, 16);
    if (D <= 256) return go(rope_kernel<E, KV8, PAIRS, 16, 2>, 16);
    if (D <= 512) return go(rope_kernel<E, KV8, PAIRS, 16, 4>, 16);
    if (D <= 640) return go(rope_kernel<E, KV8, PAIRS, 16, 5>, 16);
    return go(rope_kernel<E, KV8, PAIRS, 16, 8>, 16);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool bf16, bool kv8, hipStream_t stream) {
    if (a.pairs != 0) {
        if (bf16) return kv8 ? run<BF16T, true, true>(a, stream) : run<BF16T, false, true>(a, stream);
        return kv8 ? run<F16T, true, true>(a, stream) : run<F16T, false, true>(a, stream);
    }
    if (bf16) return kv8 ? run<BF16T, true, false>(a, stream) : run<BF16T, false, false>(a, stream);
    return kv8 ? run<F16T, true, false>(a, stream) : run<F16T, false, false>(a, stream);
}

}  // namespace dcpa
