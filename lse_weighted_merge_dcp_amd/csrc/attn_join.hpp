// attn_join.hpp -- one row from its parts: the outputs and log-sum-exps of the key
// ranges that went to different workgroups, on one scale.  Shared by attn.hip and
// attn_prefix.hip, which find a row's parts each in its own way.
#pragma once
#include "attn_tile.hpp"

namespace dcpa {

// Row (t, head) from n parts, part(k) the place of the k-th; a wave's work, each lane four columns (NC times), or
// that of a workgroup of four waves (TOGETHER; `share`: their sums).  Eight parts under way at once (four of
// wide rows).
template <typename E, int NC, bool TOGETHER, typename A, typename F>
__device__ __forceinline__ void join_parts(const A& p, f32x4 (&share)[TOGETHER ? 4 : 1][NC][64], int t, int head, int n,
                                           F&& part) {
    constexpr int FLY = NC == 1 ? 8 : 4;       // parts under way at once
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    float top = -INFINITY;
    bool bad = false;
    for (int k = lane; k < n; k += 64) {
        const float y = p.ws_l[part(k)];
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
    for (int k0 = 0; k0 < n; k0 += 64) {
        // a lane to a part's weight
        const int here = min(64, n - k0);
        const float f = lane < here ? exp2_fast(p.ws_l[part(k0 + lane)] - ref) : 0.0f;
        sum += f;
#pragma unroll 1
        for (int k = TOGETHER ? wave * FLY : 0; k < here; k += TOGETHER ? 4 * FLY : FLY) {
            f32x4 y[FLY][NC];
#pragma unroll
            for (int i = 0; i < FLY; ++i)
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const int col = min(j * 256 + lane * 4, p.Dv - 4);
                    y[i][j] = *(const f32x4*)(p.ws_o + part(k0 + min(k + i, here - 1)) * p.Dv + col);
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
        if (wave != 0) return;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    char* o = p.out + (int64_t)t * p.o_T + (int64_t)head * p.o_H;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int col = j * 256 + lane * 4;
        if (col < p.Dv)
            store4<E>(o + col * 2, acc[j * 4] * inv, acc[j * 4 + 1] * inv, acc[j * 4 + 2] * inv, acc[j * 4 + 3] * inv);
    }
    if (lane == 0 && p.lse != nullptr)
        p.lse[(int64_t)t * p.l_T + (int64_t)head * p.l_H] =
            (sum == 0.0f ? -INFINITY : ref + __builtin_amdgcn_logf(sum)) * p.lmul;
}

}  // namespace dcpa
