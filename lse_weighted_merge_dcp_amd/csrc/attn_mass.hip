// attn_mass.hip -- accumulated attention weight of every cached key.
//
// For one key head and a key j, the sum over the rows that see it of
// 2^(s_j c - g), g the row's merged log-sum-exp in powers of two.  Scores are
// computed transposed as in attn_tile.hpp: a wave keeps the fragments of 32
// keys in registers (A operand) and walks over the query rows (B operand, 32
// at a time); each lane adds up the weights of its own query row, and one sum
// over the 32 lanes at the end gives the keys' totals.  No two waves write the
// same key, so there are no atomics; where rows are many and keys few, the
// rows are split and mass_join adds the parts in order.
#include "attn_device.hpp"

namespace dcpa {

namespace {

constexpr int kKeys = 128;     // keys of a workgroup's step: 32 to a wave

// Key steps of all sequences, and the parts the rows are cut into so that
// steps * parts comes near the target.
__device__ __forceinline__ int row_parts(const Batch& m, int target) {
    if (target <= 0) return 1;
    const int lane = threadIdx.x & 63;
    int64_t steps = 0;
    int most = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64)
        if (b0 + lane < m.B) {
            const Seq s = load_seq(m, b0 + lane);
            if (s.n > 0) steps += (s.kv + kKeys - 1) / kKeys;
            most = max(most, s.n);
        }
    steps = sum_wave(steps);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) most = max(most, __shfl_xor(most, d, 64));
    const int64_t tiles = ((int64_t)most * m.G + 31) / 32;
    return (int)max((int64_t)1, min(min((int64_t)target / max((int64_t)1, steps), tiles), (int64_t)64));
}

struct Step {
    Seq s;
    int b, step, slot;
    bool ok;
};
__device__ __forceinline__ Step find_step(const Batch& m, int id) {
    Step u;
    u.ok = false;
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64) {
        int n = 0;
        if (b0 + lane < m.B) {
            const Seq s = load_seq(m, b0 + lane);
            n = s.n > 0 ? (s.kv + kKeys - 1) / kKeys : 0;
        }
        const int incl = base + scan_incl(n, lane);
        const uint64_t past = __ballot(incl > id);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            u.b = b0 + at;
            u.s = load_seq(m, u.b);
            u.step = id - (__builtin_amdgcn_readlane(incl, at) - __builtin_amdgcn_readlane(n, at));
            u.slot = id;
            u.ok = u.step >= 0;
            return u;
        }
        base = __builtin_amdgcn_readlane(incl, 63);
    }
    return u;
}

__device__ __forceinline__ float* mass_at(const MassArgs& p, int b, int hk, int key) {
    const uint32_t page = fdiv((uint32_t)key, p.m.fpage);
    const int id = p.m.table[(int64_t)b * p.m.t_B + page];
    if ((uint32_t)id >= (uint32_t)p.m.pages) return nullptr;
    return p.mass + (int64_t)id * p.m_P + (int64_t)(key - (int)(page * p.m.fpage.d)) * p.m_S + (int64_t)hk * p.m_H;
}

template <typename E, bool KV8, int DK>
__global__ __launch_bounds__(256, 2) void mass_kernel(MassArgs p) {
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int parts = row_parts(p.m, p.target);
    const uint32_t per = (uint32_t)(p.m.Hkv * parts);
    // a fixed grid walks over the steps
    for (uint32_t id = blockIdx.x;; id += gridDim.x) {
        const Step u = find_step(p.m, (int)(id / per));
        if (!u.ok) return;
        const int hk = (int)(id % (uint32_t)p.m.Hkv), part = (int)(id / (uint32_t)p.m.Hkv % (uint32_t)parts);
        const int key0 = u.step * kKeys + wave * 32, key = key0 + r;
        // the wave's keys as A operand
        u32x4 kf[DK / 16];
        bool have = false;
        const char* kr = nullptr;
        if (key < u.s.kv) {
            const uint32_t page = fdiv((uint32_t)key, p.m.fpage);
            const int pid = p.m.table[(int64_t)u.b * p.m.t_B + page];
            have = (uint32_t)pid < (uint32_t)p.m.pages;
            if (have) kr = p.k + (int64_t)pid * p.k_P + (int64_t)(key - (int)(page * p.m.fpage.d)) * p.k_S + (int64_t)hk * p.k_H;
        }
#pragma unroll
        for (int s = 0; s < DK / 16; ++s) {
            const int c = 2 * s + h;
            kf[s] = u32x4{0, 0, 0, 0};
            if (have && c * 8 < p.Dk) {
                if constexpr (KV8) kf[s] = widen8<E>(*(const u32x2*)(kr + c * 8));
                else kf[s] = *(const u32x4*)(kr + c * 16);
            }
        }
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
        const int nrows = u.s.n * p.m.G, tiles = (nrows + 31) / 32;
        const int per_part = (tiles + parts - 1) / parts;
        const int first = part * per_part, end = min(tiles, first + per_part);
#pragma unroll 1
        for (int t = first; t < end; ++t) {
            const int row = min(t * 32 + r, nrows - 1);
            const int token = (int)fdiv((uint32_t)row, p.m.fG), head = hk * p.m.G + row - token * p.m.G;
            const int lim = t * 32 + r < nrows ? visible(p.m, u.s, token) - key0 - 4 * h : 0;
            if (__ballot(lim > 0) == 0) continue;
            const char* q = p.q + (int64_t)(u.s.first + token) * p.q_T + (int64_t)head * p.q_H;
            float g = p.lse[(int64_t)(u.s.first + token) * p.l_T + (int64_t)head * p.l_H] * p.lmul;
            if (g == -INFINITY) g = INFINITY;      // a row that saw nothing anywhere gives nothing
            f32x16 s;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const int c = 2 * k + h;
                u32x4 b = {0, 0, 0, 0};
                if (c * 8 < p.Dk) b = *(const u32x4*)(q + c * 16);
                s = Mat<E>::mma(kf[k], b, s);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = exp2_fast(__builtin_fmaf(s[i], p.c, -g));
                acc[i] += 8 * (i / 4) + i % 4 < lim ? x : 0.0f;
            }
        }
        // totals over the 32 query lanes; lane r = 0 of each half writes
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) acc[i] += __shfl_xor(acc[i], d, 64);
        }
        float mine = acc[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mine = (r & 15) == i ? acc[i] : mine;
        if (r < 16) {
            const int place = 8 * (r / 4) + r % 4 + 4 * h, k = key0 + place;
            if (parts > 1) {
                p.ws[(((int64_t)u.slot * p.m.Hkv + hk) * parts + part) * kKeys + wave * 32 + place] = mine;
            } else if (k < u.s.kv) {
                float* m = mass_at(p, u.b, hk, k);
                if (m != nullptr) *m += mine;
            }
        }
    }
}

__global__ __launch_bounds__(128) void mass_join(MassArgs p) {
    const int parts = row_parts(p.m, p.target);
    if (parts == 1) return;
    for (uint32_t id = blockIdx.x;; id += gridDim.x) {
        const Step u = find_step(p.m, (int)(id / (uint32_t)p.m.Hkv));
        if (!u.ok) return;
        const int hk = (int)(id % (uint32_t)p.m.Hkv), key = u.step * kKeys + (int)threadIdx.x;
        if (key >= u.s.kv) continue;
        float* m = mass_at(p, u.b, hk, key);
        if (m == nullptr) continue;
        const float* w = p.ws + ((int64_t)u.slot * p.m.Hkv + hk) * parts * kKeys + threadIdx.x;
        float sum = 0.0f;
        for (int i = 0; i < parts; ++i) sum += w[(int64_t)i * kKeys];
        *m += sum;
    }
}

}  // namespace

MassPlan plan_mass(const Batch& m) {
    MassPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    // with few rows to a sequence the keys alone fill the chip, or nothing does
    const int target = 1024 / m.Hkv;
    pl.target = rows <= (int64_t)128 * m.B || target < 2 ? 0 : target;
    pl.units = 2048;
    // parts > 1 only while steps * parts <= target
    pl.ws_bytes = pl.target == 0 ? 0 : (int64_t)pl.target * m.Hkv * kKeys * 4;
    return pl;
}

namespace {
template <typename E, bool KV8> hipError_t run(const MassArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.units), block(256);
    const hipError_t e = a.Dk <= 64    ? launch(mass_kernel<E, KV8, 64>, grid, block, stream, a)
                         : a.Dk <= 128 ? launch(mass_kernel<E, KV8, 128>, grid, block, stream, a)
                         : a.Dk <= 256 ? launch(mass_kernel<E, KV8, 256>, grid, block, stream, a)
                                       : launch(mass_kernel<E, KV8, 576>, grid, block, stream, a);
    if (e != hipSuccess || a.target == 0) return e;
    return launch(mass_join, dim3(1024), dim3(128), stream, a);
}
}  // namespace

hipError_t launch_mass(const MassArgs& a, bool bf16, bool kv8, hipStream_t stream) {
    if (bf16) return kv8 ? run<BF16T, true>(a, stream) : run<BF16T, false>(a, stream);
    return kv8 ? run<F16T, true>(a, stream) : run<F16T, false>(a, stream);
}

}  // namespace dcpa
