// attn_evict.hip -- keep the cached keys of highest accumulated weight.
//
// evict_select: one workgroup to a sequence and key head.  The weights are
// read as integers in the order of their floats, and the budget-th largest is
// found eight bits at a time (four passes, counts in LDS); the ties at that
// value go to the lowest indices, and a prefix sum over the kept flags writes
// the list in the order of the keys.
// evict_gather: copies the kept rows and weights to their new places, a group
// of lanes to a row.
#include "attn_device.hpp"

namespace dcpa {

namespace {

// Larger is better; NaN above +infinity, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (x != x) return 0xffffffffu;
    return (u & 0x80000000u) != 0 ? ~u : u | 0x80000000u;
}

constexpr int kThreads = 1024;

__global__ __launch_bounds__(kThreads) void evict_select(EvictArgs p) {
    __shared__ uint32_t count[256];
    __shared__ uint32_t prefix_s, want_s;
    __shared__ int wave_sum_s[2][kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int hk = (int)(blockIdx.x % (uint32_t)p.Hkv), b = (int)(blockIdx.x / (uint32_t)p.Hkv);
    const int L = min(max(p.kv[b], 0), p.max_keys), n = min(L, p.budget);
    if (hk == 0 && tid == 0) p.new_len[b] = n;
    int32_t* kept = p.kept + (int64_t)b * p.kp_B + (int64_t)hk * p.kp_H;
    for (int i = n + tid; i < p.budget; i += kThreads) kept[i] = -1;
    if (L <= p.budget) {
        for (int i = tid; i < n; i += kThreads) kept[i] = i;
        return;
    }
    const int32_t* table = p.table + (int64_t)b * p.t_B;
    const int lo = p.sink, hi = L - p.recent;        // keys lo .. hi-1 compete
    auto value = [&](int j) -> uint32_t {
        const uint32_t page = fdiv((uint32_t)j, p.fpage);
        const int id = table[page];
        if ((uint32_t)id >= (uint32_t)p.pages) return rank_of(-INFINITY);
        const float* m = (const float*)p.mass + (int64_t)id * p.m_P + (int64_t)(j - (int)(page * p.fpage.d)) * p.m_S +
                         (int64_t)hk * p.m_H;
        return rank_of(*m);
    };
    // the want-th largest of them (want = budget - sink - recent; hi - lo > want)
    if (tid == 0) {
        prefix_s = 0;
        want_s = (uint32_t)(p.budget - p.sink - p.recent);
    }
    uint32_t prefix = 0, want = (uint32_t)(p.budget - p.sink - p.recent);
    const bool any = want > 0;
    for (int shift = 24; any && shift >= 0; shift -= 8) {
        __syncthreads();
        if (tid < 256) count[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
        for (int j = lo + tid; j < hi; j += kThreads) {
            const uint32_t x = value(j);
            if ((x & mask) == prefix) atomicAdd(&count[(x >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t left = want, d = 255;
            while (d > 0 && count[d] < left) left -= count[d--];
            prefix_s = prefix | d << shift;
            want_s = left;
        }
        __syncthreads();
        prefix = prefix_s;
        want = want_s;          // how many keys of exactly this value are kept, from the lowest
    }
    // the list, in order
    int out = 0, ties = 0;
    for (int j0 = 0; j0 < L; j0 += kThreads) {
        const int j = j0 + tid;
        const bool in = j < L;
        const uint32_t x = in && any && j >= lo && j < hi ? value(j) : 0;
        const bool tie = in && any && j >= lo && j < hi && x == prefix;
        const uint64_t tb = __ballot(tie);
        const uint64_t below = (1ull << lane) - 1;
        __syncthreads();
        if (lane == 0) wave_sum_s[0][wave] = __popcll(tb);
        __syncthreads();
        int before = ties, all = 0;
        for (int k = 0; k < kThreads / 64; ++k) {
            if (k < wave) before += wave_sum_s[0][k];
            all += wave_sum_s[0][k];
        }
        before += __popcll(tb & below);
        ties += all;
        const bool keep = in && (j < lo || j >= hi || (any && (x > prefix || (tie && (uint32_t)before < want))));
        const uint64_t kb = __ballot(keep);
        if (lane == 0) wave_sum_s[1][wave] = __popcll(kb);
        __syncthreads();
        int at = out;
        all = 0;
        for (int k = 0; k < kThreads / 64; ++k) {
            if (k < wave) at += wave_sum_s[1][k];
            all += wave_sum_s[1][k];
        }
        at += __popcll(kb & below);
        if (keep && at < p.budget) kept[at] = j;
        out += all;
    }
}

// A wave to each (sequence, key head, kept place).
template <int V>
__global__ __launch_bounds__(256) void evict_gather(EvictArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + dcp::wave_id();
    const int64_t per = (int64_t)p.Hkv * p.budget;
    const int b = (int)(row / per);
    if (b >= p.B) return;
    const int rest = (int)(row - b * per), i = (int)((uint32_t)rest / (uint32_t)p.Hkv), hk = rest - i * p.Hkv;
    const int j = p.kept[(int64_t)b * p.kp_B + (int64_t)hk * p.kp_H + i];
    if (j < 0) return;
    const uint32_t sp = fdiv((uint32_t)j, p.fpage), dp = fdiv((uint32_t)i, p.fpage);
    const int from = p.table[(int64_t)b * p.t_B + sp], to = p.dst[(int64_t)b * p.d_B + dp];
    if ((uint32_t)to >= (uint32_t)p.pages) return;
    const bool have = (uint32_t)from < (uint32_t)p.pages;
    const int64_t ss = j - (int)(sp * p.fpage.d), ds = i - (int)(dp * p.fpage.d);
    const char* ks = p.k + (int64_t)from * p.k_P + ss * p.k_S + (int64_t)hk * p.k_H;
    char* kd = p.k + (int64_t)to * p.k_P + ds * p.k_S + (int64_t)hk * p.k_H;
    for (int o = lane * V; o < p.k_bytes; o += 64 * V)
        dcp::vstore<V>(kd + o, have ? dcp::vload<V>(ks + o) : dcp::vzero<V>());
    if (p.v != nullptr) {
        const char* vs = p.v + (int64_t)from * p.v_P + ss * p.v_S + (int64_t)hk * p.v_H;
        char* vd = p.v + (int64_t)to * p.v_P + ds * p.v_S + (int64_t)hk * p.v_H;
        for (int o = lane * V; o < p.v_bytes; o += 64 * V)
            dcp::vstore<V>(vd + o, have ? dcp::vload<V>(vs + o) : dcp::vzero<V>());
    }
    if (lane == 0) {
        float* m = (float*)p.mass;
        m[(int64_t)to * p.m_P + ds * p.m_S + (int64_t)hk * p.m_H] =
            have ? m[(int64_t)from * p.m_P + ss * p.m_S + (int64_t)hk * p.m_H] : -INFINITY;
    }
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a, hipStream_t stream) {
    const hipError_t e = launch(evict_select, dim3((uint32_t)(a.B * a.Hkv)), dim3(kThreads), stream, a);
    if (e != hipSuccess) return e;
    const dim3 grid((uint32_t)(((int64_t)a.B * a.Hkv * a.budget + 3) / 4));
    return a.wide ? launch(evict_gather<16>, grid, dim3(256), stream, a) : launch(evict_gather<8>, grid, dim3(256), stream, a);
}

}  // namespace dcpa
