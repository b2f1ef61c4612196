// attn_evict.hip -- keep the cached keys of highest accumulated weight.
//
// evict_select: one workgroup to a sequence and key head.  The weights are
// read once, as integers in the order of their floats, and held in registers
// (the first 32768 keys; longer caches read the rest again).  The value of the
// last kept key is found 11, 11 and 10 bits at a time by counting in LDS; the
// first 11 bits tell an eighth of a power of two apart, so that the counts of
// ordinary weights spread over enough places, and after it few keys are left.
// (Digits of 8 bits, read again for each, took 100 us for 64 heads of 16384
// keys: all the weights count in a few places there.  Halving by compares and
// barriers alone took 36 us.)  Ties go to the lowest indices, and prefix sums
// over the flags write the list in the order of the keys.  64 heads of 16384
// keys: 23 us, a chain of passes and barriers.
// evict_gather: copies the kept rows and weights to their new places, a group
// of lanes to a row.  Bound by the bytes of the rows: 64 x 4096 rows of 256 + 256
// bytes in 54 us, 5.0 TB/s.  It writes the new lengths too: they
// may lie where the old ones do, which all workgroups of evict_select read.
#include "attn_device.hpp"

namespace dcpa {

namespace {

// Larger is better; NaN above +infinity, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (x != x) return 0xffffffffu;
    return (u & 0x80000000u) != 0 ? ~u : u | 0x80000000u;
}

constexpr int kThreads = 1024, kWaves = kThreads / 64, kHeld = 32;   // kHeld values to a thread
constexpr int kBins = 2048;
static_assert(kBins == 2 * kThreads, "two places to a thread");

__global__ __launch_bounds__(kThreads) void evict_select(EvictArgs p) {
    __shared__ __attribute__((aligned(16))) uint32_t bins[kBins];
    __shared__ int wave_s[kWaves], digit_s, left_s, same_s;
    __shared__ int flags_s[kHeld * kWaves];
    __shared__ int total_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int hk = (int)(blockIdx.x % (uint32_t)p.Hkv), b = (int)(blockIdx.x / (uint32_t)p.Hkv);
    const int L = min(max(p.kv[b], 0), p.max_keys), n = min(L, p.budget);
    int32_t* kept = p.kept + (int64_t)b * p.kp_B + (int64_t)hk * p.kp_H;
    for (int i = n + tid; i < p.budget; i += kThreads) kept[i] = -1;
    if (L <= p.budget) {
        for (int i = tid; i < n; i += kThreads) kept[i] = i;
        return;
    }
    const int32_t* table = p.table + (int64_t)b * p.t_B;
    const int lo = p.sink, hi = L - p.recent;        // keys lo .. hi-1 compete, for `want` places
    const int want = p.budget - p.sink - p.recent;
    // 0 for a key that does not compete (every weight's rank is above 0)
    auto value = [&](int j) -> uint32_t {
        if (j < lo || j >= hi) return 0;
        const uint32_t page = fdiv((uint32_t)j, p.fpage);
        const int id = table[page];
        if ((uint32_t)id >= (uint32_t)p.pages) return rank_of(-INFINITY);
        return rank_of(*((const float*)p.mass + (int64_t)id * p.m_P + (int64_t)(j - (int)(page * p.fpage.d)) * p.m_S +
                         (int64_t)hk * p.m_H));
    };
    // value i of thread tid is key i * kThreads + tid
    const int rounds = (L + kThreads - 1) / kThreads, held = min(rounds, kHeld);
    uint32_t x[kHeld];
    // eight at a time: page numbers, then weights, so that their latencies overlap
    auto load8 = [&](int i0, uint32_t* to) {
        int id[8];
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) id[i] = table[fdiv((uint32_t)min((i0 + i) * kThreads + tid, L - 1), p.fpage)];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = min((i0 + i) * kThreads + tid, L - 1);
            const int place = j - (int)(fdiv((uint32_t)j, p.fpage) * p.fpage.d);
            w[i] = -INFINITY;
            if ((uint32_t)id[i] < (uint32_t)p.pages)
                w[i] = *((const float*)p.mass + (int64_t)id[i] * p.m_P + (int64_t)place * p.m_S + (int64_t)hk * p.m_H);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = (i0 + i) * kThreads + tid;
            to[i] = j >= lo && j < hi ? rank_of(w[i]) : 0;
        }
    };
#pragma unroll
    for (int g = 0; g < kHeld; g += 8) {
#pragma unroll
        for (int i = g; i < g + 8; ++i) x[i] = 0;
        if (g < held) load8(g, x + g);
    }
    // keys above `edge` are kept, and `ties` of those equal to it
    uint32_t edge = 0xffffffffu;
    int ties = 0;
    if (want > 0) {
        uint32_t prefix = 0;
        int left = want, shift = 21;
        bool exact = false;
        for (;;) {
            const uint32_t high = shift == 21 ? 0u : ~0u << (shift == 10 ? 21 : 10);
            const uint32_t mask = shift == 0 ? 1023u : 2047u;
            for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
            __syncthreads();
            auto add = [&](uint32_t v) {
                if (v != 0 && (v & high) == prefix) atomicAdd(&bins[v >> shift & mask], 1u);
            };
#pragma unroll
            for (int g = 0; g < kHeld; g += 8)
                if (g < held)
#pragma unroll
                    for (int i = g; i < g + 8; ++i) add(x[i]);
            for (int i = kHeld; i < rounds; ++i) add(value(i * kThreads + tid));
            __syncthreads();
            // thread t takes the two places 2047 - 2t and 2046 - 2t, the largest values first
            const int top = kBins - 1 - 2 * tid;
            const int c0 = (int)bins[top], c1 = (int)bins[top - 1], incl = scan_incl(c0 + c1);
            if (lane == 63) wave_s[wave] = incl;
            __syncthreads();
            int before = incl - c0 - c1;
            for (int k = 0; k < wave; ++k) before += wave_s[k];
            if (before < left && before + c0 + c1 >= left) {
                const bool first = before + c0 >= left;
                digit_s = first ? top : top - 1;
                left_s = left - before - (first ? 0 : c0);
                same_s = first ? c0 : c1;
            }
            __syncthreads();
            prefix |= (uint32_t)digit_s << shift;
            left = left_s;                    // of the keys of this prefix that are kept
            exact = same_s == left;
            if (exact || shift == 0) break;
            shift = shift == 21 ? 10 : 0;
            __syncthreads();
        }
        // (all keys of the prefix are kept, or the ties of one value are broken below)
        edge = exact ? prefix - 1 : prefix;
        ties = exact ? 0 : left;
    }
    // Exclusive prefix sums of the flags' counts, in the order of the keys; the total.
    auto scan_flags = [&](int entries) -> int {
        __syncthreads();
        if (wave == 0) {
            int carry = 0;
            for (int e0 = 0; e0 < entries; e0 += 64) {
                const int e = e0 + lane, c = e < entries ? flags_s[e] : 0, incl = scan_incl(c);
                if (e < entries) flags_s[e] = carry + incl - c;
                carry += __builtin_amdgcn_readlane(incl, 63);
            }
            if (lane == 0) total_s = carry;
        }
        __syncthreads();
        return total_s;
    };
    const uint64_t below = (1ull << lane) - 1;
    int ties_left = ties, out = 0;
    // (one turn for what is held; further turns for the rest of a longer cache)
    for (int i0 = 0; i0 < rounds; i0 += kHeld) {
        const int end = min(rounds - i0, kHeld);
        if (i0 > 0) {
#pragma unroll
            for (int g = 0; g < kHeld; g += 8)
                if (g < end) load8(i0 + g, x + g);
        }
        uint64_t tied = 0;         // bit i: value i equals the edge and is kept
        __syncthreads();
        if (ties_left > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (i < end) {
                    const uint64_t t = __ballot(x[i] == edge);
                    if (lane == 0) flags_s[i * kWaves + wave] = __popcll(t);
                }
            const int all = scan_flags(end * kWaves);
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (i < end) {
                    const uint64_t t = __ballot(x[i] == edge);
                    const int rank = flags_s[i * kWaves + wave] + __popcll(t & below);
                    if (x[i] == edge && rank < ties_left) tied |= 1ull << i;
                }
            ties_left -= min(ties_left, all);
            __syncthreads();
        }
        auto keeps = [&](int i) {
            const int j = (i0 + i) * kThreads + tid;
            return j < L && (j < lo || j >= hi || x[i] > edge || (tied >> i & 1u) != 0);
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < end) {
                const uint64_t k = __ballot(keeps(i));
                if (lane == 0) flags_s[i * kWaves + wave] = __popcll(k);
            }
        const int all = scan_flags(end * kWaves);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < end) {
                const bool keep = keeps(i);
                const uint64_t k = __ballot(keep);
                const int at = out + flags_s[i * kWaves + wave] + __popcll(k & below);
                if (keep && at < p.budget) kept[at] = (i0 + i) * kThreads + tid;
            }
        out += all;
    }
}

// LPR lanes to a (sequence, kept place, key head), ROWS of them at a time so
// that their loads overlap.  V bytes to a lane and step.
template <int V, int LPR>
__global__ __launch_bounds__(256) void evict_gather(EvictArgs p) {
    constexpr int ROWS = 4, GROUPS = 256 / LPR;
    const int lane = (int)(threadIdx.x % LPR);
    const int64_t first = ((int64_t)blockIdx.x * ROWS) * GROUPS + threadIdx.x / LPR;
    const int64_t rows = (int64_t)p.B * p.budget * p.Hkv;
    const char *ks[ROWS], *vs[ROWS], *ms[ROWS];
    char *kd[ROWS], *vd[ROWS], *md[ROWS];
    bool go[ROWS], have[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        // rows in the order of the destination: place after place, its heads together
        const int64_t row = first + (int64_t)r * GROUPS;
        const uint32_t at = (uint32_t)min(row, rows - 1);
        const uint32_t bi = fdiv(at, p.fHkv), hk = at - bi * p.fHkv.d, b = fdiv(bi, p.fbudget), i = bi - b * p.fbudget.d;
        const int j = p.kept[(int64_t)b * p.kp_B + (int64_t)hk * p.kp_H + i];
        const uint32_t src = (uint32_t)max(j, 0), sp = fdiv(src, p.fpage), dp = fdiv(i, p.fpage);
        const int to = p.dst[(int64_t)b * p.d_B + dp];
        const int from = j >= 0 ? p.table[(int64_t)b * p.t_B + sp] : -1;
        go[r] = row < rows && j >= 0 && (uint32_t)to < (uint32_t)p.pages;
        have[r] = (uint32_t)from < (uint32_t)p.pages;
        const int64_t ss = src - sp * p.fpage.d, ds = i - dp * p.fpage.d;
        ks[r] = p.k + (int64_t)from * p.k_P + ss * p.k_S + (int64_t)hk * p.k_H;
        kd[r] = p.k + (int64_t)to * p.k_P + ds * p.k_S + (int64_t)hk * p.k_H;
        vs[r] = p.v + (int64_t)from * p.v_P + ss * p.v_S + (int64_t)hk * p.v_H;
        vd[r] = p.v + (int64_t)to * p.v_P + ds * p.v_S + (int64_t)hk * p.v_H;
        ms[r] = p.mass + ((int64_t)from * p.m_P + ss * p.m_S + (int64_t)hk * p.m_H) * 4;
        md[r] = p.mass + ((int64_t)to * p.m_P + ds * p.m_S + (int64_t)hk * p.m_H) * 4;
    }
    const int most = max(p.k_bytes, p.v_bytes);
    for (int o = lane * V; o < most; o += LPR * V) {
        dcp::Vec<V> x[ROWS], y[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            x[r] = y[r] = dcp::vzero<V>();
            if (go[r] && have[r] && o < p.k_bytes) x[r] = dcp::vload_stream<V>(ks[r] + o);
            if (go[r] && have[r] && o < p.v_bytes) y[r] = dcp::vload_stream<V>(vs[r] + o);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (go[r] && o < p.k_bytes) dcp::vstore<V>(kd[r] + o, x[r]);
            if (go[r] && o < p.v_bytes) dcp::vstore<V>(vd[r] + o, y[r]);
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (go[r]) *(float*)md[r] = have[r] ? *(const float*)ms[r] : -INFINITY;
        // the lane of a sequence's first row writes its length (nobody else reads the old one here)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t row = first + (int64_t)r * GROUPS;
            const uint32_t at = (uint32_t)min(row, rows - 1), b = fdiv(fdiv(at, p.fHkv), p.fbudget);
            if (row < rows && at == b * p.fbudget.d * p.fHkv.d)
                p.new_len[b] = min(min(max(p.kv[b], 0), p.max_keys), p.budget);
        }
    }
}

template <int V> hipError_t run_gather(const EvictArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.Hkv * a.budget;
    const int steps = ((a.k_bytes > a.v_bytes ? a.k_bytes : a.v_bytes) + V - 1) / V;
    auto grid = [&](int lpr) { return dim3((uint32_t)((rows * lpr + 1023) / 1024)); };
    if (steps <= 8) return launch(evict_gather<V, 8>, grid(8), dim3(256), stream, a);
    if (steps <= 16) return launch(evict_gather<V, 16>, grid(16), dim3(256), stream, a);
    return launch(evict_gather<V, 32>, grid(32), dim3(256), stream, a);
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a, hipStream_t stream) {
    const hipError_t e = launch(evict_select, dim3((uint32_t)(a.B * a.Hkv)), dim3(kThreads), stream, a);
    if (e != hipSuccess) return e;
    return a.wide ? run_gather<16>(a, stream) : run_gather<8>(a, stream);
}

}  // namespace dcpa
