// attn_plan.hip -- a step's lengths, page tables and cache slots from the
// numbers of new tokens of its sequences.
//
// plan_lengths: one workgroup, a thread to a sequence, prefix sums over the
// batch for first rows, new pages and pages given back; then a thread to a page
// that moves, which finds its sequence by halving in LDS.  Everything that a
// sequence reads of its old lengths is read before the same thread writes the
// new ones, so these may lie in the same place.
// plan_tokens: a thread to a token row.  Few rows are done by plan_lengths itself.
//
// Bound by latency: a chain of dependent loads (lengths, free list, table) with
// a barrier between any two.
#include "attn_device.hpp"

namespace dcpa {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMost = 1 << 30;          // lengths, rows and pages stay below it

__device__ __forceinline__ int owned(const PlanArgs& p, int x) {
    const uint32_t u = (uint32_t)x, full = fdiv(u, p.fblock), rest = u - full * p.fblock.d;
    return (int)(full * (uint32_t)p.inter) + min(max((int)rest - p.rank * p.inter, 0), p.inter);
}
__device__ __forceinline__ int pages_for(const PlanArgs& p, int keys) {
    return (int)min(fdiv((uint32_t)keys + (uint32_t)p.page_size - 1u, p.fpage), (uint32_t)p.width);
}

// Inclusive sum over the workgroup; every thread gets the whole in `all`.
__device__ __forceinline__ int scan_block(int x, int most, int& all, int (&wave_s)[kWaves]) {
    x = scan_upto(x, most);
    const int wave = threadIdx.x >> 6;
    __syncthreads();                    // (the last call's sums have been read)
    if ((threadIdx.x & 63) == 63) wave_s[wave] = x;
    __syncthreads();
    all = 0;
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = all;
        all = add_to(all, wave_s[w], most);
    }
    return add_to(before, x, most);
}

// The first i in [0, n) with ends(i) > at (n if there is none; ends do not fall).
template <typename F> __device__ __forceinline__ int find_end(int n, int at, F&& ends) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends(mid) > at) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Row t of the step: sequence b, whose rows are [first, end); b == B: padding.
__device__ __forceinline__ void write_token(const PlanArgs& p, int t, int b, int first, int end) {
    int pos = -1, seq = -1;
    int64_t slot = -1;
    if (b < p.B) {
        const int n = end - first, L = p.seq_out[b] - n, base = owned(p, L);
        const int before = p.kv_out[b] - (owned(p, L + n) - base);
        pos = L + t - first;
        seq = b;
        const uint32_t full = fdiv((uint32_t)pos, p.fblock);
        const int rest = (int)((uint32_t)pos - full * p.fblock.d) - p.rank * p.inter;
        if (rest >= 0 && rest < p.inter) {
            const uint32_t j = (uint32_t)(before + (int)(full * (uint32_t)p.inter) + rest - base), at = fdiv(j, p.fpage);
            if (at < (uint32_t)p.width) {
                const int page = p.table[(int64_t)b * p.t_B + at];
                if (page >= 0) slot = (int64_t)page * p.page_size + (int)(j - at * p.fpage.d);
            }
        }
    }
    p.positions[t] = pos;
    p.sequence[t] = seq;
    p.slots[t] = slot;
}

__global__ __launch_bounds__(kThreads) void plan_lengths(PlanArgs p) {
    __shared__ int wave_s[kWaves];
    __shared__ int ends_s[kThreads], first_s[kThreads], rows_s[kThreads];
    const int tid = threadIdx.x;
    // the batch's 1024 sequences from b0 on, a thread to each
    int n = 0, L = 0, m = 0, keep = 0;
    bool ended = false;
    auto load = [&](int b0) {
        const int b = b0 + tid;
        n = L = m = keep = 0;
        ended = false;
        if (b >= p.B) return;
        n = p.new_len[b];
        L = min(max(p.seq[b], 0), kMost - 1);
        m = min(max(p.kv[b], 0), kMost - 1);
        if (p.keep != nullptr) keep = max(p.keep[b], 0);
        ended = n < 0;
        n = min(max(n, 0), kMost - 1 - L);
    };
    auto sequence_of = [&](int k) { return find_end(kThreads, k, [&](int i) { return ends_s[i]; }); };
    load(0);
    bool any = false;
    for (int b = tid; b < p.B; b += kThreads) any |= (b == tid ? ended : p.new_len[b] < 0);
    int count = min(max(p.count[0], 0), p.free_max);

    // pages of ended sequences, in the order of sequences and pages, onto the list
    if (__syncthreads_or(any) != 0) {
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            if (b0 > 0) load(b0);
            int total;
            const int back = ended ? max(pages_for(p, m) - keep, 0) : 0;
            const int incl = scan_block(back, kMost, total, wave_s);
            ends_s[tid] = incl;
            first_s[tid] = keep;
            __syncthreads();
            for (int k0 = 0; k0 < total; k0 += kThreads) {
                const int k = k0 + tid;
                int page = -1;
                if (k < total) {
                    const int i = sequence_of(k);
                    page = p.table[(int64_t)(b0 + i) * p.t_B + first_s[i] + (k - (i > 0 ? ends_s[i - 1] : 0))];
                }
                int pushed;
                const int at = count + scan_block(page >= 0 ? 1 : 0, kMost, pushed, wave_s) - 1;
                if (page >= 0 && at < p.free_max) p.free[at] = page;
                count = min(count + pushed, p.free_max);
            }
            __syncthreads();
        }
        if (p.B > kThreads) load(0);
    }

    int rows = 0, taken = 0;
    if (tid == 0) p.cu[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        if (b0 > 0) load(b0);
        int all, pages;
        // tokens that find no row are not taken
        const int end = add_to(rows, scan_block(n, p.T, all, wave_s), p.T);
        rows_s[tid] = end;
        __syncthreads();
        n = end - (tid > 0 ? rows_s[tid - 1] : rows);
        rows = add_to(rows, all, p.T);
        const int kv = m + owned(p, L + n) - owned(p, L), held = pages_for(p, m);
        ends_s[tid] = scan_block(ended || b0 + tid >= p.B ? 0 : max(pages_for(p, kv) - held, 0), kMost, pages, wave_s);
        first_s[tid] = held;
        if (b0 + tid < p.B) {
            p.cu[b0 + tid + 1] = end;
            p.seq_out[b0 + tid] = ended ? 0 : L + n;
            p.kv_out[b0 + tid] = ended ? 0 : kv;
        }
        __syncthreads();
        for (int k = tid; k < pages; k += kThreads) {
            const int i = sequence_of(k);
            const int from = count - 1 - add_to(taken, k, kMost);
            p.table[(int64_t)(b0 + i) * p.t_B + first_s[i] + (k - (i > 0 ? ends_s[i - 1] : 0))] = from >= 0 ? p.free[from] : -1;
        }
        taken = add_to(taken, pages, kMost);
        __syncthreads();
    }
    if (tid == 0) p.count_out[0] = count - taken;
    if (p.T > p.rows_here) return;
    __syncthreads();
    for (int t = tid; t < p.T; t += kThreads) {
        const int b = p.B <= kThreads ? find_end(p.B, t, [&](int i) { return rows_s[i]; })
                                      : find_end(p.B, t, [&](int i) { return p.cu[i + 1]; });
        const bool real = b < p.B;
        write_token(p, t, b, real ? p.cu[b] : 0, real ? p.cu[b + 1] : 0);
    }
}

__global__ __launch_bounds__(256) void plan_tokens(PlanArgs p) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= p.T) return;
    const int b = find_end(p.B, (int)t, [&](int i) { return p.cu[i + 1]; });
    const bool real = b < p.B;
    write_token(p, (int)t, b, real ? p.cu[b] : 0, real ? p.cu[b + 1] : 0);
}

}  // namespace

hipError_t launch_plan(const PlanArgs& arg, hipStream_t stream) {
    PlanArgs a = arg;
    a.rows_here = 4096;
    const hipError_t e = launch(plan_lengths, dim3(1), dim3(kThreads), stream, a);
    if (e != hipSuccess || a.T <= a.rows_here) return e;
    return launch(plan_tokens, dim3((uint32_t)(((int64_t)a.T + 255) / 256)), dim3(256), stream, a);
}

}  // namespace dcpa
