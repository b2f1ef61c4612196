// attn_plan.hip -- a step's lengths, page tables and cache slots from the
// numbers of new tokens of its sequences.
//
// plan_lengths: one workgroup, a thread to a sequence, prefix sums over the
// batch for first rows, new pages and pages given back; then a thread to a page
// that moves, which finds its sequence by halving in LDS.  Everything that a
// sequence reads of its old lengths is read before the same thread writes the
// new ones, so these may lie in the same place.
// plan_tokens: a thread to a token row.  Up to 4096 rows are done by plan_lengths
// itself, and up to four tokens to a sequence by the sequence's own thread, which has
// all they need but a page.
//
// Bound by latency: dependent loads (lengths, free list, table), barriers between
// any two, and code that is run once and fetched as it runs.  256 sequences of one
// token, some ending: 16 us a call, most of it the caller's; 24 prompt chunks with
// 32000 tokens 18 us, of which plan_tokens takes 4.
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
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    __syncthreads();                    // (the last call's sums have been read)
    if (lane == 63) wave_s[wave] = x;
    __syncthreads();
    // (a lane to a wave: a loop over them all is five times the code, and code that is run once waits to be fetched)
    const int to = scan_upto(lane < kWaves ? wave_s[lane] : 0, most);
    all = __builtin_amdgcn_readlane(to, kWaves - 1);
    return wave > 0 ? add_to(__builtin_amdgcn_readlane(to, wave - 1), x, most) : x;
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

// The slot of position pos of a sequence that had L positions, `before` of its keys cached here, or -1.
// page_at(i): entry i of its table row.
template <typename F> __device__ __forceinline__ int64_t slot_of(const PlanArgs& p, int pos, int L, int before, F&& page_at) {
    const uint32_t full = fdiv((uint32_t)pos, p.fblock);
    const int rest = (int)((uint32_t)pos - full * p.fblock.d) - p.rank * p.inter;
    if (rest < 0 || rest >= p.inter) return -1;
    const uint32_t j = (uint32_t)(before + (int)(full * (uint32_t)p.inter) + rest - owned(p, L)), at = fdiv(j, p.fpage);
    if (at >= (uint32_t)p.width) return -1;
    const int page = page_at((int)at);
    return page < 0 ? -1 : (int64_t)page * p.page_size + (int)(j - at * p.fpage.d);
}
__device__ __forceinline__ void write_row(const PlanArgs& p, int t, int pos, int seq, int64_t slot) {
    p.positions[t] = pos;
    p.sequence[t] = seq;
    p.slots[t] = slot;
}
// Row t of the step: sequence b, whose rows are [first, end); b == B: padding.
__device__ __forceinline__ void write_token(const PlanArgs& p, int t, int b, int first, int end) {
    if (b >= p.B) {
        write_row(p, t, -1, -1, -1);
        return;
    }
    const int n = end - first, L = p.seq_out[b] - n, before = p.kv_out[b] - (owned(p, L + n) - owned(p, L)), pos = L + t - first;
    const int32_t* row = p.table + (int64_t)b * p.t_B;
    write_row(p, t, pos, b, slot_of(p, pos, L, before, [&](int i) { return row[i]; }));
}

__global__ __launch_bounds__(kThreads) void plan_lengths(PlanArgs p) {
    constexpr int EACH = 8;             // pages of a thread that are given back at a time
    constexpr int FEW = 4;              // new tokens and pages up to which a sequence's thread writes them itself
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
    auto sequence_of = [&](int k) { return find_end(min(p.B, kThreads), k, [&](int i) { return ends_s[i]; }); };
    load(0);
    bool any = ended;
    for (int b = tid + kThreads; b < p.B; b += kThreads) any |= p.new_len[b] < 0;
    int count = min(max(p.count[0], 0), p.free_max);
    // the page that the sequence's first new key goes to, if it has it already (few sequences: asked for ahead of all else)
    const bool one = p.B <= kThreads && p.T <= p.rows_here;
    int last = -1;
    if (one && n > 0) {
        const uint32_t at = fdiv((uint32_t)m, p.fpage);
        if (at < (uint32_t)p.width && at * p.fpage.d < (uint32_t)m) last = p.table[(int64_t)tid * p.t_B + at];
    }

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
            for (int k0 = 0; k0 < total; k0 += kThreads * EACH) {
                int page[EACH];
                bool gap = false;
#pragma unroll
                for (int e = 0; e < EACH; ++e) {
                    const int k = k0 + e * kThreads + tid;
                    page[e] = -1;
                    if (k < total) {
                        const int i = sequence_of(k);
                        page[e] = p.table[(int64_t)(b0 + i) * p.t_B + first_s[i] + (k - (i > 0 ? ends_s[i - 1] : 0))];
                        gap |= page[e] < 0;
                    }
                }
                // (entries without a page leave no gaps in the list)
                const bool gaps = __syncthreads_or(gap) != 0;
#pragma unroll 1
                for (int e = 0; e < EACH; ++e) {
                    int pg = -1;
#pragma unroll
                    for (int i = 0; i < EACH; ++i) pg = i == e ? page[i] : pg;
                    // (unsigned: places behind a full list of nearly 2^31 pages pass 2^31)
                    uint32_t at = (uint32_t)count + (uint32_t)tid;
                    int pushed = min(max(total - k0 - e * kThreads, 0), kThreads);
                    if (gaps) at = (uint32_t)count + (uint32_t)(scan_block(pg >= 0 ? 1 : 0, kMost, pushed, wave_s) - 1);
                    if (pg >= 0 && at < (uint32_t)p.free_max) p.free[at] = pg;
                    count = add_to(count, pushed, p.free_max);
                }
            }
            __syncthreads();
        }
        if (p.B > kThreads) load(0);
    }

    int rows = 0, taken = 0;
    bool done = false;                   // the token rows are written
    if (tid == 0) p.cu[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        if (b0 > 0) load(b0);
        int all, pages;
        // tokens that find no row are not taken
        const int end = add_to(rows, scan_block(n, p.T, all, wave_s), p.T);
        rows_s[tid] = end;
        __syncthreads();
        const int first = tid > 0 ? rows_s[tid - 1] : rows;
        n = end - first;
        rows = add_to(rows, all, p.T);
        const int kv = m + owned(p, L + n) - owned(p, L), held = pages_for(p, m);
        const int need = ended || b0 + tid >= p.B ? 0 : max(pages_for(p, kv) - held, 0);
        const int incl = scan_block(need, kMost, pages, wave_s);
        if (b0 + tid < p.B) {
            p.cu[b0 + tid + 1] = end;
            p.seq_out[b0 + tid] = ended ? 0 : L + n;
            p.kv_out[b0 + tid] = ended ? 0 : kv;
        }
        // (the barriers of the scan stand between what was given back and what is taken)
        if (one && __syncthreads_or(n > FEW || need > FEW) == 0) {
            int got[FEW];
            int32_t* row = p.table + (int64_t)tid * p.t_B;
#pragma unroll
            for (int i = 0; i < FEW; ++i) {
                const int from = count - 1 - (incl - need + i);
                got[i] = i < need && from >= 0 ? p.free[from] : -1;
            }
#pragma unroll
            for (int i = 0; i < FEW; ++i)
                if (i < need) row[held + i] = got[i];
#pragma unroll
            for (int i = 0; i < FEW; ++i)
                if (i < n)
                    write_row(p, first + i, L + i, tid, slot_of(p, L + i, L, m, [&](int at) {
                                  int page = last;
#pragma unroll
                                  for (int e = 0; e < FEW; ++e) page = at == held + e ? got[e] : page;
                                  return page;
                              }));
            for (int t = rows + tid; t < p.T; t += kThreads) write_row(p, t, -1, -1, -1);
            done = true;
        } else {
            ends_s[tid] = incl;
            first_s[tid] = held;
            __syncthreads();
            for (int k = tid; k < pages; k += kThreads) {
                const int i = sequence_of(k);
                const int from = count - 1 - add_to(taken, k, kMost);
                p.table[(int64_t)(b0 + i) * p.t_B + first_s[i] + (k - (i > 0 ? ends_s[i - 1] : 0))] = from >= 0 ? p.free[from] : -1;
            }
        }
        taken = add_to(taken, pages, kMost);
        __syncthreads();
    }
    if (tid == 0) p.count_out[0] = count - taken;
    if (p.B == 0)
        for (int t = tid; t < p.T; t += kThreads) write_row(p, t, -1, -1, -1);
    if (done || p.B == 0 || p.T > p.rows_here) return;
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
    // (1024 rows more in the one workgroup take 1.2 us, a second launch 4.  Counted with
    // the caller's time, which hides some of the workgroup's, a call gains up to 2 us
    // between 4096 and some 10000 rows if they stay here; one in a graph loses as much.)
    a.rows_here = 4096;
    const hipError_t e = launch(plan_lengths, dim3(1), dim3(kThreads), stream, a);
    if (e != hipSuccess || a.T <= a.rows_here) return e;
    return launch(plan_tokens, dim3((uint32_t)(((int64_t)a.T + 255) / 256)), dim3(256), stream, a);
}

}  // namespace dcpa
