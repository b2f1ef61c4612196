// The C ABI of libdcpattn on the host alone: random arguments, valid and not, from
// tiny to far beyond any memory, through the real checks, plans and launchers
// (compiled for the host only, with an empty device image), and every launch
// checked against the limits.  Nothing here touches a GPU: the HIP entry points
// are these recorders.
//
//     attn_launch_check <calls> <seed>  ->  "ok calls accepted launches largest_grid"
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include <random>

#include "../include/dcpattn.h"

static int64_t launches = 0, largest = 0;
static bool bad = false;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
    static void* handle[1];
    return handle;
}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void**) {}
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipErrorUnknown; }
}
hipError_t hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
    const int64_t items = (int64_t)grid.x * block.x;
    ++launches;
    if (grid.x > largest) largest = grid.x;
    if (kernel == nullptr || args == nullptr || args[0] == nullptr || grid.x < 1 || grid.y != 1 || grid.z != 1 ||
        grid.x > (1u << 25) || items > (int64_t(1) << 31) || block.x < 64 || block.x > 1024 || block.x % 64 != 0)
        bad = true;
    return hipSuccess;
}

static std::mt19937_64 rng;
static int64_t upto(int64_t n) { return (int64_t)(rng() % (uint64_t)(n + 1)); }
// a size around a power of two, spread over the logarithm
static int64_t size(int bits) {
    const int64_t x = (int64_t(1) << upto(bits)) + upto(2) - 1;
    return upto(40) == 0 ? -x : x;
}
static int64_t wild() { return upto(60) == 0 ? (int64_t)rng() : 0; }
// (the arguments may be anything: their own products wrap)
static int64_t mul(int64_t a, int64_t b) { return (int64_t)((uint64_t)a * (uint64_t)b); }
static int64_t add(int64_t a, int64_t b) { return (int64_t)((uint64_t)a + (uint64_t)b); }
static int64_t stride(int64_t n) { return upto(50) == 0 ? (int64_t)rng() : mul(add(n, 7) / 8 * 8, 1 + upto(2)); }
static double scale() {
    const double odd[] = {0.0, -1.0, 1e300, 1e-300, 0.0 / 0.0 * 0.0, 1.0 / 1e-308};
    return upto(30) == 0 ? odd[upto(5)] : 0.1 + 0.01 * (double)upto(100);
}

int main(int argc, char** argv) {
    const int64_t calls = argc > 1 ? atoll(argv[1]) : 1000;
    rng.seed(argc > 2 ? (uint64_t)atoll(argv[2]) : 1);
    void* const at = (void*)(uintptr_t)0x100000;        // never followed
    int64_t accepted = 0;
    for (int64_t i = 0; i < calls && !bad; ++i) {
        const bool wide = upto(3) == 0;
        const int64_t Hkv = size(wide ? 16 : 4), Hq = upto(30) == 0 ? size(17) : mul(Hkv, size(wide ? 8 : 4)), D = 8 * size(7);
        const int64_t page = size(wide ? 20 : 7), pages = size(wide ? 31 : 14);
        int st;
        switch (upto(3)) {
            case 0: {
                dcpa_rope_args a{};
                a.T = add(size(wide ? 30 : 14), wild());
                a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.Dv = upto(1) ? D : 8 * size(7);
                a.q = a.k = at; a.q_out = a.k_cache = a.v_cache = at; a.v = upto(2) ? at : nullptr;
                a.q_H = a.k_H = a.qo_H = a.kc_H = stride(a.D); a.v_H = a.vc_H = stride(a.Dv);
                a.q_T = a.qo_T = stride(mul(a.Hq, a.q_H)); a.k_T = a.kc_S = stride(mul(a.Hkv, a.k_H)); a.v_T = a.vc_S = stride(mul(a.Hkv, a.v_H));
                a.kc_P = stride(mul(page, a.kc_S)); a.vc_P = stride(mul(page, a.vc_S));
                a.q_weight = a.k_weight = at; a.positions = (const int32_t*)at; a.cos_sin = (const float*)at; a.slots = (const int64_t*)at;
                a.rot = upto(2) ? a.D / 16 * 16 : 16 * upto(10); a.cs_P = a.rot; a.q_norm = upto(1) ? a.D : 0; a.k_norm = upto(1) ? a.D : 8 * upto(4);
                a.interleaved = upto(1); a.positions_max = size(31); a.num_pages = pages; a.page_size = page;
                a.dtype = 1 + upto(1); a.cache_dtype = upto(2) ? a.dtype : DCP_FP8_E4M3;
                a.eps = scale(); a.k_scale = scale(); a.v_scale = scale();
                st = dcpa_qk_norm_rope_append(&a, nullptr);
                break;
            }
            case 1:
            case 2: {
                dcpa_attn_args a{};
                a.B = size(wide ? 20 : 8); a.T = upto(2) ? mul(a.B, size(wide ? 12 : 6)) : add(size(wide ? 30 : 12), wild());
                a.Hq = Hq; a.Hkv = Hkv; a.Dk = D; a.Dv = upto(1) ? D : 8 * size(6);
                a.q = a.k = at; a.v = upto(2) ? at : nullptr; a.out = at; a.lse = (float*)at;
                a.q_H = a.k_H = stride(a.Dk); a.v_H = a.o_H = stride(a.Dv);
                a.q_T = stride(mul(a.Hq, a.q_H)); a.o_T = stride(mul(a.Hq, a.o_H)); a.k_S = stride(mul(a.Hkv, a.k_H)); a.v_S = stride(mul(a.Hkv, a.v_H));
                a.k_P = stride(mul(page, a.k_S)); a.v_P = stride(mul(page, a.v_S)); a.l_T = a.Hq; a.l_H = 1;
                a.block_table = a.cu_q = a.kv_len = a.seq_len = (const int32_t*)at;
                a.num_pages = pages; a.page_size = page; a.max_pages = size(wide ? 30 : 10); a.t_B = a.max_pages;
                a.N = 1 + upto(7); a.rank = upto(a.N - 1); a.interleave = size(6); a.causal = upto(1);
                a.dtype = 1 + upto(1); a.cache_dtype = upto(2) ? a.dtype : DCP_FP8_E4M3; a.lse_base = upto(1);
                a.scale = scale(); a.k_scale = scale(); a.v_scale = scale();
                const bool weights = upto(1);
                const int64_t ws = weights ? dcpa_attn_mass_workspace(&a) : dcpa_paged_attn_workspace(&a);
                if (ws > (int64_t(1) << 50)) bad = true;
                a.workspace = at; a.workspace_bytes = ws;
                auto call = [&] { return weights ? dcpa_attn_mass(&a, (float*)at, mul(page, a.Hkv), a.Hkv, 1, nullptr) : dcpa_paged_attn(&a, nullptr); };
                if (ws > 0) {                            // one byte less is refused, and nothing launched
                    const int64_t before = launches;
                    a.workspace_bytes = ws - 1;
                    st = call();
                    if (st == DCP_OK || launches != before) bad = true;
                    a.workspace_bytes = ws;
                }
                st = call();
                if (ws < 0 && st == DCP_OK) bad = true;   // (the query refuses what the call refuses)
                break;
            }
            default: {
                dcpa_evict_args a{};
                a.B = size(wide ? 20 : 8); a.Hkv = Hkv; a.Dk = D; a.Dv = upto(1) ? D : 8 * size(6); a.esize = int64_t(1) << upto(2);
                a.mass = (float*)at; a.k = at; a.v = upto(2) ? at : nullptr; a.block_table = a.kv_len = a.dst_table = (const int32_t*)at;
                a.new_len = a.kept = (int32_t*)at;
                a.m_H = 1; a.m_S = a.Hkv; a.m_P = mul(page, a.Hkv); a.k_H = stride(a.Dk); a.v_H = stride(a.Dv);
                a.k_S = stride(mul(a.Hkv, a.k_H)); a.v_S = stride(mul(a.Hkv, a.v_H)); a.k_P = stride(mul(page, a.k_S)); a.v_P = stride(mul(page, a.v_S));
                a.num_pages = pages; a.page_size = page; a.max_pages = size(wide ? 30 : 10); a.t_B = a.max_pages;
                a.dst_pages = size(wide ? 30 : 10); a.d_B = a.dst_pages;
                a.budget = upto(5) ? 1 + upto(mul(page, a.dst_pages) > 0 ? mul(page, a.dst_pages) - 1 : 0) : size(30);
                a.n_sink = upto(4); a.n_recent = upto(64); a.kp_H = a.budget; a.kp_B = mul(a.budget, a.Hkv);
                st = dcpa_cache_evict(&a, nullptr);
            }
        }
        accepted += st == DCP_OK;
    }
    if (bad) {
        printf("launch outside the limits, or a workspace that does not bind\n");
        return 1;
    }
    printf("ok %lld %lld %lld %lld\n", (long long)calls, (long long)accepted, (long long)launches, (long long)largest);
    return 0;
}
