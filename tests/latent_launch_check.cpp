// The calls around shared and latent caches and the batch plan (dcpa_prefix_attn, dcpa_pair_attn, dcpa_project,
// dcpa_latent_expand, dcpa_batch_plan) on the host alone: random arguments, valid and not, from
// tiny to far beyond any memory, through the real checks, plans and launchers
// (compiled for the host only, with an empty device image), and every launch
// checked against the limits.  Nothing here touches a GPU: the HIP entry points
// are these recorders.
//
//     latent_launch_check <calls> <seed>  ->  "ok calls accepted launches largest_grid"
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
        const int64_t Hkv = size(wide ? 16 : 4), Hq = mul(Hkv, size(wide ? 8 : 4)), D = 8 * size(7);
        const int64_t page = size(wide ? 20 : 7), pages = size(wide ? 31 : 14);
        int st;
        switch (upto(4)) {
            case 0: {
                dcpa_project_args a{};
                a.T = add(size(wide ? 30 : 12), wild()); a.H = size(wide ? 16 : 8); a.N = 8 * size(7); a.K = 8 * size(7); a.copy = upto(1) ? 8 * size(5) : 0;
                a.x = a.w = at; a.y = at;
                a.x_H = stride(add(a.K, a.copy)); a.x_T = stride(mul(a.H, a.x_H)); a.y_H = stride(add(a.N, a.copy)); a.y_T = stride(mul(a.H, a.y_H));
                const bool turned = upto(1);
                a.w_N = turned ? 1 : stride(a.K); a.w_K = turned ? stride(a.N) : 1; a.w_H = stride(mul(a.N, a.K));
                a.dtype = 1 + upto(1);
                st = dcpa_project(&a, nullptr);
                break;
            }
            case 1: {
                dcpa_expand_args a{};
                a.B = size(wide ? 20 : 6); a.H = size(wide ? 16 : 7); a.Dn = 8 * size(6); a.Dr = upto(1) ? 8 * size(3) : 0; a.Dv = 8 * size(6); a.Dc = 8 * size(6);
                a.max_keys = add(size(wide ? 30 : 14), wild()); a.num_pages = pages; a.page_size = page; a.max_pages = size(wide ? 30 : 10);
                a.cache = a.w_k = a.w_v = at; a.k = a.v = at; a.block_table = a.kv_len = (const int32_t*)at;
                if (upto(1)) a.k_rest = a.v_rest = at;
                if (upto(1)) a.places = (int32_t*)at;
                a.c_S = stride(add(a.Dc, a.Dr)); a.c_P = stride(mul(page, a.c_S)); a.t_B = a.max_pages; a.p_B = a.max_keys;
                a.wk_N = a.wv_N = stride(a.Dc); a.wk_H = stride(mul(a.Dn, a.wk_N)); a.wv_H = stride(mul(a.Dv, a.wv_N));
                a.k_H = stride(add(a.Dn, a.Dr)); a.v_H = a.vr_H = stride(a.Dv); a.kr_H = stride(a.Dn);
                a.k_S = stride(mul(a.H, a.k_H)); a.v_S = stride(mul(a.H, a.v_H)); a.kr_S = stride(mul(a.H, a.kr_H)); a.vr_S = a.v_S;
                a.k_B = stride(mul(a.max_keys, a.k_S)); a.v_B = stride(mul(a.max_keys, a.v_S)); a.kr_B = stride(mul(a.max_keys, a.kr_S)); a.vr_B = a.v_B;
                a.dtype = 1 + upto(1); a.cache_dtype = upto(2) ? a.dtype : DCP_FP8_E4M3; a.k_scale = scale();
                st = dcpa_latent_expand(&a, nullptr);
                break;
            }
            case 2: {
                static int32_t some[64];
                dcpa_plan_args a{};
                a.B = size(wide ? 20 : 8); a.T = add(size(wide ? 30 : 14), wild()); a.max_pages = size(wide ? 30 : 10); a.page_size = page;
                a.free_max = size(wide ? 31 : 14); a.t_B = upto(20) ? a.max_pages : stride(8);
                a.N = 1 + upto(7); a.rank = upto(a.N - 1); a.interleave = size(6);
                int32_t* const far = (int32_t*)(uintptr_t)(0x100000 + (uintptr_t)(upto(3) == 0 ? 4 * upto(1 << 20) : (uintptr_t)1 << 32));
                a.new_len = (const int32_t*)at; a.seq_len = some; a.kv_len = far; a.seq_out = upto(1) ? some : far + (1 << 26); a.kv_out = far;
                a.block_table = a.free_pages = (int32_t*)at; a.free_count = some; a.free_count_out = some; a.cu_q = a.positions = a.sequence = (int32_t*)at;
                a.slots = (int64_t*)at; a.keep_pages = nullptr;
                st = dcpa_batch_plan(&a, nullptr);
                break;
            }
            default: {
                dcpa_attn_args a{};
                a.B = size(wide ? 20 : 8); a.T = upto(2) ? mul(a.B, size(wide ? 12 : 6)) : add(size(wide ? 30 : 12), wild());
                a.Hq = Hq; a.Hkv = Hkv; a.Dk = D; a.Dv = upto(1) ? D : 8 * size(6);
                const bool two = upto(1);
                a.q = a.k = at; a.v = two || upto(2) ? at : nullptr; a.out = at; a.lse = (float*)at;
                a.q_H = a.k_H = stride(a.Dk); a.v_H = a.o_H = stride(a.Dv);
                a.q_T = stride(mul(a.Hq, a.q_H)); a.o_T = stride(mul(a.Hq, a.o_H)); a.k_S = stride(mul(a.Hkv, a.k_H)); a.v_S = stride(mul(a.Hkv, a.v_H));
                a.k_P = stride(mul(page, a.k_S)); a.v_P = stride(mul(page, a.v_S)); a.l_T = a.Hq; a.l_H = 1;
                a.block_table = a.cu_q = a.kv_len = a.seq_len = (const int32_t*)at;
                a.num_pages = pages; a.page_size = page; a.max_pages = size(wide ? 30 : 10); a.t_B = a.max_pages;
                a.N = 1 + upto(7); a.rank = upto(a.N - 1); a.interleave = size(6); a.causal = upto(1);
                a.dtype = 1 + upto(1); a.cache_dtype = two || upto(2) ? a.dtype : DCP_FP8_E4M3; a.lse_base = upto(1); a.wide_weights = upto(1);
                a.scale = scale(); a.k_scale = scale(); a.v_scale = scale();
                const int64_t groups = size(wide ? 20 : 5), Dr = 8 * (1 + upto(a.Dk > 8 ? a.Dk / 8 - 1 : 0));
                const int64_t ws = two ? dcpa_pair_attn_workspace(&a) : dcpa_prefix_attn_workspace(&a, groups);
                if (ws > (int64_t(1) << 50)) bad = true;
                a.workspace = at; a.workspace_bytes = ws;
                auto call = [&] {
                    return two ? dcpa_pair_attn(&a, at, a.k_P, a.k_S, a.k_H, Dr, at, a.v_P, a.v_S, a.v_H, nullptr)
                               : dcpa_prefix_attn(&a, (const int32_t*)at, (const int32_t*)at, groups, nullptr);
                };
                if (ws > 0) {                            // one byte less is refused, and nothing launched
                    const int64_t before = launches;
                    a.workspace_bytes = ws - 1;
                    st = call();
                    if (st == DCP_OK || launches != before) bad = true;
                    a.workspace_bytes = ws;
                }
                st = call();
                if (ws < 0 && st == DCP_OK) bad = true;   // (the query refuses what the call refuses)
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
