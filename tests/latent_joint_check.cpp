// dcpa_latent_attn on the host alone, as latent_launch_check.cpp has the calls that it is made of: random arguments of
// the expansion and of the attention over it, valid and not; a refused call launches nothing, an accepted one stays within
// the limits of a launch, and the workspace query's size is enough, a byte less refused.  Nothing here touches a
// GPU: the HIP entry points are these recorders.
//
//     latent_joint_check <calls> <seed>  ->  "ok calls accepted launches largest_grid"
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
    ++launches;
    if (grid.x > largest) largest = grid.x;
    if (kernel == nullptr || args == nullptr || args[0] == nullptr || grid.x < 1 || grid.y != 1 || grid.z != 1 ||
        (int64_t)grid.x * block.x > (int64_t(1) << 31) || block.x < 64 || block.x > 1024 || block.x % 64 != 0)
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
// (the arguments may be anything: their own products wrap)
static int64_t mul(int64_t a, int64_t b) { return (int64_t)((uint64_t)a * (uint64_t)b); }
static int64_t add(int64_t a, int64_t b) { return (int64_t)((uint64_t)a + (uint64_t)b); }
static int64_t odd(int64_t n) { return upto(150) == 0 ? (int64_t)rng() : n; }
static double scale() {
    const double odd[] = {0.0, -1.0, 1e300, 1e-300, 3e38, 1e-40, 1.0 / 1e-308};
    return upto(20) == 0 ? odd[upto(6)] : 1.0 / (double)(int64_t(1) << upto(30));
}

int main(int argc, char** argv) {
    const int64_t calls = argc > 1 ? atoll(argv[1]) : 1000;
    rng.seed(argc > 2 ? (uint64_t)atoll(argv[2]) : 1);
    void* const at = (void*)(uintptr_t)0x100000;        // never followed
    int64_t accepted = 0;
    for (int64_t i = 0; i < calls && !bad; ++i) {
        const bool wide = upto(3) == 0;
        dcpa_expand_args e{};
        e.B = size(wide ? 18 : 5); e.H = size(wide ? 14 : 6); e.Dn = 8 * size(4); e.Dr = upto(1) ? 8 * size(3) : 0; e.Dv = 8 * size(5); e.Dc = 8 * size(6);
        e.max_keys = upto(30) == 0 ? 0 : size(wide ? 28 : 13); e.num_pages = size(wide ? 31 : 14); e.page_size = size(wide ? 20 : 7); e.max_pages = size(wide ? 24 : 10);
        e.cache = e.w_k = e.w_v = at; e.k = e.v = at; e.block_table = e.kv_len = (const int32_t*)at; e.places = upto(30) ? (int32_t*)at : nullptr;
        if (upto(1)) e.k_rest = e.v_rest = at;
        if (upto(60) == 0) e.v_rest = nullptr;
        e.c_S = add(e.Dc, e.Dr); e.c_P = mul(e.page_size, e.c_S); e.t_B = e.max_pages; e.p_B = odd(e.max_keys);
        e.wk_N = e.wv_N = e.Dc; e.wk_H = mul(e.Dn, e.wk_N); e.wv_H = mul(e.Dv, e.wv_N);
        e.k_H = add(e.Dn, e.Dr); e.v_H = e.vr_H = e.Dv; e.kr_H = e.Dn;
        e.k_S = odd(mul(e.H, e.k_H)); e.v_S = mul(e.H, e.v_H); e.kr_S = mul(e.H, e.kr_H); e.vr_S = odd(mul(e.H, e.vr_H));
        e.k_B = mul(e.max_keys, e.k_S); e.v_B = odd(mul(e.max_keys, e.v_S)); e.kr_B = odd(mul(e.max_keys, e.kr_S)); e.vr_B = mul(e.max_keys, e.vr_S);
        e.dtype = 1 + upto(1); e.cache_dtype = upto(2) ? e.dtype : DCP_FP8_E4M3; e.k_scale = scale();
        dcpa_attn_args a{};
        a.B = upto(60) ? e.B : size(5); a.T = upto(20) == 0 ? 0 : upto(2) ? mul(e.B, size(wide ? 12 : 6)) : size(wide ? 30 : 12);
        a.Hq = mul(e.H, upto(3) ? 1 : size(3));
        a.q = at; a.out = at; a.lse = (float*)at; a.cu_q = a.seq_len = (const int32_t*)at;
        a.q_H = add(e.Dn, e.Dr); a.q_T = odd(mul(a.Hq, a.q_H)); a.o_H = e.Dv; a.o_T = mul(a.Hq, a.o_H); a.l_T = a.Hq; a.l_H = 1;
        a.N = 1 + upto(7); a.rank = upto(a.N - 1); a.interleave = size(6); a.causal = upto(1);
        a.dtype = upto(60) ? e.dtype : 1 + upto(1); a.lse_base = upto(1); a.wide_weights = upto(1); a.scale = scale();
        const int64_t ws = dcpa_latent_attn_workspace(&e, &a);
        if (ws > (int64_t(1) << 50)) bad = true;
        a.workspace = at; a.workspace_bytes = ws;
        auto call = [&] {
            const int64_t before = launches;
            const int st = dcpa_latent_attn(&e, &a, nullptr);
            if (st != DCP_OK && launches != before) bad = true;       // refused, but something was launched
            return st;
        };
        if (ws > 0) {
            a.workspace_bytes = ws - 1;
            if (call() == DCP_OK) bad = true;
            a.workspace_bytes = ws;
        }
        const int st = call();
        if (ws < 0 && st == DCP_OK) bad = true;   // (the query refuses what the call refuses)
        accepted += st == DCP_OK;
    }
    if (bad) {
        printf("launch outside the limits, of a refused call, or a workspace that does not bind\n");
        return 1;
    }
    printf("ok %lld %lld %lld %lld\n", (long long)calls, (long long)accepted, (long long)launches, (long long)largest);
    return 0;
}
