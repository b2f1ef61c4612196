// How the attention and weight calls of single tokens are laid out, for the batch sizes and key heads on the
// command line: "B Hkv" pairs, one line each: "attn slots share tiles units ws  weights slots share units ws".
// Host code alone; the HIP entry points below are never called.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include "../lse_weighted_merge_dcp_amd/csrc/attn_launch.hpp"

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
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return hipErrorUnknown; }

namespace dcpa {
hipError_t launch_latent(const AttnArgs&, dim3, bool, bool, bool, hipStream_t) { return hipErrorUnknown; }
}

int main(int argc, char** argv) {
    for (int i = 1; i + 1 < argc; i += 2) {
        dcpa::Batch m{};
        m.B = m.T = atoi(argv[i]);
        m.G = 8;
        m.Hkv = atoi(argv[i + 1]);
        const dcpa::AttnPlan a = dcpa::plan_attn(m, 128, 128, true);
        const dcpa::MassPlan w = dcpa::plan_mass(m, 128, true);
        if (!a.by_keys || !w.few) return 1;
        printf("%d %d %d %d %lld  %d %d %d %lld\n", a.slots, a.share, a.tiles, a.units, (long long)a.ws_bytes, w.slots, w.share, w.units,
               (long long)w.ws_bytes);
    }
    return 0;
}
