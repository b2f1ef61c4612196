// attn_latent.hip -- attention in the latent layout (attn_latent.hpp) of a batch
// of single sequences.
#include "attn_latent.hpp"

namespace dcpa {

namespace {

template <typename E, bool KV8, bool EXACT> __global__ __launch_bounds__(256, 1) void attn_latent(AttnArgs p) {
    latent_rows<E, KV8, EXACT, false>(p);
}
template <typename E, bool KV8, bool EXACT> __global__ __launch_bounds__(256, 1) void latent_wide(AttnArgs p) {
    latent_rows<E, KV8, EXACT, true>(p);
}

}  // namespace

hipError_t launch_latent(const AttnArgs& a, dim3 grid, bool bf16, bool kv8, bool wide, hipStream_t stream) {
    const dim3 block(256);
    auto run = [&](auto e, auto k) {
        using E = decltype(e);
        constexpr bool K8 = decltype(k)::value;
        if (wide)
            return a.Dk == latent::DK ? launch(latent_wide<E, K8, true>, grid, block, stream, a)
                              : launch(latent_wide<E, K8, false>, grid, block, stream, a);
        return a.Dk == latent::DK ? launch(attn_latent<E, K8, true>, grid, block, stream, a)
                          : launch(attn_latent<E, K8, false>, grid, block, stream, a);
    };
    if (bf16) return kv8 ? run(BF16T{}, std::true_type{}) : run(BF16T{}, std::false_type{});
    return kv8 ? run(F16T{}, std::true_type{}) : run(F16T{}, std::false_type{});
}

}  // namespace dcpa
