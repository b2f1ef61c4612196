// attn_prefix_rows.hpp -- the kernels of attn_prefix.hip for rows of up to 256
// columns, for one payload type (a file each, which compile side by side).
#pragma once
#include "attn_keys.hpp"
#include "attn_prefix.hpp"
#include "attn_rows.hpp"

namespace dcpa {

namespace {

template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, bool WIDE>
__global__ __launch_bounds__(256, DK > 192 ? 1 : 2) void prefix_rows(GroupArgs p) {
    __shared__ RowsLds<DK, DV, KT> lds;
    rows_of<E, KV8, EXACT, DK, DV, KT, WIDE>(p, lds);
}
// The same where rows are few: a sequence's own keys shared out over the waves, which keeps more loads under
// way.  keys_of() holds every weight in two products, and so do the shared keys here (as attention of each sequence by
// itself would): 64 sequences behind 32768 keys, 64 / 8 heads, 73 us, with one product for the shared keys 69; 48 of four
// tokens over an 8-bit cache 54 and 46.
template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, int DO>
__global__ __launch_bounds__(256, DO > 128 ? 1 : 2) void prefix_few(GroupArgs p) {
    __shared__ union Lds {
        RowsLds<DK, DV, KT> rows;
        KeysLds<KV8, DO, DO> keys;
    } lds;
    const int hk = (int)(blockIdx.x % (uint32_t)p.m.Hkv), unit = (int)(blockIdx.x / (uint32_t)p.m.Hkv);
    const GroupUnit u = unit_of<KT>(p, p.rows, unit);
    if (u.b1 > u.b0) rows_of<E, KV8, EXACT, DK, DV, KT, true>(p, lds.rows);
    else keys_of<E, KV8, DO, DO>(p, lds.keys, u, hk, unit);
}
template <typename E, bool KV8, bool WIDE> hipError_t run(const GroupArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.units * a.m.Hkv)), block(256);
    hipError_t e;
    const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
    const bool few = a.own_rows == 32;
    auto rows = [&](auto exact, auto dk, auto dv, auto kt, auto own) {
        constexpr bool X = decltype(exact)::value;
        constexpr int K = decltype(dk)::value, V = decltype(dv)::value, T = decltype(kt)::value, O = decltype(own)::value;
        // (8-bit rows of 128 columns wait in registers to be widened: with 64 keys to a tile the loop would spill)
        constexpr int TF = KV8 && K == 128 ? 32 : T;
        return few ? launch(prefix_few<E, KV8, X, K, V, TF, O>, grid, block, stream, a)
                   : launch(prefix_rows<E, KV8, X, K, V, T, WIDE>, grid, block, stream, a);
    };
    constexpr std::integral_constant<int, 32> n32{};
    constexpr std::integral_constant<int, 64> n64{};
    constexpr std::integral_constant<int, 128> n128{};
    constexpr std::integral_constant<int, 192> n192{};
    constexpr std::integral_constant<int, 256> n256{};
    if (d <= 64) e = rows(std::false_type{}, n64, n64, n64, n64);
    else if (d <= 128) e = a.Dk == 128 && a.Dv == 128 ? rows(std::true_type{}, n128, n128, n64, n128) : rows(std::false_type{}, n128, n128, n64, n128);
    else e = a.Dk <= 192 && a.Dv <= 128 ? rows(std::false_type{}, n192, n128, n32, n256) : rows(std::false_type{}, n256, n256, n32, n256);
    return e;
}

template <typename E> hipError_t run_rows(const GroupArgs& a, bool kv8, bool wide, hipStream_t stream) {
    if (wide) return kv8 ? run<E, true, true>(a, stream) : run<E, false, true>(a, stream);
    return kv8 ? run<E, true, false>(a, stream) : run<E, false, false>(a, stream);
}

}  // namespace

}  // namespace dcpa
