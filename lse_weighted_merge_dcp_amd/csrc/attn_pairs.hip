// attn_pairs.hip -- attention over keys and values in two parts: a 16-bit value
// and what its rounding left.
//
// Keys and values that are made for one call (latent_expand) are no cache that
// was rounded before: rounding them would put a score off by 2^-9 of its terms,
// far more than fp32 sums and powers do.  The two parts together hold them to
// 2^-16 (bf16) or 2^-22 (fp16), for 8 more matrix instructions beside 12 in the
// scores of 128 + 64 columns and twice as many in the values.
// Bound by matrix instructions, as rows_of().  A chunk of 3 ragged sequences to 1500
// tokens over 4500 keys, 32 heads of 192 / 128 columns: 535 to 580 us; keys and
// values rounded once 343, with results that are off by more than their own rounding.
#include "attn_rows.hpp"

namespace dcpa {

namespace {

template <typename E, bool EXACT, int DK, int DV, int DR, bool WIDE>
__global__ __launch_bounds__(256, DK > 192 ? 1 : 2) void attn_pairs(PairArgs p) {
    __shared__ PairLds<DK, DV, 32, DR> lds;
    rows_of<E, false, EXACT, DK, DV, 32, WIDE, DR>(p, lds);
}

template <typename E, bool WIDE> hipError_t run(const PairArgs& a, const AttnPlan& pl, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)pl.units * a.m.Hkv)), block(256);
    if (a.Dk <= 128 && a.Dv <= 64 && a.Dr <= 64) return launch(attn_pairs<E, false, 128, 64, 64, WIDE>, grid, block, stream, a);
    if (a.Dk == 192 && a.Dv == 128 && a.Dr == 128) return launch(attn_pairs<E, true, 192, 128, 128, WIDE>, grid, block, stream, a);
    if (a.Dk <= 192 && a.Dv <= 128 && a.Dr <= 128) return launch(attn_pairs<E, false, 192, 128, 128, WIDE>, grid, block, stream, a);
    return launch(attn_pairs<E, false, 256, 256, 256, WIDE>, grid, block, stream, a);
}

}  // namespace

AttnPlan plan_pairs(const Batch& m, int Dv) {
    // as plan_attn() lays out many rows
    AttnPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.latent = pl.by_keys = false;
    pl.rows = 128;
    const int64_t most = rows / pl.rows + m.B, each = (int64_t)m.T * ((m.G + pl.rows - 1) / pl.rows);
    pl.tiles = (int32_t)(most < each ? most : each);
    const int64_t chip = 512;
    pl.slots = pl.share = (int32_t)((chip + m.Hkv - 1) / m.Hkv);
    if ((int64_t)pl.tiles * m.Hkv >= chip) pl.slots = 0;
    pl.units = pl.slots > pl.tiles ? pl.slots : pl.tiles;
    pl.ws_bytes = pl.slots == 0 ? 0 : (int64_t)pl.units * m.Hkv * pl.rows * (Dv + 1) * 4;
    return pl;
}

hipError_t launch_pairs(const PairArgs& a, const AttnPlan& pl, bool bf16, bool asked, hipStream_t stream) {
    // few rows to a sequence: weights in two products, as where their keys are shared out over the waves (attn_keys.hpp)
    const bool wide = asked || (int64_t)a.m.T * a.m.G <= (int64_t)32 * a.m.B;
    const hipError_t e = bf16 ? (wide ? run<BF16T, true>(a, pl, stream) : run<BF16T, false>(a, pl, stream))
                              : (wide ? run<F16T, true>(a, pl, stream) : run<F16T, false>(a, pl, stream));
    if (e != hipSuccess || pl.slots == 0) return e;
    return join_rows(a, 32, bf16, stream);
}

}  // namespace dcpa
