// attn.hip -- attention of new tokens over a rank's paged cache, with the
// partial output and log-sum-exp that the merge takes.
//
// attn_rows: 128 query rows of a key head to a workgroup (attn_rows.hpp).
// attn_keys: up to 32 rows, the keys shared out over the waves (attn_keys.hpp).
// attn_join: joins the key ranges of one row tile that went to different
// workgroups.
#include "attn_join.hpp"
#include "attn_keys.hpp"
#include "attn_rows.hpp"

namespace dcpa {

namespace {

template <typename E, bool KV8, bool EXACT, int DK, int DV, int KT, bool WIDE>
__global__ __launch_bounds__(256, DK > 192 ? 1 : 2) void attn_rows(AttnArgs p) {
    __shared__ RowsLds<DK, DV, KT> lds;
    rows_of<E, KV8, EXACT, DK, DV, KT, WIDE>(p, lds);
}

template <typename E, bool KV8, int DK, int DV>
__global__ __launch_bounds__(256, DK > 128 ? 1 : 2) void attn_keys(AttnArgs p) {
    __shared__ KeysLds<KV8, DK, DV> lds;
    int hk, unit;
    heads_together(p.m, hk, unit);
    if (unit >= p.units) return;
    keys_of<E, KV8, DK, DV>(p, lds, unit_of<128>(p, 32, unit), hk, unit);
}

// ---------------------------------------------------------------------------
// attn_join: the rows of sequences whose keys were split; each lane holds four
// columns (eight where the rows are wide).  Few rows have many parts: the four
// waves of a workgroup share a row's (TOGETHER).  Many rows have few: a wave goes
// from row to row, and works out the lengths once.  Bound by latency: eight parts
// under way at once (7 rows of 155 parts: 9 us, 54 us one part after the other by
// one wave; 2048 rows by a wave each 8 us, by a workgroup each 14 us).  Where the
// lengths turn out even nothing was split, and nothing is joined.
// ---------------------------------------------------------------------------
template <typename E, int STEP, int NC, bool TOGETHER>
__global__ __launch_bounds__(256) void attn_join(AttnArgs p) {
    __shared__ f32x4 share[TOGETHER ? 4 : 1][NC][64];
    const int lane = threadIdx.x & 63, wave = (int)dcp::wave_id();
    int longest;
    const int chunk = key_chunk<STEP>(p.m, p.rows, p.slots, p.share, longest);
    if (__ballot(longest > chunk) == 0) return;       // nothing was split
    // lengths and units of sequences b0 .. b0 + 63, a lane to each
    struct Line {
        Seq s;
        int splits, incl;
    };
    auto line_at = [&](int b0, int base) {
        Line x{};
        int tiles = 0;
        if (b0 + lane < p.m.B) {
            x.s = load_seq(p.m, b0 + lane);
            tiles = (x.s.n * p.m.G + p.rows - 1) / p.rows;
        }
        x.splits = max(1, (x.s.kv + chunk - 1) / chunk);
        x.incl = base + scan_incl(tiles * x.splits);
        return x;
    };
    const Line start = line_at(0, 0);
    const int64_t all = (int64_t)p.m.T * p.m.G * p.m.Hkv;
    const int64_t stride = TOGETHER ? gridDim.x : (int64_t)gridDim.x * 4;
#pragma unroll 1
    for (int64_t id = TOGETHER ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave; id < all; id += stride) {
        const uint32_t at_row = fdiv((uint32_t)id, p.m.fHkv);
        const int hk = (int)((uint32_t)id - at_row * p.m.fHkv.d), t = (int)fdiv(at_row, p.m.fG), head = (int)at_row - t * p.m.G;
        Line x = start;
        uint64_t found = 0;
        for (int b0 = 0;; b0 += 64, x = line_at(b0, __builtin_amdgcn_readlane(x.incl, 63))) {
            found = __ballot(t >= x.s.first && t < x.s.first + x.s.n);
            if (found != 0 || b0 + 64 >= p.m.B) break;
        }
        if (found == 0) continue;
        const int at = __builtin_ctzll(found);
        const Seq s = seq_of(x.s, at);
        const int ns = __builtin_amdgcn_readlane(x.splits, at);
        if (ns == 1) continue;                // written whole
        const int row = (t - s.first) * p.m.G + head, tile = row / p.rows, in_tile = row - tile * p.rows;
        // (a sequence's last tile comes first)
        const int slot = __builtin_amdgcn_readlane(x.incl, at) - (tile + 1) * ns;
        if (slot < 0) continue;
        // the ranges that the tile's last row has keys in
        const int last = min((tile + 1) * p.rows, s.n * p.m.G) - 1;
        const int kend = visible(p.m, s, (int)fdiv((uint32_t)last, p.m.fG));
        const int parts = min(max(1, (kend + chunk - 1) / chunk), p.units - slot);
        const int64_t first = ((int64_t)hk * p.units + slot) * p.rows + in_tile;
        join_parts<E, NC, TOGETHER>(p, share, t, hk * p.m.G + head, parts, [&](int k) { return first + (int64_t)k * p.rows; });
    }
}

}  // namespace

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
AttnPlan plan_attn(const Batch& m, int Dk, int Dv, bool pieces) {
    AttnPlan pl;
    const int64_t rows = (int64_t)m.T * m.G;
    pl.latent = Dk > 256 || Dv > 256;
    // few rows a sequence: 32-row tiles whose waves share out the keys
    pl.by_keys = !pl.latent && pieces && rows <= (int64_t)32 * m.B;
    pl.rows = pl.by_keys ? 32 : 128;
    // row tiles, at most: a tile holds rows of one sequence
    const int64_t most = rows / pl.rows + m.B, each = (int64_t)m.T * ((m.G + pl.rows - 1) / pl.rows);
    pl.tiles = (int32_t)(most < each ? most : each);
    // Workgroups that run at once: one latent workgroup to a CU, two of the others.  Fewer row
    // tiles than that: the keys are split so that the units fill the chip once; decode of ragged
    // batches (few rows, a few tokens to a sequence of latent ones) up to four times over (see
    // fill_slots()).
    const int64_t busy = (int64_t)pl.tiles * m.Hkv;
    const int64_t chip = pl.latent ? 256 : pl.by_keys ? 1024 : 512;
    pl.slots = pl.share = (int32_t)((chip + m.Hkv - 1) / m.Hkv);
    const bool decode = pl.by_keys || (pl.latent && m.T <= (int64_t)8 * m.B);
    if (decode) fill_slots(pl.tiles, pl.slots, pl.share);
    if (busy >= (decode ? 4 * chip : chip)) pl.slots = 0;
    pl.units = pl.slots > pl.tiles ? pl.slots : pl.tiles;
    pl.ws_bytes = pl.slots == 0 ? 0 : (int64_t)pl.units * m.Hkv * pl.rows * (Dv + 1) * 4;
    return pl;
}

namespace {

template <typename E, int STEP>
hipError_t run_join(const AttnArgs& a, hipStream_t stream) {
    // a workgroup to a row up to what the chip holds at once, then a wave, and no more waves than that
    const int64_t rows = (int64_t)a.m.T * a.m.G * a.m.Hkv;
    const dim3 block(256);
    if (rows <= 1024) {
        const dim3 grid((uint32_t)rows);
        return a.Dv <= 256 ? launch(attn_join<E, STEP, 1, true>, grid, block, stream, a)
                           : launch(attn_join<E, STEP, 2, true>, grid, block, stream, a);
    }
    const dim3 grid((uint32_t)(rows < 8192 ? (rows + 3) / 4 : 2048));
    return a.Dv <= 256 ? launch(attn_join<E, STEP, 1, false>, grid, block, stream, a)
                       : launch(attn_join<E, STEP, 2, false>, grid, block, stream, a);
}

template <typename E, bool KV8, bool WIDE>
hipError_t run_rows(const AttnArgs& a, const AttnPlan& pl, dim3 grid, dim3 block, hipStream_t stream) {
    // (whole rows need no test of columns)
    const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
    hipError_t e;
    if (d <= 64)
        e = a.Dk == 64 && a.Dv == 64 ? launch(attn_rows<E, KV8, true, 64, 64, 64, WIDE>, grid, block, stream, a)
                                     : launch(attn_rows<E, KV8, false, 64, 64, 64, WIDE>, grid, block, stream, a);
    else if (d <= 128)
        e = a.Dk == 128 && a.Dv == 128 ? launch(attn_rows<E, KV8, true, 128, 128, 64, WIDE>, grid, block, stream, a)
                                       : launch(attn_rows<E, KV8, false, 128, 128, 64, WIDE>, grid, block, stream, a);
    else {
        e = a.Dk <= 192 && a.Dv <= 128   ? launch(attn_rows<E, KV8, false, 192, 128, 32, WIDE>, grid, block, stream, a)
            : a.Dk <= 192 && a.Dv <= 192 ? launch(attn_rows<E, KV8, false, 192, 192, 32, WIDE>, grid, block, stream, a)
                                         : launch(attn_rows<E, KV8, false, 256, 256, 32, WIDE>, grid, block, stream, a);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 32>(a, stream);
    }
    if (e != hipSuccess || pl.slots == 0) return e;
    return run_join<E, 64>(a, stream);
}

template <typename E, bool KV8>
hipError_t run(const AttnArgs& a, const AttnPlan& pl, bool wide, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)pl.units * a.m.Hkv)), block(256);
    hipError_t e;
    if (pl.by_keys) {
        const int d = a.Dk > a.Dv ? a.Dk : a.Dv;
        const dim3 near((uint32_t)((int64_t)(pl.units + 7) / 8 * 8 * a.m.Hkv));      // (see heads_together())
        e = d <= 64    ? launch(attn_keys<E, KV8, 64, 64>, near, block, stream, a)
            : d <= 128 ? launch(attn_keys<E, KV8, 128, 128>, near, block, stream, a)
                       : launch(attn_keys<E, KV8, 256, 256>, near, block, stream, a);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 128>(a, stream);
    }
    if (pl.latent) {
        e = launch_latent(a, grid, std::is_same_v<E, BF16T>, KV8, wide, stream);
        if (e != hipSuccess || pl.slots == 0) return e;
        return run_join<E, 32>(a, stream);
    }
    return wide ? run_rows<E, KV8, true>(a, pl, grid, block, stream) : run_rows<E, KV8, false>(a, pl, grid, block, stream);
}

}  // namespace

hipError_t join_rows(const AttnArgs& a, int step, bool bf16, hipStream_t stream) {
    if (step == 32) return bf16 ? run_join<BF16T, 32>(a, stream) : run_join<F16T, 32>(a, stream);
    return bf16 ? run_join<BF16T, 64>(a, stream) : run_join<F16T, 64>(a, stream);
}

hipError_t launch_attn(const AttnArgs& arg, const AttnPlan& pl, bool bf16, bool kv8, bool wide, hipStream_t stream) {
    AttnArgs a = arg;
    if (!pl.latent && a.v == nullptr) {        // narrow rows: the values are read as columns of their own
        a.v = a.k;
        a.v_P = a.k_P; a.v_S = a.k_S; a.v_H = a.k_H;
    }
    if (bf16) return kv8 ? run<BF16T, true>(a, pl, wide, stream) : run<BF16T, false>(a, pl, wide, stream);
    return kv8 ? run<F16T, true>(a, pl, wide, stream) : run<F16T, false>(a, pl, wide, stream);
}

}  // namespace dcpa
