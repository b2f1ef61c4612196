// attn_latent.hip -- attention in the latent layout: many query heads share
// one key row of up to 576 columns, whose first Dv <= 512 are its value.
//
// A workgroup takes 128 query rows, a wave 32 of them against tiles of 32 keys
// in LDS; keys and values are the same tile, so a key is fetched once for the
// 2 * (576 + 512) * 128 operations done with it.  A wave's 32 x 512 outputs
// fill the 256 accumulation registers and its queries 132 of the others (three of
// their 36 fragments lie in LDS), so one wave runs on a SIMD and nothing but its own order of instructions hides a
// latency: key and value fragments are read from LDS several products ahead,
// the next tile comes straight into LDS meanwhile.  The products read 70 KB of
// LDS per wave and tile (4 waves: 2176 clocks at 128 bytes a clock), as long as
// their 68 matrix instructions take.  Between those instructions stand the powers
// of the present tile, the maximum of the next, the addresses and the nine
// requests of the one after that.  1024 tokens of 96 heads over 2048 keys a rank:
// 416 us, 1.02 PFLOP/s; 64 sequences of one token, 128 heads: 180 us.
// The weights are rounded to the payload type for the product with the values,
// whose error is then that of the output's own rounding once more.  WIDE: what the
// rounding left takes a second product, 100 matrix instructions to a tile for 68, and the
// two calls above take 532 and 220 us.
//
// The compiler would move outputs between the two halves of the register file
// around every use outside a product, and spill.  So the outputs live in a0 ..
// a255 by name: every instruction that touches them is written in asm here (the
// compiler itself takes no accumulation register in this kernel, which a test
// of the compiled code checks).
#include "attn_common.hpp"

namespace dcpa {

namespace {

// The scores' products, in ordinary registers.  The compiler does not see that
// these are matrix instructions, so the waits it would add stand here: two
// states before the first of a row (a vector instruction may have written an
// operand just before; between two products none writes an operand, which the
// test of the compiled code checks too), and settle() between the last product
// and the first other use (an 8-pass product's result may be read 11 states
// later).
template <typename E> __device__ __forceinline__ void mma_first(f32x16& d, u32x4 a, u32x4 b) {
    if constexpr (std::is_same_v<E, BF16T>)
        asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(d) : "v"(a), "v"(b));
    else
        asm("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(d) : "v"(a), "v"(b));
}
template <typename E> __device__ __forceinline__ void mma_next(f32x16& d, u32x4 a, u32x4 b) {
    if constexpr (std::is_same_v<E, BF16T>)
        asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
    else
        asm("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void settle(f32x16& d) { asm volatile("s_nop 15\n\ts_nop 3" : "+v"(d)); }

// Output block CB (32 columns) is a[16 CB .. 16 CB + 15].
template <typename E, int CB> __device__ __forceinline__ void out_mma(u32x4 a, u32x4 b) {
    if constexpr (std::is_same_v<E, BF16T>)
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]"
                     :: "v"(a), "v"(b), "n"(16 * CB), "n"(16 * CB + 15));
    else
        asm volatile("v_mfma_f32_32x32x16_f16 a[%2:%3], %0, %1, a[%2:%3]"
                     :: "v"(a), "v"(b), "n"(16 * CB), "n"(16 * CB + 15));
}
template <int I> __device__ __forceinline__ void out_scale4(float f) {
    float t0, t1, t2, t3;
    asm volatile("v_accvgpr_read_b32 %0, a[%5]\n\tv_accvgpr_read_b32 %1, a[%6]\n\t"
                 "v_accvgpr_read_b32 %2, a[%7]\n\tv_accvgpr_read_b32 %3, a[%8]\n\t"
                 "v_mul_f32 %0, %0, %4\n\tv_mul_f32 %1, %1, %4\n\tv_mul_f32 %2, %2, %4\n\tv_mul_f32 %3, %3, %4\n\t"
                 "v_accvgpr_write_b32 a[%5], %0\n\tv_accvgpr_write_b32 a[%6], %1\n\t"
                 "v_accvgpr_write_b32 a[%7], %2\n\tv_accvgpr_write_b32 a[%8], %3"
                 : "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3)
                 : "v"(f), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
}
template <int I> __device__ __forceinline__ f32x4 out_read4() {
    float t0, t1, t2, t3;
    asm volatile("v_accvgpr_read_b32 %0, a[%4]\n\tv_accvgpr_read_b32 %1, a[%5]\n\t"
                 "v_accvgpr_read_b32 %2, a[%6]\n\tv_accvgpr_read_b32 %3, a[%7]"
                 : "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3) : "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
    return f32x4{t0, t1, t2, t3};
}
template <int I> __device__ __forceinline__ void out_zero4() {
    asm volatile("v_accvgpr_write_b32 a[%0], 0\n\tv_accvgpr_write_b32 a[%1], 0\n\t"
                 "v_accvgpr_write_b32 a[%2], 0\n\tv_accvgpr_write_b32 a[%3], 0"
                 :: "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
}
#define DCPA_A8(x) "a" #x "0", "a" #x "1", "a" #x "2", "a" #x "3", "a" #x "4", "a" #x "5", "a" #x "6", "a" #x "7", "a" #x "8", "a" #x "9"
// Declares the accumulation registers as written: the kernel is given them, and
// the compiler keeps no value of its own in one of them across this place.  It
// stands wherever a value could be live for long.
__device__ __forceinline__ void out_claim() {
    asm volatile("" ::: DCPA_A8(), DCPA_A8(1), DCPA_A8(2), DCPA_A8(3), DCPA_A8(4), DCPA_A8(5), DCPA_A8(6), DCPA_A8(7),
                 DCPA_A8(8), DCPA_A8(9), DCPA_A8(10), DCPA_A8(11), DCPA_A8(12), DCPA_A8(13), DCPA_A8(14), DCPA_A8(15),
                 DCPA_A8(16), DCPA_A8(17), DCPA_A8(18), DCPA_A8(19), DCPA_A8(20), DCPA_A8(21), DCPA_A8(22),
                 DCPA_A8(23), DCPA_A8(24), "a250", "a251", "a252", "a253", "a254", "a255");
}
#undef DCPA_A8

template <int N, typename F> __device__ __forceinline__ void times(F&& f) {
    [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }(
        std::make_integer_sequence<int, N>{});
}

constexpr int DK = 576, DV = 512, KT = 32;
// A tile in LDS: 32 rows of the first 512 columns (1 KB each), then 32 rows of
// the other 64.  Chunk c of row r lies at c ^ swz(r) of its part.
constexpr int MAIN = KT * 1024, KB = MAIN + KT * 128;

// 16 bytes at base + off of every lane (base the same for the wave) to LDS.
__device__ __forceinline__ void dma16_from(uint64_t base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(to)) : "memory");
}
__device__ __forceinline__ uint64_t lane64(uint64_t x, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane) << 32;
}

// EXACT: rows of all 576 columns (others are padded with zeros).
template <typename E, bool KV8, bool EXACT, bool WIDE>
__device__ __forceinline__ void latent_rows(const AttnArgs& p) {
    constexpr int R = 128, STEPS = DK / 16, CBS = DV / 32;
    // Tiles t and t + 1 are read while t + 2 and t + 3 arrive.  8-bit rows arrive as
    // they lie in the cache and are widened when their turn comes.
    constexpr int NBUF = KV8 ? 3 : 4, RAW = KV8 ? KT * DK : 0;
    __shared__ __attribute__((aligned(1024))) char tile[NBUF * KB + 2 * RAW];
    __shared__ uint8_t there_at[8][4];
    // page numbers of the keys of 8 tiles, and of the next 8
    constexpr int GROUP = 8;
    static_assert(GROUP * KT == 256, "a key to a thread");
    __shared__ int32_t page_of[2][GROUP * KT];
    // what the registers do not hold of the queries: the last QL fragments
    constexpr int QL = 3, QR = STEPS - QL;
    __shared__ u32x4 query_s[QL][256];

    const int hk = (int)(blockIdx.x % (uint32_t)p.m.Hkv), unit = (int)(blockIdx.x / (uint32_t)p.m.Hkv);
    const Unit u = find_unit<KT>(p.m, R, p.slots, p.share, unit);
    if (!u.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = (int)dcp::wave_id(), r = lane & 31, h = lane >> 5;
    const int nrows = u.s.n * p.m.G, row0 = u.tile * R, wave_row = wave * 32;
    const int last_row = min(row0 + R, nrows) - 1;
    const int kend = visible(p.m, u.s, (int)fdiv((uint32_t)last_row, p.m.fG));
    const int k0 = u.split * u.chunk, k1 = (int)min((int64_t)kend, (int64_t)k0 + u.chunk);
    if (u.split > 0 && k0 >= k1) return;      // (the join counts the ranges by itself)
    const int tiles = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;

    // --- tiles into LDS: a wave fetches 8 rows, lane l knows where row l / 8 of them lies
    const int64_t koff = (int64_t)hk * p.k_H;
    const int32_t* table = p.m.table + (int64_t)u.b * p.m.t_B;
    const int my_key = k0 + wave * 8 + lane / 8;
    const uint32_t lds0 = lds_addr(&tile[0]);
    auto page_at = [&](int key) { return key < k1 ? table[fdiv((uint32_t)key, p.m.fpage)] : -1; };
    uint64_t row_at = 0;           // of the tile that is fetched next
    auto page_for = [&](int t) {
        return t < tiles ? page_of[t / GROUP & 1][t % GROUP * KT + wave * 8 + lane / 8] : -1;
    };
    auto place_rows = [&](int t, int page) {
        const uint32_t key = (uint32_t)(my_key + t * KT);
        const uint32_t place = key - fdiv(key, p.m.fpage) * p.m.fpage.d;
        row_at = page_row(page, p.m, p.k, p.k_P, p.k_S, koff, place);
        // one bit for each of the 8 rows
        const uint64_t bits = __ballot((lane & 7) == 0 && (uint32_t)page < (uint32_t)p.m.pages);
        there_at[t & 7][wave] = (uint8_t)(bits * 0x0102040810204080ull >> 56);
    };
    auto buffer = [&](int t) { return lds0 + (uint32_t)(t % NBUF * KB); };
    // byte offsets of the lane's piece of a row: the wave's rows differ in known bits of swz()
    const uint32_t my_off = (uint32_t)((lane ^ (wave & 1)) * 16);
    const uint32_t my_rest = (uint32_t)((64 + ((lane & 7) ^ swz<8>(wave * 8 + lane / 8))) * 16);
    // the wave's rows of a tile, in nine pieces: of each row the first 512 columns, then what is
    // left of all eight
    auto fetch_piece = [&](uint32_t buf, auto piece) {
        constexpr int i = decltype(piece)::value;
        if constexpr (i < 8) {
            const uint32_t off = my_off ^ (uint32_t)(swz<64>(i) * 16);
            const uint32_t to = buf + (uint32_t)((wave * 8 + i) * 1024);
            if constexpr (EXACT) dma16_from(lane64(row_at, 8 * i), off, to);
            else dma16((const char*)at_or_zeros((int)off < p.Dk * 2, lane64(row_at, 8 * i) + off),
                       __builtin_amdgcn_readfirstlane(to));
        } else {
            dma16((const char*)at_or_zeros(EXACT || (int)my_rest < p.Dk * 2, row_at + my_rest),
                  __builtin_amdgcn_readfirstlane(buf + (uint32_t)(MAIN + wave * 1024)));
        }
    };
    // 8-bit: rows as they are (576 bytes each) behind the tiles
    auto raw = [&](int t) { return lds0 + (uint32_t)(NBUF * KB + (t & 1) * RAW + wave * 8 * DK); };
    auto fetch_raw = [&](int t) {
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            // 288 pieces of 16 bytes: 36 to a row; the last round is half empty and repeats the last piece
            const int ch = min(i * 64 + lane, 8 * 36 - 1), row = ch / 36, c = ch % 36;
            const uint64_t base = (uint64_t)(uint32_t)__shfl((int)(uint32_t)row_at, row * 8, 64) |
                                  (uint64_t)(uint32_t)__shfl((int)(uint32_t)(row_at >> 32), row * 8, 64) << 32;
            if (i < 4 || lane < 32)
                dma16((const char*)at_or_zeros(c * 16 + 16 <= p.Dk && (base & 15) == 0, base + (uint64_t)(c * 16)),
                      __builtin_amdgcn_readfirstlane(raw(t) + (uint32_t)(i * 1024)));
        }
    };
    auto widen = [&](int t, uint64_t rows) {
        const uint32_t buf = buffer(t);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            // (all lanes take part in the exchange; the last round's upper half repeats a piece)
            const int ch = min(i * 64 + lane, 8 * 36 - 1);
            const int row = ch / 36, c = ch % 36, in_tile = wave * 8 + row;
            u32x4 x = lds_read16(raw(t) + (uint32_t)(ch * 16));
            // rows that are only 8-byte aligned, and the half piece at a row's end
            const uint64_t base = (uint64_t)(uint32_t)__shfl((int)(uint32_t)rows, row * 8, 64) |
                                  (uint64_t)(uint32_t)__shfl((int)(uint32_t)(rows >> 32), row * 8, 64) << 32;
            if (c * 16 < p.Dk && ((base & 15) != 0 || c * 16 + 16 > p.Dk)) {
                const u32x2 lo = *(const u32x2*)(base + (uint64_t)(c * 16));
                u32x2 hi = {0, 0};
                if (c * 16 + 16 <= p.Dk) hi = *(const u32x2*)(base + (uint64_t)(c * 16 + 8));
                x = u32x4{lo.x, lo.y, hi.x, hi.y};
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = 2 * c + k;
                const uint32_t to = d < 64 ? (uint32_t)(in_tile * 1024 + (d ^ swz<64>(in_tile)) * 16)
                                           : (uint32_t)(MAIN + in_tile * 128 + ((d - 64) ^ swz<8>(in_tile)) * 16);
                lds_write16(buf + to, widen8<E>(k == 0 ? u32x2{x.x, x.y} : u32x2{x.z, x.w}));
            }
        }
    };
    // tile t asked for; its rows have been placed
    auto fetch = [&](int t) {
        if constexpr (KV8) fetch_raw(t);
        else times<9>([&](auto i) { fetch_piece(buffer(t), i); });
    };
    auto load_pages = [&](int group, int32_t (&x)[1]) {
        x[0] = page_at(k0 + group * GROUP * KT + tid);
    };
    auto keep_pages = [&](int group, const int32_t (&x)[1]) {
        page_of[group & 1][tid] = x[0];
    };

    out_claim();
    times<DV / 8>([&](auto i) { out_zero4<i * 4>(); });
    u32x4 q[QR];
    const int my_row = min(row0 + wave_row + r, last_row), token = (int)fdiv((uint32_t)my_row, p.m.fG);
    const int vis = visible(p.m, u.s, token) - k0;
    {
        u32x4 all[STEPS];
        load_query<DK>(all, p.q + (int64_t)(u.s.first + token) * p.q_T +
                                (int64_t)(hk * p.m.G + my_row - token * p.m.G) * p.q_H, p.Dk, h);
#pragma unroll
        for (int i = 0; i < QR; ++i) q[i] = all[i];
#pragma unroll
        for (int i = 0; i < QL; ++i) query_s[i][tid] = all[QR + i];
    }
    auto query = [&](int st) { return st < QR ? q[min(st, QR - 1)] : query_s[max(st, QR) - QR][tid]; };
    const int vmin = __builtin_amdgcn_readlane(vis, 0), vmax = __builtin_amdgcn_readlane(vis, 31);
    const bool work = row0 + wave_row < nrows;          // (waves behind the last row only help to fetch)
    float mc = kNoMax, l = 0.0f;
    bool odd = false;

    // Lane constants of the fragment reads (see attn_tile.hpp).  A step's chunk differs from the
    // first one's in bits that the places are xored into anyway, so one address serves all; values
    // are read where the keys' places put them, the second four rows of a fragment at the other
    // chunk of a pair.
    const uint32_t ka = (uint32_t)(r * 1024 + (h ^ swz<64>(r)) * 16);
    const uint32_t kt = (uint32_t)(MAIN + r * 128 + (h ^ swz<8>(r)) * 16);
    const int g = (lane >> 4) & 1, li = lane & 15;
    const uint32_t va = (uint32_t)((4 * h + li / 4) * 1024 + (li & 1) * 8 +
                                   ((2 * g + (li & 3) / 2) ^ swz<64>(4 * h + li / 4)) * 16);
    auto key_fragment = [&](uint32_t buf, int st) {
        if (st < 32) return lds_read16(((buf + ka) ^ (uint32_t)((st & 7) * 32)) + (uint32_t)((st >> 3) * 256));
        return lds_read16((buf + kt) ^ (uint32_t)((st - 32) * 32));
    };
    auto value_fragment = [&](uint32_t buf, int i) {          // i = 2 * block + half of the keys
        const uint32_t off = (uint32_t)((i >> 3) * 256 + (i & 1) * 16 * 1024), turn = (uint32_t)((i >> 1 & 3) * 64);
        const u32x2 x = lds_read_tr(((buf + va) ^ turn) + off);
        const u32x2 y = lds_read_tr(((buf + va) ^ (turn | 16u)) + off + 8 * 1024);
        return u32x4{x.x, x.y, y.x, y.y};
    };
    constexpr int AHEAD = 4, VAHEAD = 4;
    constexpr int SETTLED = 5;         // products after which the result of the one before them is in its registers
#define DCPA_PIN __builtin_amdgcn_sched_barrier(0)

    // what arrives first: tile 0, then 1 and 2
    f32x16 s;
    uint64_t rows1 = 0, rows2 = 0;     // 8-bit: of the two tiles that are still to be widened
    if (tiles > 0) {
        int32_t x[1];
        load_pages(0, x);
        keep_pages(0, x);
        meet();
#pragma unroll 1
        for (int t = 0; t < 3; ++t) {
            place_rows(t, page_for(t));
            if (KV8 && t == 2) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            fetch(t);
            if (KV8 && t == 0) {
                dma_wait();
                widen(0, row_at);
            }
            if (KV8 && t == 1) rows1 = row_at;
            if (KV8 && t == 2) rows2 = row_at;
        }
        // (tiles 1 and 2 may still be on their way)
        if constexpr (!KV8) asm volatile("s_waitcnt vmcnt(18)" ::: "memory");
        meet();
        if (work && vmax > 0) {
            const uint32_t buf = buffer(0);
            times<STEPS>([&](auto st) {
                if constexpr (st == 0) mma_first<E>(s, key_fragment(buf, st), query(st));
                else mma_next<E>(s, key_fragment(buf, st), query(st));
            });
            settle(s);
        }
    }
    out_claim();

    // masks of tile t's scores, where there is something to mask
    bool whole = true;
    float best = -INFINITY;            // of the scores of this half-wave's keys
    auto present = [&](int t) { return (uint32_t)__builtin_amdgcn_readfirstlane(*(const int*)&there_at[t & 7][0]); };
    auto mask = [&](int t, uint32_t there, f32x16& x) {
        whole = there == 0xffffffffu && vmin >= (t + 1) * KT;
        if (whole) return;
        settle(x);
        const uint32_t bits = there >> (4 * h);
        const int lim = vis - t * KT - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = 8 * (i / 4) + i % 4;
            x[i] = (bits >> j & 1u) != 0 && j < lim ? x[i] : -INFINITY;
        }
    };
    if (tiles > 0 && work && vmax > 0) {
        mask(0, present(0), s);
#pragma unroll
        for (int i = 0; i < 16; ++i) best = fmaxf(best, s[i]);
    }

    // One tile's weights and outputs, with the next tile's scores between: the
    // exponentials run in the shadow of its matrix instructions, one to two of them
    // (an exponential takes half a product's time).  The nine pieces of tile t + 3
    // are asked for all along, so that the four waves' requests do not queue up.
    auto advance = [&](int t, uint32_t buf, uint32_t nbuf, uint32_t to, auto next) {
        constexpr bool NEXT = decltype(next)::value;
        u32x4 kf[AHEAD], vf[VAHEAD];
        const int page = page_for(t + 3);
        const uint32_t there = NEXT ? present(t + 1) : 0;      // (read early, ahead of the fragments)
        if constexpr (NEXT) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) kf[i] = key_fragment(nbuf, i);
        }
        const bool full = whole;
        const float top = half_max(best) * p.c;
        if (__ballot(top > mc + Mat<E>::kTop + kLazy) != 0) {
            const float next_mc = top > mc + Mat<E>::kTop ? top - Mat<E>::kTop : mc;
            const float f = exp2_fast(mc - next_mc);
            mc = next_mc;
            l *= f;
            asm volatile("s_nop 15\n\ts_nop 3");
            times<DV / 8>([&](auto i) { out_scale4<i * 4>(f); });
        }
        uint32_t pr[8], rest[8];
        float sum = 0.0f;
        f32x16 n;
        u32x4 ql[QL];
        if constexpr (KV8) {
            place_rows(t + 3, page);
            fetch(t + 3);
        }
        DCPA_PIN;
        times<STEPS>([&](auto st) {
            if constexpr (NEXT) {
                if constexpr (st == 0) mma_first<E>(n, kf[0], q[0]);
                else if constexpr (st < QR) mma_next<E>(n, kf[st % AHEAD], q[st]);
                else mma_next<E>(n, kf[st % AHEAD], ql[st - QR]);
                DCPA_PIN;
                if constexpr (st + AHEAD < STEPS) kf[st % AHEAD] = key_fragment(nbuf, st + AHEAD);
                if constexpr (st + AHEAD >= QR && st + AHEAD < STEPS) ql[st + AHEAD - QR] = query_s[st + AHEAD - QR][tid];
            }
            if constexpr (st < 32 && st % 2 == 0) {
                s[st / 2] = exp2_fast(__builtin_fmaf(s[st / 2], p.c, -mc));
                if constexpr (st % 4 == 0) asm volatile("" : "+v"(s));
            } else if constexpr (st < 32) {
                // (pinned here: the compiler would compute them later, between the products that need them)
                sum += s[st / 2];
                asm volatile("" : "+v"(sum));
                if constexpr (st % 4 == 3) {
                    pr[st / 4] = Mat<E>::pack2(s[st / 2 - 1], s[st / 2]);
                    asm volatile("" : "+v"(pr[st / 4]));
                    if constexpr (WIDE) {
                        rest[st / 4] = Mat<E>::pack2(s[st / 2 - 1] - Mat<E>::low(pr[st / 4]), s[st / 2] - Mat<E>::high(pr[st / 4]));
                        asm volatile("" : "+v"(rest[st / 4]));
                    }
                }
            }
            if constexpr (!KV8 && st == 2) place_rows(t + 3, page);
            if constexpr (!KV8 && st % 7 == 5) fetch_piece(to, std::integral_constant<int, st / 7>{});
            if constexpr (st >= STEPS - VAHEAD) vf[st - (STEPS - VAHEAD)] = value_fragment(buf, 2 * (st - (STEPS - VAHEAD)));
            DCPA_PIN;
        });
        l += sum;
        if constexpr (NEXT) mask(t + 1, there, n);
        best = -INFINITY;
        const u32x4 p0 = {pr[0], pr[1], pr[2], pr[3]}, p1 = {pr[4], pr[5], pr[6], pr[7]};
        DCPA_PIN;
        asm volatile("s_nop 1");      // (the weights were written just before)
        times<2 * CBS>([&](auto i) {
            // the two halves of the keys one after the other, so that a product does not wait for
            // the one before it
            constexpr int half = i / CBS, cb = i % CBS, m = i + VAHEAD;
            out_mma<E, cb>(vf[i % VAHEAD], half == 0 ? p0 : p1);
            if constexpr (WIDE) {
                constexpr int at = half * 4;
                DCPA_PIN;
                out_mma<E, cb>(vf[i % VAHEAD], u32x4{rest[at], rest[at + 1], rest[at + 2], rest[at + 3]});
            }
            if constexpr (m < 2 * CBS) vf[i % VAHEAD] = value_fragment(buf, m % CBS * 2 + m / CBS);
            DCPA_PIN;
            // the next tile's maximum; its last product was done four products ago
            if constexpr (NEXT && i >= SETTLED && (i - SETTLED) % 3 == 0 && (i - SETTLED) / 3 < 8) {
                constexpr int k = (i - SETTLED) / 3 * 2;
                if constexpr (k == 0) asm volatile("" : "+v"(n));
                best = fmaxf(best, fmaxf(n[k], n[k + 1]));
                asm volatile("" : "+v"(best));
                DCPA_PIN;
            }
            if constexpr (!KV8 && i % 7 == 5 && 5 + i / 7 < 9) {
                fetch_piece(to, std::integral_constant<int, 5 + i / 7>{});
                DCPA_PIN;
            }
        });
        out_claim();
        if (!full) odd |= odd_values<E, false>(buf, MAIN);
        if constexpr (NEXT) s = n;
    };

    uint32_t at0 = buffer(0), at1 = buffer(1), at2 = buffer(2), at3 = buffer(3);    // of tiles t .. t + 3
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        out_claim();
        // this wave's rows of tile t + 1 are there; the pieces of t + 2 may still be on their way
        if constexpr (KV8) {
            asm volatile("s_waitcnt vmcnt(5)" ::: "memory");
            if (t + 1 < tiles) widen(t + 1, rows1);
            rows1 = rows2;
        } else {
            asm volatile("s_waitcnt vmcnt(9)" ::: "memory");
        }
        meet();               // tile t + 1 is there, and every wave is done with tile t - 1
        if (t % GROUP == 0 && t + GROUP < tiles) {
            int32_t x[1];
            load_pages(t / GROUP + 1, x);
            keep_pages(t / GROUP + 1, x);
        }
        // (behind the last tile the rows are the row of zeros: the count above stays the same)
        if (work && vmax > t * KT) {
            if (t + 1 < tiles && vmax > (t + 1) * KT) advance(t, at0, at1, at3, std::true_type{});
            else advance(t, at0, at1, at3, std::false_type{});
        } else {
            place_rows(t + 3, page_for(t + 3));
            fetch(t + 3);
        }
        if constexpr (KV8) rows2 = row_at;
        const uint32_t past = at0;
        at0 = at1;
        at1 = at2;
        at2 = KV8 ? past : at3;
        at3 = past;
    }
#undef DCPA_PIN
    dma_wait();               // nothing may arrive in LDS after the workgroup's end

    if (odd) {
        meet();               // (the others meet once more before they write)
        slow_rows<E, KV8, DK, DV>(late_args<AttnArgs>(), u, hk, unit, R, row0, row0 + wave_row, min(row0 + wave_row + 32, nrows), k0, k1);
        return;
    }
    asm volatile("s_nop 15\n\ts_nop 3");
    out_claim();
    const AttnArgs& e = late_args<AttnArgs>();
    const float lsum = half_sum(l);
    float f, lse2;
    finish(lsum, mc, e.vs, f, lse2);
    const int my = row0 + wave_row + r;
    const int64_t part = ((int64_t)hk * e.units + unit) * R;
    const bool split = u.splits > 1;
    if (h == 0 && my < nrows) {
        if (split) e.ws_l[part + wave_row + r] = lse2;
        else if (e.lse != nullptr)
            e.lse[(int64_t)(u.s.first + token) * e.l_T + (int64_t)(hk * e.m.G + my_row - token * e.m.G) * e.l_H] = lse2 * e.lmul;
    }
    // The lanes hold columns of a row; through LDS, half the columns at a time, they become
    // stretches of rows, which are written whole.  (Each wave its own 32 KB; chunk c of row r at c ^ r.)
    const uint32_t mine = lds0 + (uint32_t)(wave * 32768);
    int ln = lane;
    asm volatile("" : "+v"(ln));             // (keeps the addresses below from being held all along)
    const int er = ln & 31, eh = ln >> 5;
    static_assert(sizeof(tile) >= 4 * 32768, "room for half the outputs");
    const int Dv = e.Dv;
    const FastDiv fG = e.m.fG;
    const int64_t o_T = e.o_T, o_H = e.o_H;
    char* out = e.out + (int64_t)u.s.first * o_T + (int64_t)hk * e.m.G * o_H;
    float* parts = e.ws_o + (part + wave_row) * Dv;
    meet();                   // (other waves may still have been reading tiles, or fallen out)
    times<2>([&](auto part_of) {
        constexpr int P = decltype(part_of)::value;
        times<DV / 16>([&](auto i) {
            f32x4 x = out_read4<P * (DV / 4) + i * 4>();
            x = lsum == 0.0f ? f32x4{0, 0, 0, 0} : x * f;
            lds_write16(mine + (uint32_t)(er * 1024 + ((2 * i + eh) ^ er) * 16), __builtin_bit_cast(u32x4, x));
        });
        // (this wave's LDS accesses stay in order)
        const int col = P * (DV / 2) + ln * 4;
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 8) {
            f32x4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = __builtin_bit_cast(f32x4, lds_read16(mine + (uint32_t)((k0 + k) * 1024 + (ln ^ (k0 + k)) * 16)));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int row = row0 + wave_row + k0 + k;
                if (row < nrows && col < Dv) {
                    if (split) {
                        *(f32x4*)(parts + (int64_t)(k0 + k) * Dv + col) = x[k];
                    } else {
                        const int tok = (int)fdiv((uint32_t)row, fG);
                        store4<E>(out + (int64_t)tok * o_T + (int64_t)(row - tok * (int)fG.d) * o_H + col * 2, x[k][0], x[k][1],
                                  x[k][2], x[k][3]);
                    }
                }
            }
        }
    });
}

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
            return a.Dk == DK ? launch(latent_wide<E, K8, true>, grid, block, stream, a)
                              : launch(latent_wide<E, K8, false>, grid, block, stream, a);
        return a.Dk == DK ? launch(attn_latent<E, K8, true>, grid, block, stream, a)
                          : launch(attn_latent<E, K8, false>, grid, block, stream, a);
    };
    if (bf16) return kv8 ? run(BF16T{}, std::true_type{}) : run(BF16T{}, std::false_type{});
    return kv8 ? run(F16T{}, std::true_type{}) : run(F16T{}, std::false_type{});
}

}  // namespace dcpa
