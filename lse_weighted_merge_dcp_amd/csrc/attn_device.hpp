// attn_device.hpp -- device helpers of the cached-attention kernels: matrix
// instructions, the LDS layout of a key tile, loads that go straight into
// LDS, and the mapping of workgroups to sequences.
#pragma once
#include <type_traits>

#include "attn_launch.hpp"
#include "dcp_device.hpp"

namespace dcpa {

using dcp::BF16T;
using dcp::F16T;
using dcp::fdiv;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

#define DCPA_LDS __attribute__((address_space(3)))

// --------------------------------------------------------------------------
// v_mfma 32x32x16: D[m][n] += sum_k A[m][k] B[k][n].  Lane l holds A[l%32][8h
// .. 8h+7] and B[8h .. 8h+7][l%32] with h = l / 32, and D[8(i/4) + i%4 +
// 4h][l%32] in register i of 16.
// --------------------------------------------------------------------------
template <typename E> struct Mat;
template <> struct Mat<BF16T> {
    static __device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) {
        bf16x2 v;
        v.x = (__bf16)a;
        v.y = (__bf16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    // the two halves of a pack2, widened
    static __device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
    static __device__ __forceinline__ float high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
    static constexpr uint32_t kExp = 0x7f807f80u;   // exponent bits of the two halves
    // The weights' exponent is free: with the row maximum at 2^0 the smallest
    // bf16 is far below fp32's resolution of the sum.
    static constexpr float kTop = 0.0f;
};
template <> struct Mat<F16T> {
    static __device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) {
        f16x2 v;
        v.x = (_Float16)a;
        v.y = (_Float16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ float low(uint32_t v) { return (float)__builtin_bit_cast(f16x2, v).x; }
    static __device__ __forceinline__ float high(uint32_t v) { return (float)__builtin_bit_cast(f16x2, v).y; }
    static constexpr uint32_t kExp = 0x7c007c00u;
    // fp16 loses relative precision below 2^-14: the row maximum stands at
    // 2^8, so that weights down to 2^-22 of the largest keep 11 bits.
    static constexpr float kTop = 8.0f;
};

// A new row maximum rescales sums and outputs only when it is more than this
// many powers of two above the old reference: weights reach 2^(kTop + 6) at
// most (2^14 < 65504 in fp16), and almost no tile rescales.
constexpr float kLazy = 6.0f;
constexpr float kNoMax = -3.0e38f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The other half-wave's value beside one's own: lanes l and l ^ 32 get the
// same result.
__device__ __forceinline__ float half_max(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// --------------------------------------------------------------------------
// A tile in LDS is [rows][C chunks of 16 bytes]; chunk c of row r lies at place
// c ^ swz(r).  LDS serves 64 banks, 256 bytes, a clock: a key fragment's read
// takes one chunk column of 16 rows at a time, which then lie in 16 different
// places of 256 bytes; a value fragment's transposing read 64 bytes of four
// neighbouring rows, or 32 bytes of eight.  (Counters: no bank conflicts in
// either; with the rows' low three bits alone both took twice the clocks.)
// Rows of an odd number of 128 bytes already alternate between the halves.
// --------------------------------------------------------------------------
template <int C> __device__ __forceinline__ int swz(int r) {
    if constexpr (C % 16 == 0) return (r & 3) << 2 | (r >> 2 & 1) << 1 | (r >> 3 & 1);
    else return (r >> 1 & 1) << 2 | (r >> 2 & 1) << 1 | (r >> 3 & 1);
}
// For values in a tile of their own: rows r and r + 8 at the same place.
template <int C> __device__ __forceinline__ int swz_v(int r) { return swz<C>(r & 7); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const DCPA_LDS char*)p;
}
__device__ __forceinline__ u32x4 lds_read16(uint32_t a) { return *(const DCPA_LDS u32x4*)(uintptr_t)a; }
__device__ __forceinline__ void lds_write16(uint32_t a, u32x4 x) { *(DCPA_LDS u32x4*)(uintptr_t)a = x; }
// Four 8-byte pieces of 16 lanes are four rows of 16 elements; lane i of the 16
// gets column i of the four rows.
__device__ __forceinline__ u32x2 lds_read_tr(uint32_t a) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((DCPA_LDS s16x4*)(uintptr_t)a));
}

// 16 bytes of every lane from global memory to LDS at base + 16 * lane (base
// the same for the wave).  Written in asm so that the compiler does not put a
// wait for it in front of every LDS read; dma_wait() has to run before the
// data is read.  (m0 is never allocated, so writing it needs no clobber.)
__device__ __forceinline__ void dma16(const char* g, uint32_t base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"((uint64_t)g), "s"(base) : "memory");
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// All LDS accesses of this wave done, then the workgroup meets.
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Sixteen 8-byte pieces of 16 lanes are eight rows of 16 bytes; lane i of the 16
// gets column i of the eight rows.
typedef int i32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 lds_read_tr8(uint32_t a) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((DCPA_LDS i32x2*)(uintptr_t)a));
}

// What absent keys and columns are loaded from: a row of the widest cache.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[288] = {};

// a * b, b >= 0, in the two products it takes.
__device__ __forceinline__ uint64_t times64(uint32_t a, int64_t b) {
    return (uint64_t)a * (uint32_t)b + ((uint64_t)(a * (uint32_t)((uint64_t)b >> 32)) << 32);
}
// at, or the row of zeros (in bit operations: written as a choice, the compiler
// branches around the read of `at` for every piece).
__device__ __forceinline__ uint64_t at_or_zeros(bool ok, uint64_t at) {
    const uint64_t mask = 0 - (uint64_t)ok;
    return (at & mask) | ((uint64_t)kZeros & ~mask);
}

// Eight e4m3 values as eight 16-bit ones (exact: both types hold them).
template <typename E> __device__ __forceinline__ u32x4 widen8(u32x2 x) {
    u32x4 r;
    if constexpr (std::is_same_v<E, BF16T>) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, 1.0f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, 1.0f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, 1.0f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, 1.0f, true));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x.x, 1.0f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x.x, 1.0f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x.y, 1.0f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x.y, 1.0f, true));
    }
    return r;
}

// The kernel's arguments, read again where they are needed late: held from the
// start they would take scalar registers through the whole main loop.
template <typename T> __device__ __forceinline__ const T& late_args() {
    typedef const __attribute__((address_space(4))) T* Ptr;
    Ptr p = (Ptr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const T*)p;
}

// --------------------------------------------------------------------------
// lengths
// --------------------------------------------------------------------------
// Positions below x that lie on this rank.
__device__ __forceinline__ int owned(const Batch& m, int x) {
    const uint32_t u = (uint32_t)max(x, 0), full = fdiv(u, m.fblock), rest = u - full * m.fblock.d;
    return (int)(full * (uint32_t)m.inter) + min(max((int)rest - m.rank * m.inter, 0), m.inter);
}

struct Seq {
    int first, n;   // token rows [first, first + n)
    int kv;         // cached keys
    int len;        // whole length
};

__device__ __forceinline__ Seq load_seq(const Batch& m, int b) {
    Seq s;
    s.first = min(max(m.cu[b], 0), m.T);
    s.n = min(max(m.cu[b + 1], s.first), m.T) - s.first;
    s.kv = min(max(m.kv[b], 0), m.max_keys);
    s.len = m.seq != nullptr ? m.seq[b] : 0;
    return s;
}

// Lane `at`'s sequence, for the whole wave.
__device__ __forceinline__ Seq seq_of(const Seq& s, int at) {
    return Seq{__builtin_amdgcn_readlane(s.first, at), __builtin_amdgcn_readlane(s.n, at),
               __builtin_amdgcn_readlane(s.kv, at), __builtin_amdgcn_readlane(s.len, at)};
}

// Keys that token i of the sequence sees.
__device__ __forceinline__ int visible(const Batch& m, const Seq& s, int i) {
    if (!m.causal) return s.kv;
    const int hidden = m.seq == nullptr ? s.n - 1 - i : owned(m, s.len) - owned(m, s.len - s.n + i + 1);
    return min(max(s.kv - hidden, 0), s.kv);
}

// Inclusive prefix sum over the wave: within rows of 16 lanes, then across them.
__device__ __forceinline__ int scan_incl(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);    // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);    // lane 15 to row 1, 47 to row 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);    // lane 31 to rows 2 and 3
    return x;
}
// Sums that stop at `most` (<= 2^30): what a lane adds never passes 2^31.
__device__ __forceinline__ int add_to(int a, int b, int most) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)most); }
template <int CTRL, int ROWS> __device__ __forceinline__ int scan_step(int x, int most) {
    return add_to(x, __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false), most);
}
// scan_incl() of such sums.
__device__ __forceinline__ int scan_upto(int x, int most) {
    x = scan_step<0x111, 0xf>(x, most);
    x = scan_step<0x112, 0xf>(x, most);
    x = scan_step<0x114, 0xf>(x, most);
    x = scan_step<0x118, 0xf>(x, most);
    x = scan_step<0x142, 0xa>(x, most);
    return scan_step<0x143, 0xc>(x, most);
}
// The wave's sum, largest or smallest value, for every lane: OP(a, b) over rows of 16 lanes, then across them
// (exchanges within the vector unit: a shuffle through LDS takes a hundred clocks).  `none`: OP's neutral value.
template <int CTRL, int ROWS, typename T, typename F> __device__ __forceinline__ T fold_step(T x, T none, F&& op) {
    static_assert(sizeof(T) == 4, "one register");
    const int y = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false);
    return op(x, __builtin_bit_cast(T, y));
}
template <typename T, typename F> __device__ __forceinline__ T fold_wave(T x, T none, F&& op) {
    x = fold_step<0x111, 0xf>(x, none, op);
    x = fold_step<0x112, 0xf>(x, none, op);
    x = fold_step<0x114, 0xf>(x, none, op);
    x = fold_step<0x118, 0xf>(x, none, op);
    x = fold_step<0x142, 0xa>(x, none, op);
    x = fold_step<0x143, 0xc>(x, none, op);
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
// x plus the x of the lane that CTRL names, over the rows of lanes in ROWS (each half moved as 32 bits)
template <int CTRL, int ROWS> __device__ __forceinline__ double add_from(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}
// Sum over the wave of whole numbers that add up to less than 2^53 (exact in a double, whose sum is one
// instruction and needs no carry)
__device__ __forceinline__ int64_t sum_wave(int64_t v) {
    double x = add_from<0x118, 0xf>(add_from<0x114, 0xf>(add_from<0x112, 0xf>(add_from<0x111, 0xf>((double)v))));
    x = add_from<0x143, 0xc>(add_from<0x142, 0xa>(x));
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return (int64_t)__builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63));
}

// Workgroups that read no key twice, of few rows: those of all key heads of a unit follow each other on one XCD
// (workgroups go round the eight XCDs), since a cached token's heads lie next to each other, their weights in one
// line even.
__device__ __forceinline__ void heads_together(const Batch& m, int& hk, int& unit) {
    const uint32_t id = blockIdx.x, turn = fdiv(id >> 3, m.fHkv);
    hk = (int)((id >> 3) - turn * m.fHkv.d);
    unit = (int)(turn * 8 + (id & 7));
}

// The share of a batch that one workgroup takes: row tile `tile` of sequence
// b against the keys [split * chunk, (split + 1) * chunk).  Every wave works
// it out by itself from the lengths on the device, so ragged batches are
// balanced whatever the width of the page table, and the host needs no
// lengths.
struct Unit {
    Seq s;
    int b, tile, split, splits, chunk;
    int slot;       // of the tile's first split
    bool ok;
};

constexpr int kWhole = 0x40000000;     // longer than any cache

// Row tiles and cached keys of sequence b (none behind the last one).
__device__ __forceinline__ void tiles_of(const Batch& m, int b, int rows, int& tiles, int& kv) {
    tiles = kv = 0;
    if (b < m.B) {
        const Seq s = load_seq(m, b);
        tiles = (s.n * m.G + rows - 1) / rows;
        kv = s.kv;
    }
}

// The length of a key range: the shortest multiple of STEP (to within an
// eighth of the interval) with which the whole batch needs at most `slots`
// units and none more than a `share`-th of its work; kWhole where the tiles
// alone need that many.  `longest`: the most keys that the lane met.
template <int STEP>
__device__ __forceinline__ int key_chunk(const Batch& m, int rows, int slots, int share, int& longest) {
    longest = 0;
    if (slots <= 0) return kWhole;
    const int lane = threadIdx.x & 63;
    int64_t work = 0;
    int all = 0, tiles = 0, kv = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64) {
        tiles_of(m, b0 + lane, rows, tiles, kv);
        work += (int64_t)tiles * kv;
        all += tiles;
        longest = max(longest, kv);
    }
    work = sum_wave(work);
    all = (int)sum_wave((int64_t)all);
    if (all >= slots) return kWhole;
    // units <= work / chunk + tiles: `hi` is always enough, `lo` never too long
    auto steps = [](int64_t x) { return (int)min((int64_t)(kWhole / STEP), max((int64_t)2, (x + STEP - 1) / STEP)); };
    int lo = steps((work + share - 1) / share), hi = max(lo, steps((work + slots - all - 1) / (slots - all)));
#pragma unroll 1
    for (int round = 0; round < 3 && lo < hi; ++round) {
        const int mid = lo + (hi - lo) / 2;
        int64_t units = 0;
        for (int b0 = 0; b0 < m.B; b0 += 64) {
            if (m.B > 64) tiles_of(m, b0 + lane, rows, tiles, kv);
            units += (int64_t)tiles * max(1, (kv + mid * STEP - 1) / (mid * STEP));
        }
        units = sum_wave(units);
        if (units <= slots) hi = mid;
        else lo = mid + 1;
    }
    return hi * STEP;
}

template <int STEP>
__device__ __forceinline__ int key_chunk(const Batch& m, int rows, int slots, int share) {
    int longest;
    return key_chunk<STEP>(m, rows, slots, share, longest);
}

template <int STEP>
__device__ __forceinline__ Unit find_unit(const Batch& m, int rows, int slots, int share, int id) {
    Unit u;
    u.ok = false;
    u.chunk = key_chunk<STEP>(m, rows, slots, share);
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < m.B; b0 += 64) {
        int tiles = 0, kv = 0;
        Seq mine{};
        if (b0 + lane < m.B) {
            mine = load_seq(m, b0 + lane);
            tiles = (mine.n * m.G + rows - 1) / rows;
            kv = mine.kv;
        }
        const int splits = max(1, (kv + u.chunk - 1) / u.chunk);
        const int incl = base + scan_incl(tiles * splits);
        const uint64_t past = __ballot(incl > id);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            const int t = __builtin_amdgcn_readlane(tiles, at), s = __builtin_amdgcn_readlane(splits, at);
            const int rest = id - (__builtin_amdgcn_readlane(incl, at) - t * s);
            u.b = b0 + at;
            u.s = seq_of(mine, at);
            u.splits = s;
            // the last rows see most keys: they come first
            u.split = rest % s;
            u.tile = t - 1 - rest / s;
            u.slot = id - u.split;
            // (lengths that contradict each other could lead outside the tile)
            u.ok = rest >= 0 && u.tile >= 0 && (int64_t)u.tile * rows < (int64_t)u.s.n * m.G;
            return u;
        }
        base = __builtin_amdgcn_readlane(incl, 63);
    }
    return u;
}

// How a workgroup finds its share, and what its rows see, by the arguments of the
// kernel (attn_prefix.hpp has them for sequences that share keys).
template <int STEP> __device__ __forceinline__ Unit unit_of(const AttnArgs& p, int rows, int id) {
    return find_unit<STEP>(p.m, rows, p.slots, p.share, id);
}
__device__ __forceinline__ int first_key(const Unit&) { return 0; }
// one behind the last key that a row of the tile sees; last_row: the tile's last
__device__ __forceinline__ int last_key(const AttnArgs& p, const Unit& u, int last_row) {
    return visible(p.m, u.s, (int)fdiv((uint32_t)last_row, p.m.fG));
}
__device__ __forceinline__ int sees(const AttnArgs& p, const Unit& u, int token) { return visible(p.m, u.s, token); }
// The least and the most of the lanes' `vis` (32 rows, twice): rows are in the order of their tokens, the
// first sees least, the last most.
__device__ __forceinline__ int least_seen(const Unit&, int vis) { return __builtin_amdgcn_readlane(vis, 0); }
__device__ __forceinline__ int most_seen(const Unit&, int vis) { return __builtin_amdgcn_readlane(vis, 31); }

}  // namespace dcpa
