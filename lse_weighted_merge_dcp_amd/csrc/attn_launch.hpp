// attn_launch.hpp -- internal interface between the C ABI of libdcpattn
// (attn_api.cpp) and its kernel launchers.  Payload strides are in BYTES,
// strides of 32-bit arrays in words; the ABI converts.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fastdiv.hpp"

namespace dcpa {

using dcp::FastDiv;

// Lengths and order of a batch, common to the attention and the weight kernel.
struct Batch {
    const int32_t* table;
    int64_t t_B;
    const int32_t* cu;
    const int32_t* kv;
    const int32_t* seq;      // null: one rank, or not causal
    int32_t B, T, G;         // sequences, token rows, query heads per key head
    int32_t Hkv;
    int32_t pages, page_size, max_keys;
    int32_t N, rank, inter;
    int32_t causal;
    FastDiv fG, fpage, fHkv, fblock;     // fblock: N * inter
};

struct AttnArgs {
    Batch m;
    const char* q;
    int64_t q_T, q_H;
    const char* k;
    int64_t k_P, k_S, k_H;
    const char* v;           // null: the first Dv columns of the keys
    int64_t v_P, v_S, v_H;
    char* out;
    int64_t o_T, o_H;
    float* lse;              // nullable
    int64_t l_T, l_H;
    float* ws_o;             // [units][rows][Dv]
    float* ws_l;             // [units][rows]
    int32_t Dk, Dv;
    int32_t rows;            // of a tile
    int32_t slots;           // units of one key head that the keys are split into (0: not split)
    int32_t share;           // no key range longer than this share of the batch's keys needs
    int32_t units;           // (row tile, key range) pairs of one key head the launch covers
    float c;                 // scale * k_scale * log2(e): scores in powers of two
    float vs;                // v_scale
    float lmul;              // ln 2, or 1 for base 2
};

// How a call is laid out over workgroups; the same for the workspace query
// and the launch.
struct AttnPlan {
    int rows;                // rows of a tile
    bool latent;             // wide rows, the values are columns of the keys
    bool by_keys;            // the waves of a workgroup take different keys (few rows)
    int32_t slots, share, tiles, units;
    int64_t ws_bytes;
};
// Decode: the units that fill the chip, `slots`, leave no room to split a long sequence where the row
// tiles alone are nearly as many.  From half as many tiles on half a chip's units are added to them, and a
// sequence is split where it is longer than two units' equal shares, so that even batches stay whole.
// (128 sequences of about 1000 keys, one of 131072, 8 key heads: 216 us, unsplit 1663; all of
// about 1000: 120 us either way.  256 latent ones of 128 heads: 214 and 6291 us; 126 and 118 us.)  Where
// they fill the chip four times over they stay whole: every workgroup reads all lengths to split them, 500
// sequences of 100 keys take 105 us and 512 unsplit 81.
inline void fill_slots(int32_t tiles, int32_t& slots, int32_t& share) {
    if (2 * (int64_t)tiles <= slots) return;
    share = (slots + 1) / 2;
    slots = tiles + share;
}
// pieces: the cache's rows and strides are whole pieces of 16 bytes.
AttnPlan plan_attn(const Batch& m, int Dk, int Dv, bool pieces);
// wide: the weights' remainders take a second product where rows are many or latent too.
hipError_t launch_attn(const AttnArgs& a, const AttnPlan& pl, bool bf16, bool kv8, bool wide, hipStream_t stream);

hipError_t launch_latent(const AttnArgs& a, dim3 grid, bool bf16, bool kv8, bool wide, hipStream_t stream);

struct MassArgs {
    Batch m;
    const char* q;
    int64_t q_T, q_H;
    const char* k;
    int64_t k_P, k_S, k_H;
    const float* lse;
    int64_t l_T, l_H;
    float* mass;
    int64_t m_P, m_S, m_H;
    float* ws;
    int32_t Dk;
    int32_t slots, share;    // workgroups of one key head aimed at (0: one to a sequence); see AttnArgs
    int32_t units;           // workgroups of one key head launched
    float c;
    float lmul;              // log2(e), or 1 for base 2
};
struct MassPlan {
    bool few;                // few rows to a sequence
    int32_t slots, share, units;
    int64_t ws_bytes;
};
MassPlan plan_mass(const Batch& m, int Dk, bool pieces);
hipError_t launch_mass(const MassArgs& a, bool few, bool bf16, bool kv8, hipStream_t stream);

struct RopeArgs {
    const char *q, *k, *v;
    int64_t q_T, q_H, k_T, k_H, v_T, v_H;
    const char *wq, *wk;
    const int32_t* pos;
    const float* cs;
    int64_t cs_P;
    const int64_t* slots;
    char *qo, *kc, *vc;
    int64_t qo_T, qo_H, kc_P, kc_S, kc_H, vc_P, vc_S, vc_H;
    float* mass;             // nullable; strides in words
    int64_t m_P, m_S, m_H;
    int32_t T, Hq, Hkv, D, Dv, nq, nk, off, rot, pairs;
    int32_t positions, page_size;
    int64_t slots_max;
    FastDiv fheads;          // heads of a token, queries, keys and values together
    float eps, ik, iv;       // eps, 1 / k_scale, 1 / v_scale
};
hipError_t launch_rope(const RopeArgs& a, bool bf16, bool kv8, hipStream_t stream);

struct EvictArgs {
    char* mass;
    int64_t m_P, m_S, m_H;   // words
    char *k, *v;
    int64_t k_P, k_S, k_H, v_P, v_S, v_H;
    const int32_t *table, *kv, *dst;
    int64_t t_B, d_B;
    int32_t* new_len;
    int32_t* kept;
    int64_t kp_B, kp_H;
    int32_t B, Hkv, k_bytes, v_bytes, pages, page_size, max_keys;
    int32_t budget, sink, recent;
    bool wide;               // rows and strides are 16-byte aligned (else 8)
    FastDiv fpage, fHkv, fbudget;
};
hipError_t launch_evict(const EvictArgs& a, hipStream_t stream);

// Launch kernel(arg) and return that launch's own status.
template <typename Arg>
inline hipError_t launch(void (*kernel)(Arg), dim3 grid, dim3 block, hipStream_t stream, const Arg& arg) {
    void* args[] = {const_cast<Arg*>(&arg)};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, args, 0, stream);
}

}  // namespace dcpa
