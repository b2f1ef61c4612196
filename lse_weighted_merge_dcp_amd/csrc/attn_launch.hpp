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

// Attention over keys and values in two parts, the second what the rounding of the first left.
struct PairArgs : AttnArgs {
    const char* kr;          // the first Dr columns of the keys
    int64_t kr_P, kr_S, kr_H;
    const char* vr;
    int64_t vr_P, vr_S, vr_H;
    int32_t Dr;
};
AttnPlan plan_pairs(const Batch& m, int Dv);
hipError_t launch_pairs(const PairArgs& a, const AttnPlan& pl, bool bf16, bool wide, hipStream_t stream);
// Joins the split rows of launch_attn() (step: keys of a tile).
hipError_t join_rows(const AttnArgs& a, int step, bool bf16, hipStream_t stream);

// Attention of sequences that share their first keys, group by group.  Lists that
// its first kernel leaves in the workspace: units of work, and where the units of
// each group and then each sequence stand.
struct PrefixUnit {
    int32_t b;                           // table row
    int32_t first, n, kv, len;           // rows and lengths (of the group: first row, rows, shared keys)
    int32_t begin, end;                  // keys
    int32_t tile, split, splits, chunk;
    int32_t b0, b1;                      // sequences of a group (else none)
    int32_t even;                        // all rows see all shared keys
    int32_t unused[2];
};
struct PrefixEntry {
    int32_t first, n, slot, splits, begin, kv, len, chunk;
};
struct GroupArgs : AttnArgs {
    const int32_t* cug;      // [groups + 1]: sequences
    const int32_t* same;     // [groups]: shared keys
    PrefixUnit* list;        // [units]
    PrefixEntry* entries;    // [groups + B]
    int32_t groups, step;    // step: keys of a tile
    int32_t own_rows;        // rows of a tile of a sequence against its own keys (`rows`, or 32 where they are few)
};
hipError_t launch_prefix_bf16(const GroupArgs& a, bool kv8, bool wide, hipStream_t stream);
hipError_t launch_prefix_f16(const GroupArgs& a, bool kv8, bool wide, hipStream_t stream);
int64_t prefix_list_bytes(int64_t units, int64_t entries);
// Whether the keys that groups share are read for all their rows at once, or by each sequence for itself
// (launch_attn()).  From whole tiles of rows to a sequence on (128 rows of a key head, on average) a tile that holds
// rows of several sequences saves no matrix instruction, but every row's parts go through memory: 24 chunks to 2048
// tokens behind 8192 keys (2048 here), 64 / 8 heads, took 5150 us and 2.0 GB of workspace, 2230 us and none by
// themselves; 64 sequences of 16 tokens behind 8192 keys here 386 and 295 us, of 8 tokens 218 and 238.  (8-bit rows lose
// up to a tenth so: 64 of 16 tokens 410 and 441 us, behind 1024 keys 157 and 85.)
inline bool sharing_pays(const Batch& m, int64_t groups) { return groups > 0 && (int64_t)m.T * m.G < (int64_t)128 * m.B; }
AttnPlan plan_prefix(const Batch& m, int64_t groups, int Dk, int Dv, bool pieces);
hipError_t launch_prefix(const GroupArgs& a, bool latent, bool bf16, bool kv8, bool wide, hipStream_t stream);

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

struct PlanArgs {
    const int32_t *new_len, *seq, *kv, *keep;   // keep: nullable
    int32_t* table;
    int64_t t_B;
    int32_t* free;
    const int32_t* count;
    int32_t *count_out, *seq_out, *kv_out, *cu, *positions, *sequence;
    int64_t* slots;
    int32_t B, T, width, page_size, free_max, N, rank, inter;
    int32_t rows_here;       // up to as many token rows are done by the kernel of the lengths
    FastDiv fpage, fblock;
};
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream);

// y[t, h] = x[t, h] W[h], and columns that are copied.
struct ProjectArgs {
    const char *x, *w;
    char* y;
    int64_t x_T, x_H, w_H, w_N, w_K, y_T, y_H;
    int32_t T, H, N, K, copy;
    int32_t tiles, each;     // each: tiles of a workgroup
    FastDiv fH, fnt;         // fnt: column tiles
};
// turned: the weights of a head lie as [K][N] (else as [N][K]).
hipError_t launch_project(const ProjectArgs& a, bool turned, bool bf16, hipStream_t stream);
int64_t project_tiles(int64_t T, int64_t H, int64_t N);

struct ExpandArgs {
    const char* cache;
    int64_t c_P, c_S;
    const int32_t* table;
    int64_t t_B;
    const int32_t* kv;
    const char *wk, *wv;
    int64_t wk_H, wk_N, wv_H, wv_N;
    char *ko, *vo;
    int64_t ko_B, ko_S, ko_H, vo_B, vo_S, vo_H;
    char *kr, *vr;           // what the rounding leaves; null: not asked for
    int64_t kr_B, kr_S, kr_H, vr_B, vr_S, vr_H;
    int32_t* places;         // nullable
    int64_t pl_B;
    int32_t B, H, Dn, Dr, Dv, Dc;
    int32_t most, keys;      // rows of the outputs; of these, what the page table can name
    int32_t pages, nt;       // nt: column tiles
    FastDiv fpage, fper;     // fper: Dn + Dv
    float ks;
};
hipError_t launch_expand(const ExpandArgs& a, bool bf16, bool x8, hipStream_t stream);
int64_t expand_workgroups(int64_t B, int64_t most, bool rest);

// Launch kernel(arg) and return that launch's own status.
template <typename Arg>
inline hipError_t launch(void (*kernel)(Arg), dim3 grid, dim3 block, hipStream_t stream, const Arg& arg) {
    void* args[] = {const_cast<Arg*>(&arg)};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, args, 0, stream);
}

}  // namespace dcpa
