/*
 * dcpattn.h -- C ABI of libdcpattn, the attention side of a decode-context-
 * parallel (DCP) rank on AMD Instinct MI355X (gfx950).
 *
 * Under DCP a sequence's keys and values are dealt out over N ranks in blocks
 * of `interleave` positions: position p lies on rank (p / interleave) % N.
 * Each rank keeps its share in a paged cache.  The four calls here are what a
 * layer does around the merge of dcpmerge.h:
 *
 *   dcpa_qk_norm_rope_append  norm and rotate new queries and keys, write the
 *                             keys and values this rank owns into its cache
 *   dcpa_paged_attn           attention of new tokens over the rank's cache:
 *                             the partial output and LSE that dcp_pack takes
 *   dcpa_attn_mass            accumulate the attention weight of each cached
 *                             key from the merged LSE of dcp_unpack_combine
 *   dcpa_cache_evict          keep the keys of highest accumulated weight:
 *                             gather them into new pages
 *
 * The conventions of dcpmerge.h hold: caller-owned device memory of the
 * current device, nothing allocated, no synchronisation and no state, work
 * only on `stream`, every check on the host before anything is enqueued (on
 * an error nothing is written), strides >= 0 in elements of the tensor's own
 * type, the innermost dimension contiguous, status codes of dcpmerge.h and
 * the two below.  Results are deterministic: no floating-point atomics, every
 * sum in an order fixed by the call's sizes.
 *
 * Arguments travel in a struct of 8-byte fields.
 *
 * Paged cache.  keys [num_pages, page_size, Hkv, Dk] and values [num_pages,
 * page_size, Hkv, Dv], any strides whose rows start 8-element aligned.  Cached
 * token j of sequence b lives in page block_table[b, j / page_size] at place
 * j % page_size.  v == NULL: values are the first Dv columns of the keys (the
 * latent layout).  cache_dtype is the payload dtype or DCP_FP8_E4M3; an 8-bit
 * cache stands for its values times k_scale / v_scale.  A block_table entry
 * outside [0, num_pages) is never followed: its keys are not there.
 *
 * Device-side lengths.  Sequence b's new tokens are rows cu_q[b] ..
 * cu_q[b+1]-1 of q; rows before cu_q[0] or from cu_q[B] on are left as they
 * were.  kv_len[b] is the rank's cached length after this step's keys were
 * written; it is clamped to [0, max_pages * page_size].  seq_len[b] is the
 * sequence's whole length over all ranks after this step.  cu_q has to be
 * non-decreasing; any other contents of these arrays give wrong numbers but no
 * access outside the buffers.
 *
 * Causal order.  The last token of sequence b stands at position seq_len[b]-1,
 * its n new tokens at the last n positions.  A token at position t sees the
 * rank's cached keys but those it owns at positions t+1 .. seq_len[b]-1, which
 * are the last ones cached:
 *   visible = kv_len[b] - (owned(seq_len[b]) - owned(t + 1)),
 *   owned(x) = number of positions below x that lie on this rank.
 * So a cache that dcpa_cache_evict has cut stays usable.  With causal = 0 every
 * token sees all kv_len[b] keys (an encoder's states, say).
 *
 * Limits (DCP_ERR_SHAPE beyond them): heads up to 2^16, sequences up to 2^20,
 * T * Hq up to 2^30 (T * (Hq + 2 Hkv) in the first call), max_pages *
 * page_size below 2^30, page_size up to 2^20, N * interleave up to 2^30; the
 * attention and the weights up to 2^23 workgroups (row tiles of 128 rows, of 32
 * where rows are few, times key heads, at least one to a sequence), the eviction
 * up to B * Hkv = 2^21 and B * Hkv * budget = 2^28.
 */
#ifndef DCPATTN_H
#define DCPATTN_H

#include <stdint.h>

#include "dcpmerge.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    DCPA_ERR_WORKSPACE = -20, /* workspace too small, missing or not 16-byte aligned */
    DCPA_ERR_VALUE = -21      /* a scale, eps or count outside its range             */
};

/* Static, human-readable text of a status code of this library. */
const char* dcpa_status_str(int status);

/*
 * dcpa_qk_norm_rope_append
 *
 * Per row x of D elements (one head of one token), in fp32:
 *   a_i = x_i * w_i / sqrt(mean_{i<Dn} x_i^2 + eps)   for i < Dn (Dn = 0: no norm)
 *   a_i = x_i                                         for i >= Dn
 * then the `rot` columns from rope_off on are turned by the angles of the
 * token's position p: with (c, s) = cos_sin[p, j], cos_sin[p, rot/2 + j],
 *   (u, v) <- (u c - v s, v c + u s)
 * where (u, v) are columns (j, j + rot/2) of the range, or (2j, 2j+1) if
 * interleaved != 0.  Each result is rounded once.
 *
 * q [T, Hq, D] -> q_out [T, Hq, D] (may be q itself, with the same strides), normed by
 * q_weight [q_norm].  k [T, Hkv, D], normed by k_weight [k_norm], goes to the
 * cache row slots[t] = page * page_size + place; v [T, Hkv, Dv] (nullable) goes
 * to the value cache unchanged but for its type.  A slot outside [0, num_pages
 * * page_size) is skipped: another rank owns that token.  Slots of one call
 * must differ.  mass (nullable, strides m_P, m_S, m_H in words, laid out as
 * dcpa_attn_mass takes it): the weight of every key that is written starts at 0.
 * An 8-bit cache stores x * (1 / scale) in fp32, rounded to
 * nearest even and saturated at 448.  A position outside [0, positions_max)
 * turns by the nearest row of the table.
 *
 * dtype: DCP_F16 or DCP_BF16 (q, k, v, weights).  D, Dv multiples of 8 up to
 * 1024, rope_off a multiple of 8, rot a multiple of 8 (0: no rotation), rows
 * of q, k, v and q_out 16-byte aligned, rows of a cache 8-element aligned;
 * q_norm and k_norm are 0 or multiples of 8 up to D.
 */
typedef struct {
    const void* q;        int64_t q_T, q_H;
    const void* k;        int64_t k_T, k_H;
    const void* v;        int64_t v_T, v_H;
    const void* q_weight; const void* k_weight;
    const int32_t* positions;              /* [T] */
    const float* cos_sin; int64_t cs_P;    /* [positions_max, rot] */
    const int64_t* slots;                  /* [T] */
    void* q_out;          int64_t qo_T, qo_H;
    void* k_cache;        int64_t kc_P, kc_S, kc_H;
    void* v_cache;        int64_t vc_P, vc_S, vc_H;
    float* mass;          int64_t m_P, m_S, m_H;
    int64_t T, Hq, Hkv, D, Dv, q_norm, k_norm, rope_off, rot, interleaved;
    int64_t positions_max, num_pages, page_size, dtype, cache_dtype;
    double eps, k_scale, v_scale;
} dcpa_rope_args;
int dcpa_qk_norm_rope_append(const dcpa_rope_args* a, void* stream);

/*
 * dcpa_paged_attn
 *
 * For token row t of sequence b, head h with key head h / (Hq / Hkv), over the
 * visible keys j:
 *   s_j = scale * <q[t, h], key_j>
 *   lse[t, h] = log_beta sum_j e^(s_j)          (beta: lse_base)
 *   out[t, h] = sum_j e^(s_j - log sum e^s) value_j
 * A row that sees no key gets the neutral pair out = 0, lse = -inf.  A row
 * that sees a score of NaN or +inf gets NaN in both.  What a row does not see
 * (masked keys, places behind kv_len, missing pages) never reaches it,
 * whatever bits lie there.
 *
 * Scores, sums and outputs are accumulated in fp32; the weights are rounded
 * to `dtype` for the product with the values, the output once to `dtype`.  Where
 * rows are few (at most 32 to a sequence on average, rows of a token in one key
 * head counted, Dk and Dv up to 256 and in 8 bits multiples of 16) what that
 * rounding leaves of a weight goes through a second product, so that a weight is
 * held to 2^-16 (bf16) or 2^-22 (fp16) of itself.  wide_weights != 0 asks for the
 * same in every other case, where matrix products bound the call and it takes
 * 1.2 to 1.4 times as long.
 *
 * dtype: DCP_F16 or DCP_BF16 (q, out).  Hq a multiple of Hkv.  Dk, Dv
 * multiples of 8, at most 256, or in the latent layout (v == NULL) Dk <= 576,
 * Dv <= 512, Dv <= Dk.  q rows 16-byte aligned, caches 16-byte aligned with
 * rows 8 elements aligned, out rows 4-byte aligned.  scale, k_scale and v_scale positive and finite.
 *
 * Where rows are few, the keys are split over workgroups and joined by a
 * second kernel; the split parts live in `workspace`, whose size
 * dcpa_paged_attn_workspace gives for the same arguments (pointers may be
 * NULL there; 0: none needed; < 0: the status of the refusal).
 */
typedef struct {
    const void* q;        int64_t q_T, q_H;
    const void* k;        int64_t k_P, k_S, k_H;
    const void* v;        int64_t v_P, v_S, v_H;
    const int32_t* block_table; int64_t t_B;
    const int32_t* cu_q;                   /* [B + 1] */
    const int32_t* kv_len;                 /* [B] */
    const int32_t* seq_len;                /* [B]; may be NULL if N == 1 or not causal */
    void* out;            int64_t o_T, o_H;
    float* lse;           int64_t l_T, l_H;   /* [T, Hq] words, nullable */
    void* workspace;      int64_t workspace_bytes;
    int64_t B, T, Hq, Hkv, Dk, Dv, num_pages, page_size, max_pages;
    int64_t N, rank, interleave, causal, dtype, cache_dtype, lse_base, wide_weights;
    double scale, k_scale, v_scale;
} dcpa_attn_args;
int dcpa_paged_attn(const dcpa_attn_args* a, void* stream);
int64_t dcpa_paged_attn_workspace(const dcpa_attn_args* a);

/*
 * dcpa_attn_mass
 *
 * mass[page, place, hk] += sum over the rows (t, h) of the sequence with key
 * head hk that see the key, of e^(s_j - lse[t, h] ln beta), with s_j as above
 * and lse the merged log-sum-exp over all ranks (so that the weights of one
 * row over all ranks sum to 1).  A row whose lse is -inf adds nothing.  The
 * call takes the fields of dcpa_attn_args it needs: v, Dv, v_scale (positive
 * all the same), out and wide_weights are ignored, lse is read.  mass holds fp32 with strides
 * m_P, m_S, m_H; a place's weight has to be 0 when a key is first written there,
 * which dcpa_qk_norm_rope_append sees to if it is given mass.  A page must not stand twice in the table rows of one call
 * (two sequences that share a page: two calls).  `workspace` holds the parts of
 * rows that are split over workgroups, dcpa_attn_mass_workspace gives its size.
 */
int dcpa_attn_mass(const dcpa_attn_args* a, float* mass, int64_t m_P, int64_t m_S, int64_t m_H, void* stream);
int64_t dcpa_attn_mass_workspace(const dcpa_attn_args* a);

/*
 * dcpa_cache_evict
 *
 * Of each sequence's L = kv_len[b] cached keys, every key head keeps n =
 * min(L, budget): the first n_sink, the last n_recent, and of the others those
 * of highest mass (NaN above all numbers, ties to the lowest index).  The kept
 * keys, in their old order, are copied to places 0 .. n-1 of the pages
 * dst_table[b, :], with their values (v nullable) and their mass.  kept[b, h,
 * i] is the old index of the i-th, -1 from n on; new_len[b] = n (new_len may be
 * kv_len itself, else the two arrays must lie apart: DCPA_ERR_VALUE).
 *
 * The other places of the destination pages keep what they hold, old weights too
 * (see mass in dcpa_qk_norm_rope_append).
 * Source pages are only read: destination pages must not be source pages of
 * any sequence of the call, nor appear twice.  A destination entry outside
 * [0, num_pages) drops its rows; a missing source page's keys count as mass
 * -inf and copy as zeros.  esize is the cache's element size (1, 2 or 4
 * bytes), row strides and D * esize multiples of 8 bytes.  n_sink + n_recent
 * <= budget <= dst_pages * page_size.
 */
typedef struct {
    float* mass;          int64_t m_P, m_S, m_H;
    void* k;              int64_t k_P, k_S, k_H;
    void* v;              int64_t v_P, v_S, v_H;
    const int32_t* block_table; int64_t t_B;
    const int32_t* kv_len;
    const int32_t* dst_table;   int64_t d_B;
    int32_t* new_len;
    int32_t* kept;        int64_t kp_B, kp_H;
    int64_t B, Hkv, Dk, Dv, esize, num_pages, page_size, max_pages, dst_pages;
    int64_t budget, n_sink, n_recent;
} dcpa_evict_args;
int dcpa_cache_evict(const dcpa_evict_args* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DCPATTN_H */
