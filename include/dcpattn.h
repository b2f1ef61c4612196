/*
 * dcpattn.h -- C ABI of libdcpattn, the attention side of a decode-context-
 * parallel (DCP) rank on AMD Instinct MI355X (gfx950).
 *
 * Under DCP a sequence's keys and values are dealt out over N ranks in blocks
 * of `interleave` positions: position p lies on rank (p / interleave) % N.
 * Each rank keeps its share in a paged cache.  The calls here are what a step and
 * its layers do around the merge of dcpmerge.h:
 *
 *   dcpa_batch_plan           a step's lengths, page tables, positions and slots
 *   dcpa_qk_norm_rope_append  norm and rotate new queries and keys, write the
 *                             keys and values this rank owns into its cache
 *   dcpa_paged_attn           attention of new tokens over the rank's cache:
 *                             the partial output and LSE that dcp_pack takes
 *   dcpa_prefix_attn          the same for sequences that share their first keys,
 *                             which are read once for all of a group
 *   dcpa_project              the projections on both sides of latent attention
 *   dcpa_latent_expand        keys and values of all heads from latent rows
 *   dcpa_pair_attn            attention over keys and values in two 16-bit parts,
 *                             as the expansion makes them
 *   dcpa_latent_attn          the two in one call: latent attention in its expanded form
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
 * dcpa_prefix_attn
 *
 * dcpa_paged_attn for a batch whose sequences share the first keys of their
 * caches: the same result from the same arguments, with the shared keys read once
 * for all rows of a group.  Group g is the sequences cu_group[g] ..
 * cu_group[g+1]-1; the first shared_len[g] cached keys of all of them are the
 * same (whole pages that stand in all their table rows), and are read through the
 * table row of the first of them whose kv_len is shared_len[g] or more (of the
 * longest, if there is none).  shared_len[g] is clamped to [0, max_pages *
 * page_size]; a sequence sees of the shared keys what it would see of its own (none
 * where its kv_len is 0).  Sequences outside the groups share nothing.
 * cu_group has to be non-decreasing (as cu_q, other contents give wrong numbers
 * but no access outside the buffers).
 *
 * Sequences of many rows (128 and more of a key head to each on average) gain nothing
 * from it, and neither does a batch without groups: these run as dcpa_paged_attn, every
 * sequence by its own table row.  Else the parts of every row live in `workspace`, whose
 * size dcpa_prefix_attn_workspace gives: about 512 (Dv + 1) bytes for each of
 * Hkv (B + n_groups + R / S + R / 128 + 1024 / Hkv) units, R = T Hq / Hkv, S = 32 where
 * rows are few, else 128 (256 sequences of one token, 64 / 8 heads of 128: 250 MB).  The
 * weights are held as in dcpa_paged_attn: with what their rounding leaves where rows are
 * few (those of a sequence, not of a group) or wide_weights is given, else rounded to
 * `dtype`.  Up to 2^20 groups; the limit of 2^23 workgroups counts the row tiles of
 * sequences and of groups.
 */
int dcpa_prefix_attn(const dcpa_attn_args* a, const int32_t* cu_group, const int32_t* shared_len, int64_t n_groups,
                     void* stream);
int64_t dcpa_prefix_attn_workspace(const dcpa_attn_args* a, int64_t n_groups);

/*
 * dcpa_pair_attn
 *
 * dcpa_paged_attn over keys and values in two 16-bit parts: a key is k plus, in
 * its first Dr columns, k_rest [num_pages, page_size, Hkv, Dr]; a value is v plus
 * v_rest [num_pages, page_size, Hkv, Dv].  Products of both parts go into the same
 * fp32 sums, so scores and outputs are those of the sums of the parts; the
 * weights are held as there, with what their rounding leaves where rows are few (at
 * most 32 to a sequence on average) or wide_weights is given (in the product with the
 * values' first part, not their second).  cache_dtype is dtype, v not NULL, Dk and
 * Dv at most 256, Dr a multiple of 8 up to Dk; the rests' strides are multiples of 8,
 * 16-byte aligned.  A query that is not finite gives NaN.  The workspace query is
 * dcpa_pair_attn_workspace.
 */
int dcpa_pair_attn(const dcpa_attn_args* a, const void* k_rest, int64_t kr_P, int64_t kr_S, int64_t kr_H, int64_t Dr,
                   const void* v_rest, int64_t vr_P, int64_t vr_S, int64_t vr_H, void* stream);
int64_t dcpa_pair_attn_workspace(const dcpa_attn_args* a);

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

/*
 * dcpa_batch_plan
 *
 * What a step of the calls above needs of its batch, from the number of new
 * tokens of each sequence.  seq_len and kv_len hold the lengths before the step
 * (over all ranks; cached on this rank).  For a sequence that goes on, new_len =
 * n >= 0:
 *   seq_out = seq_len + n,  kv_out = kv_len + owned(seq_len + n) - owned(seq_len),
 *   block_table[b, i] for ceil(kv_len / page_size) <= i < ceil(kv_out / page_size)
 *     (and i < max_pages): pages from the end of the free list, in the order of
 *     sequences and places, -1 once it is empty,
 * and its rows are cu_q[b] .. cu_q[b+1]-1 with, for row t, position seq_len + t -
 * cu_q[b], sequence b, and the slot that dcpa_qk_norm_rope_append takes: -1 where
 * another rank owns the position or the table has no page.  The rows from cu_q[B]
 * to T-1 get -1 in all three.  Tokens beyond row T-1, or beyond a length of 2^30 -
 * 1, are not taken: cu_q and the lengths count those that are.
 * new_len < 0: the sequence has ended.  Its lengths become 0, and its pages
 * block_table[b, i] >= 0, keep_pages[b] <= i < ceil(kv_len / page_size), go onto
 * the end of the list, ahead of any page that this call takes (keep_pages NULL:
 * 0; pages in front that others use, or that stay).  Its table row keeps its
 * entries, which no length counts any more.
 * free_pages [free_max] holds free_count[0] pages (clamped to [0, free_max];
 * pages given back beyond free_max are lost); free_count_out is what is left,
 * or, negative, minus the number of pages that were missing.
 *
 * Where caches were cut, kv_len counts what is cached, as in the other calls.
 * seq_out, kv_out and free_count_out may be the inputs themselves; other
 * overlaps of outputs with inputs or each other are not allowed (partial ones of
 * the lengths: DCPA_ERR_VALUE).  T up to 2^30 rows, free_max below 2^31; B = 0
 * and T = 0 are no special cases (cu_q[0], the rows' padding and the count are
 * written).
 */
typedef struct {
    const int32_t* new_len;                /* [B] */
    const int32_t* seq_len;                /* [B] */
    const int32_t* kv_len;                 /* [B] */
    const int32_t* keep_pages;             /* [B], nullable */
    int32_t* block_table; int64_t t_B;     /* [B, max_pages] */
    int32_t* free_pages;                   /* [free_max] */
    const int32_t* free_count;             /* [1] */
    int32_t* free_count_out;               /* [1] */
    int32_t* seq_out;                      /* [B] */
    int32_t* kv_out;                       /* [B] */
    int32_t* cu_q;                         /* [B + 1] */
    int32_t* positions;                    /* [T] */
    int32_t* sequence;                     /* [T] */
    int64_t* slots;                        /* [T] */
    int64_t B, T, max_pages, page_size, free_max, N, rank, interleave;
} dcpa_plan_args;
int dcpa_batch_plan(const dcpa_plan_args* a, void* stream);

/*
 * dcpa_project
 *
 * The projections on both sides of latent attention, head by head:
 *   y[t, h, n] = sum_{k < K} x[t, h, k] w[h, n, k]      n < N
 *   y[t, h, N + c] = x[t, h, K + c]                      c < copy
 * Queries [nope | rope] into latent space: w the heads' key weights [Dn, Dc] with
 * K = Dn, N = Dc, copy = Dr.  Latent outputs to values: w the value weights
 * [Dv, Dc] with K = Dc, N = Dv, copy = 0.  Sums in fp32, each result rounded
 * once; the copied columns keep their bits.
 *
 * dtype: DCP_F16 or DCP_BF16 (x, w, y).  N and K multiples of 8 up to 1024,
 * copy a multiple of 8 up to 1024, H up to 2^16, T * H up to 2^30.  One of w_N
 * and w_K is 1, the other a multiple of 8; the other strides are multiples of
 * 8, x, w and y 16-byte aligned.  y overlaps neither x nor w.
 */
typedef struct {
    const void* x;        int64_t x_T, x_H;
    const void* w;        int64_t w_H, w_N, w_K;
    void* y;              int64_t y_T, y_H;
    int64_t T, H, N, K, copy, dtype;
} dcpa_project_args;
int dcpa_project(const dcpa_project_args* a, void* stream);

/*
 * dcpa_latent_expand
 *
 * Keys and values of every head from cached latent rows c = [latent Dc | rope Dr]
 * (the cache of the latent layout, one key head): for cached key j < kv_len[b]
 *   k[b, j, h] = k_scale [ sum_c w_k[h, n, c] c_j[c]  (n < Dn) | c_j[Dc ..] (Dr) ]
 *   v[b, j, h] = k_scale sum_c w_v[h, n, c] c_j[c]             (n < Dv)
 * Sums in fp32, each result rounded once to dtype.  k_rest and v_rest (both or
 * neither) get what that rounding left of the sums, rounded once more, so that
 * the two together hold a result to 2^-16 (bf16) or 2^-22 (fp16, or 2^-25) of itself: keys
 * and values for dcpa_pair_attn.  A result beyond the type's largest number is infinite,
 * with a rest of 0.  (The columns of the rope have none: with k_scale = 1 they are
 * exact.)  kv_len is clamped to max_keys and to max_pages * page_size.  Rows behind
 * kv_len, and keys whose page is missing, are left as they were.
 *
 * places [B, max_keys] (nullable) gets b * max_keys + j for every such key, -1
 * where its page is missing: the block_table with which dcpa_paged_attn reads k and
 * v as caches of B * max_keys pages of one key (where they are contiguous over b).
 *
 * dtype: DCP_F16 or DCP_BF16 (w_k, w_v, k, v); cache_dtype dtype or
 * DCP_FP8_E4M3.  Dn, Dv multiples of 8 up to 512, Dr a multiple of 8 (0: none),
 * Dc a multiple of 8, Dc + Dr <= 576.  Weight rows are contiguous over Dc, all
 * strides multiples of 8, all buffers 16-byte aligned, B * max_keys below 2^30.
 * The outputs overlap neither each other nor the inputs.
 */
typedef struct {
    const void* cache;    int64_t c_P, c_S;       /* [num_pages, page_size, Dc + Dr] */
    const int32_t* block_table; int64_t t_B;
    const int32_t* kv_len;                        /* [B] */
    const void* w_k;      int64_t wk_H, wk_N;     /* [H, Dn, Dc] */
    const void* w_v;      int64_t wv_H, wv_N;     /* [H, Dv, Dc] */
    void* k;              int64_t k_B, k_S, k_H;  /* [B, max_keys, H, Dn + Dr] */
    void* v;              int64_t v_B, v_S, v_H;  /* [B, max_keys, H, Dv] */
    void* k_rest;         int64_t kr_B, kr_S, kr_H; /* [B, max_keys, H, Dn], nullable */
    void* v_rest;         int64_t vr_B, vr_S, vr_H; /* [B, max_keys, H, Dv], nullable */
    int32_t* places;      int64_t p_B;
    int64_t B, H, Dn, Dr, Dv, Dc, max_keys, num_pages, page_size, max_pages, dtype, cache_dtype;
    double k_scale;
} dcpa_expand_args;
int dcpa_latent_expand(const dcpa_expand_args* a, void* stream);

/*
 * dcpa_latent_attn
 *
 * dcpa_latent_expand and then attention over what it made, by dcpa_pair_attn where
 * k_rest and v_rest are given, else by dcpa_paged_attn.  The checks of both are made
 * before either is enqueued: on an error k, v, the rests and places are as they were.
 * `a` has q, cu_q, seq_len, out, lse, workspace, T, Hq, the ranks, causal, dtype (e's),
 * lse_base, wide_weights and scale; B is that of e.  Its other fields are ignored: keys,
 * values, lengths, heads, columns and the scale (of both keys and values) are those of
 * e, whose places are needed and whose k, v and rests are contiguous over b (k_B =
 * max_keys * k_S; so for each).  k_scale = f 2^p with the power of two p that makes 1
 * <= f < 2, held to [-15, 7] (a 16-bit cache: [-15, 0]): the keys and values that
 * are written are those divided by f, which goes to the scores and the outputs.  The
 * columns of the rope are exact in them (but for an fp16 cache with k_scale < 1,
 * where they are off by up to 2^-25).  The workspace query takes the same
 * arguments (k_rest NULL or not; other pointers may be NULL).
 */
int dcpa_latent_attn(const dcpa_expand_args* e, const dcpa_attn_args* a, void* stream);
int64_t dcpa_latent_attn_workspace(const dcpa_expand_args* e, const dcpa_attn_args* a);

#ifdef __cplusplus
}
#endif

#endif /* DCPATTN_H */
