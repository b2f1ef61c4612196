// attn_api.cpp -- the C ABI of libdcpattn (declared in include/dcpattn.h).
//
// As in api.cpp every check runs on the host before anything is enqueued, and
// the calls keep no state.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/dcpattn.h"
#include "attn_launch.hpp"

namespace {

using namespace dcpa;

constexpr int64_t kMaxStride = int64_t(1) << 56;
constexpr int64_t kMaxSpan = int64_t(1) << 60;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxGrid = int64_t(1) << 23;   // workgroups of a launch (2^31 work-items)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

int esize_of(int64_t dtype) { return dtype == DCP_F16 || dtype == DCP_BF16 ? 2 : dtype == DCP_FP8_E4M3 ? 1 : 0; }
bool aligned(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
bool multiples(std::initializer_list<int64_t> xs, int64_t a) {
    for (int64_t x : xs)
        if (x % a != 0) return false;
    return true;
}
bool strides_ok(std::initializer_list<int64_t> xs) {
    for (int64_t x : xs)
        if (x < 0 || x > kMaxStride) return false;
    return true;
}
struct Dim {
    int64_t n, s;
};
bool span_ok(std::initializer_list<Dim> dims, int64_t esize) {
    int64_t span = 0;
    for (const Dim& d : dims) {
        if (d.n <= 1 || d.s == 0) continue;
        if (d.n - 1 > kMaxSpan / (d.s * esize)) return false;
        span += (d.n - 1) * d.s * esize;
        if (span >= kMaxSpan) return false;
    }
    return true;
}
bool positive(double x) { return x > 0.0 && x <= 3.0e38 && (float)x > 0.0f; }
int status(hipError_t e) { return e == hipSuccess ? DCP_OK : DCP_ERR_LAUNCH; }

bool cache_shape_ok(int64_t pages, int64_t page_size, int64_t max_pages) {
    return pages >= 0 && pages < (int64_t(1) << 31) && page_size >= 1 && page_size <= (int64_t(1) << 20) &&
           max_pages >= 0 && max_pages < (int64_t(1) << 31) && max_pages * page_size < (int64_t(1) << 30);
}

bool ranks_ok(int64_t N, int64_t rank, int64_t inter) {
    return N >= 1 && N <= (1 << 20) && rank >= 0 && rank < N && inter >= 1 && inter <= (1 << 20) &&
           N * inter <= (int64_t(1) << 30);
}
uintptr_t apart(uintptr_t x, uintptr_t y) { return x < y ? y - x : x - y; }

// The checks that the attention and the weights share; fills `m`.
int check_batch(const dcpa_attn_args* a, Batch& m) {
    if (a->dtype != DCP_F16 && a->dtype != DCP_BF16) return DCP_ERR_DTYPE;
    if (a->cache_dtype != a->dtype && a->cache_dtype != DCP_FP8_E4M3) return DCP_ERR_DTYPE;
    if (a->lse_base != DCP_LSE_BASE_E && a->lse_base != DCP_LSE_BASE_2) return DCP_ERR_LSE_BASE;
    if (a->B < 0 || a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hkv > a->Hq || a->Hq > (1 << 16) ||
        a->B > (int64_t(1) << 20) || a->T > kMaxRows || a->T * a->Hq > kMaxRows)
        return DCP_ERR_SHAPE;
    if (a->Hq % a->Hkv != 0) return DCP_ERR_HEADS_NOT_DIVISIBLE;
    if (a->Dk < 8 || a->Dk % 8 != 0 || a->Dk > 576) return DCP_ERR_SHAPE;
    if (!cache_shape_ok(a->num_pages, a->page_size, a->max_pages)) return DCP_ERR_SHAPE;
    if (!ranks_ok(a->N, a->rank, a->interleave)) return DCP_ERR_SHAPE;
    if (!positive(a->scale) || !positive(a->k_scale) || !positive(a->v_scale) ||
        !positive(a->scale * a->k_scale * 1.4426950408889634))
        return DCPA_ERR_VALUE;
    if (!strides_ok({a->q_T, a->q_H, a->k_P, a->k_S, a->k_H, a->t_B, a->l_T, a->l_H})) return DCP_ERR_STRIDE;
    const int ec = esize_of(a->cache_dtype);
    if (!span_ok({{a->T, a->q_T}, {a->Hq, a->q_H}, {a->Dk, 1}}, 2) ||
        !span_ok({{a->num_pages, a->k_P}, {a->page_size, a->k_S}, {a->Hkv, a->k_H}, {a->Dk, 1}}, ec) ||
        !span_ok({{a->B, a->t_B}, {a->max_pages, 1}}, 4) || !span_ok({{a->T, a->l_T}, {a->Hq, a->l_H}}, 4))
        return DCP_ERR_STRIDE;
    m.table = a->block_table;
    m.t_B = a->t_B;
    m.cu = a->cu_q;
    m.kv = a->kv_len;
    m.causal = a->causal != 0;
    // one rank owns every position: the keys hidden from a token are just the new tokens behind it
    m.seq = a->causal && a->N > 1 ? a->seq_len : nullptr;
    m.B = (int32_t)a->B;
    m.T = (int32_t)a->T;
    m.G = (int32_t)(a->Hq / a->Hkv);
    m.Hkv = (int32_t)a->Hkv;
    m.pages = (int32_t)a->num_pages;
    m.page_size = (int32_t)a->page_size;
    m.max_keys = (int32_t)(a->max_pages * a->page_size);
    m.N = (int32_t)a->N;
    m.rank = (int32_t)a->rank;
    m.inter = (int32_t)a->interleave;
    m.fG = dcp::make_fastdiv((uint32_t)m.G);
    m.fpage = dcp::make_fastdiv((uint32_t)m.page_size);
    m.fHkv = dcp::make_fastdiv((uint32_t)m.Hkv);
    m.fblock = dcp::make_fastdiv((uint32_t)(m.N * m.inter));
    return DCP_OK;
}

// Whether key rows are whole pieces of 16 bytes.
bool key_pieces(const dcpa_attn_args* a) {
    return a->cache_dtype != DCP_FP8_E4M3 || multiples({a->Dk, a->k_P, a->k_S, a->k_H}, 16);
}
bool cache_pieces(const dcpa_attn_args* a) {
    return key_pieces(a) && (a->cache_dtype != DCP_FP8_E4M3 ||
                             (a->Dv % 16 == 0 && (!a->v || multiples({a->v_P, a->v_S, a->v_H}, 16))));
}
AttnPlan plan_of(const dcpa_attn_args* a, const Batch& m) { return plan_attn(m, (int)a->Dk, (int)a->Dv, cache_pieces(a)); }

// Pointers and alignment of what both calls read.
int check_inputs(const dcpa_attn_args* a) {
    if (!a->q || !a->cu_q || !a->kv_len || (a->max_pages > 0 && !a->block_table) || (a->num_pages > 0 && !a->k) ||
        (a->causal && a->N > 1 && !a->seq_len))
        return DCP_ERR_NULL;
    if (!aligned(a->q, 16) || !multiples({a->q_T, a->q_H}, 8) || !aligned(a->k, 16) ||
        !multiples({a->k_P, a->k_S, a->k_H}, 8) || !aligned(a->block_table, 4) || !aligned(a->cu_q, 4) ||
        !aligned(a->kv_len, 4) || !aligned(a->seq_len, 4) || !aligned(a->lse, 4))
        return DCP_ERR_ALIGN;
    return DCP_OK;
}

int check_shapes(const dcpa_attn_args* a, Batch& m) {
    if (int st = check_batch(a, m)) return st;
    const bool shared = a->v == nullptr;
    if (a->Dv < 8 || a->Dv % 8 != 0 || a->Dv > 512) return DCP_ERR_SHAPE;
    if (shared ? a->Dv > a->Dk : a->Dk > 256 || a->Dv > 256) return DCP_ERR_SHAPE;
    if (!strides_ok({a->v_P, a->v_S, a->v_H, a->o_T, a->o_H})) return DCP_ERR_STRIDE;
    if (!span_ok({{a->num_pages, a->v_P}, {a->page_size, a->v_S}, {a->Hkv, a->v_H}, {a->Dv, 1}},
                 esize_of(a->cache_dtype)) ||
        !span_ok({{a->T, a->o_T}, {a->Hq, a->o_H}, {a->Dv, 1}}, 2))
        return DCP_ERR_STRIDE;
    return DCP_OK;
}
// No more workgroups than a launch may have, those that join rows among them.
bool grid_ok(const dcpa_attn_args* a, const AttnPlan& pl, const Batch& m) {
    return ((int64_t)pl.units + 7) * m.Hkv <= kMaxGrid && (pl.slots == 0 || a->T * a->Hq / 4 < kMaxGrid);
}
int check_attn(const dcpa_attn_args* a, Batch& m) {
    if (int st = check_shapes(a, m)) return st;
    return grid_ok(a, plan_of(a, m), m) ? DCP_OK : DCP_ERR_SHAPE;
}
int check_prefix(const dcpa_attn_args* a, int64_t groups, Batch& m, AttnPlan& pl) {
    if (int st = check_shapes(a, m)) return st;
    if (groups < 0 || groups > (int64_t(1) << 20)) return DCP_ERR_SHAPE;
    pl = sharing_pays(m, groups) ? plan_prefix(m, groups, (int)a->Dk, (int)a->Dv, cache_pieces(a)) : plan_of(a, m);
    return grid_ok(a, pl, m) ? DCP_OK : DCP_ERR_SHAPE;
}

int check_pairs(const dcpa_attn_args* a, Batch& m, AttnPlan& pl) {
    if (int st = check_shapes(a, m)) return st;
    if (a->cache_dtype != a->dtype) return DCP_ERR_DTYPE;
    if (a->v == nullptr && a->num_pages > 0) return DCP_ERR_NULL;
    if (a->Dk > 256 || a->Dv > 256) return DCP_ERR_SHAPE;
    pl = plan_pairs(m, (int)a->Dv);
    return grid_ok(a, pl, m) ? DCP_OK : DCP_ERR_SHAPE;
}

// Alignment of what the attention calls write, and of the values.
int check_outputs(const dcpa_attn_args* a) {
    if (!a->out) return DCP_ERR_NULL;
    if (!aligned(a->v, 16) || (a->v && !multiples({a->v_P, a->v_S, a->v_H}, 8)) || !aligned(a->out, 4) ||
        !multiples({a->o_T, a->o_H}, 2))
        return DCP_ERR_ALIGN;
    return DCP_OK;
}
// The arguments of the attention kernels (m is there already); lists: bytes of the workspace in front of the parts.
int fill_attn(const dcpa_attn_args* a, const AttnPlan& pl, AttnArgs& k, int64_t lists = 0) {
    const int ec = esize_of(a->cache_dtype);
    if (pl.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < pl.ws_bytes || !aligned(a->workspace, 16)))
        return DCPA_ERR_WORKSPACE;
    k.q = (const char*)a->q;
    k.q_T = a->q_T * 2; k.q_H = a->q_H * 2;
    k.k = (const char*)a->k;
    k.k_P = a->k_P * ec; k.k_S = a->k_S * ec; k.k_H = a->k_H * ec;
    k.v = (const char*)a->v;
    k.v_P = a->v_P * ec; k.v_S = a->v_S * ec; k.v_H = a->v_H * ec;
    k.out = (char*)a->out;
    k.o_T = a->o_T * 2; k.o_H = a->o_H * 2;
    k.lse = a->lse;
    k.l_T = a->l_T; k.l_H = a->l_H;
    k.Dk = (int32_t)a->Dk;
    k.Dv = (int32_t)a->Dv;
    k.rows = pl.rows;
    k.slots = pl.slots;
    k.share = pl.share;
    k.units = pl.units;
    k.ws_o = (float*)((char*)a->workspace + lists);
    k.ws_l = a->workspace == nullptr ? nullptr : k.ws_o + (int64_t)pl.units * k.m.Hkv * pl.rows * a->Dv;
    k.c = (float)(a->scale * a->k_scale * 1.4426950408889634);
    // (in the latent layout the values are the keys' own columns)
    k.vs = (float)(a->v ? a->v_scale : a->k_scale);
    k.lmul = a->lse_base == DCP_LSE_BASE_E ? kLn2 : 1.0f;
    return DCP_OK;
}

// The checks of an attention call and its arguments; any: there are rows.
int prepare_attn(const dcpa_attn_args* a, AttnArgs& k, AttnPlan& pl, bool& any) {
    any = false;
    if (int st = check_attn(a, k.m)) return st;
    if (a->B == 0 || a->T == 0) return DCP_OK;
    any = true;
    if (int st = check_inputs(a)) return st;
    if (int st = check_outputs(a)) return st;
    pl = plan_of(a, k.m);
    return fill_attn(a, pl, k);
}
int run_attn(const dcpa_attn_args* a, const AttnArgs& k, const AttnPlan& pl, void* stream) {
    return status(launch_attn(k, pl, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, a->wide_weights != 0,
                              (hipStream_t)stream));
}

// The second part of keys or values.
struct Rest {
    const void* at;
    int64_t P, S, H;
};
int prepare_pairs(const dcpa_attn_args* a, const Rest& kr, int64_t Dr, const Rest& vr, PairArgs& k, AttnPlan& pl, bool& any) {
    any = false;
    if (int st = check_pairs(a, k.m, pl)) return st;
    if (Dr < 8 || Dr % 8 != 0 || Dr > a->Dk) return DCP_ERR_SHAPE;
    if (!strides_ok({kr.P, kr.S, kr.H, vr.P, vr.S, vr.H}) ||
        !span_ok({{a->num_pages, kr.P}, {a->page_size, kr.S}, {a->Hkv, kr.H}, {Dr, 1}}, 2) ||
        !span_ok({{a->num_pages, vr.P}, {a->page_size, vr.S}, {a->Hkv, vr.H}, {a->Dv, 1}}, 2))
        return DCP_ERR_STRIDE;
    if (a->B == 0 || a->T == 0) return DCP_OK;
    any = true;
    if (int st = check_inputs(a)) return st;
    if (a->num_pages > 0 && (!kr.at || !vr.at)) return DCP_ERR_NULL;
    if (int st = check_outputs(a)) return st;
    if (!aligned(kr.at, 16) || !aligned(vr.at, 16) || !multiples({kr.P, kr.S, kr.H, vr.P, vr.S, vr.H}, 8)) return DCP_ERR_ALIGN;
    if (int st = fill_attn(a, pl, k)) return st;
    k.kr = (const char*)kr.at;
    k.kr_P = kr.P * 2; k.kr_S = kr.S * 2; k.kr_H = kr.H * 2;
    k.vr = (const char*)vr.at;
    k.vr_P = vr.P * 2; k.vr_S = vr.S * 2; k.vr_H = vr.H * 2;
    k.Dr = (int32_t)Dr;
    return DCP_OK;
}
int run_pairs(const dcpa_attn_args* a, const PairArgs& k, const AttnPlan& pl, void* stream) {
    return status(launch_pairs(k, pl, a->dtype == DCP_BF16, a->wide_weights != 0, (hipStream_t)stream));
}

// What the expansion takes, without its pointers.
int check_expand(const dcpa_expand_args* a) {
    if (a->dtype != DCP_F16 && a->dtype != DCP_BF16) return DCP_ERR_DTYPE;
    if (a->cache_dtype != a->dtype && a->cache_dtype != DCP_FP8_E4M3) return DCP_ERR_DTYPE;
    auto cols = [](int64_t d) { return d >= 8 && d % 8 == 0 && d <= 512; };
    if (a->B < 0 || a->B > (int64_t(1) << 20) || a->H < 1 || a->H > (1 << 16) || !cols(a->Dn) || !cols(a->Dv) ||
        a->Dr < 0 || a->Dr % 8 != 0 || a->Dc < 8 || a->Dc % 8 != 0 || a->Dr > 576 || a->Dc > 576 || a->Dc + a->Dr > 576 ||
        a->max_keys < 0 || a->max_keys >= kMaxRows || a->B * a->max_keys >= kMaxRows ||
        !cache_shape_ok(a->num_pages, a->page_size, a->max_pages))
        return DCP_ERR_SHAPE;
    if (expand_workgroups(a->B, a->max_keys, a->k_rest != nullptr) > kMaxGrid / 2) return DCP_ERR_SHAPE;
    if (!positive(a->k_scale)) return DCPA_ERR_VALUE;
    const int ec = esize_of(a->cache_dtype);
    if (!strides_ok({a->c_P, a->c_S, a->t_B, a->wk_H, a->wk_N, a->wv_H, a->wv_N, a->k_B, a->k_S, a->k_H, a->v_B, a->v_S,
                     a->v_H, a->kr_B, a->kr_S, a->kr_H, a->vr_B, a->vr_S, a->vr_H, a->p_B}) ||
        !span_ok({{a->B, a->kr_B}, {a->max_keys, a->kr_S}, {a->H, a->kr_H}, {a->Dn, 1}}, 2) ||
        !span_ok({{a->B, a->vr_B}, {a->max_keys, a->vr_S}, {a->H, a->vr_H}, {a->Dv, 1}}, 2) ||
        !span_ok({{a->num_pages, a->c_P}, {a->page_size, a->c_S}, {a->Dc + a->Dr, 1}}, ec) ||
        !span_ok({{a->B, a->t_B}, {a->max_pages, 1}}, 4) || !span_ok({{a->B, a->p_B}, {a->max_keys, 1}}, 4) ||
        !span_ok({{a->H, a->wk_H}, {a->Dn, a->wk_N}, {a->Dc, 1}}, 2) ||
        !span_ok({{a->H, a->wv_H}, {a->Dv, a->wv_N}, {a->Dc, 1}}, 2) ||
        !span_ok({{a->B, a->k_B}, {a->max_keys, a->k_S}, {a->H, a->k_H}, {a->Dn + a->Dr, 1}}, 2) ||
        !span_ok({{a->B, a->v_B}, {a->max_keys, a->v_S}, {a->H, a->v_H}, {a->Dv, 1}}, 2))
        return DCP_ERR_STRIDE;
    return DCP_OK;
}
// Its checks and arguments; any: there is something to expand.
int prepare_expand(const dcpa_expand_args* a, ExpandArgs& k, bool& any) {
    any = false;
    if (int st = check_expand(a)) return st;
    if (a->B == 0 || a->max_keys == 0) return DCP_OK;
    any = true;
    if ((a->max_pages > 0 && !a->block_table) || !a->kv_len || !a->w_k || !a->w_v || !a->k || !a->v || (a->num_pages > 0 && !a->cache) || !a->k_rest != !a->v_rest)
        return DCP_ERR_NULL;
    for (const void* x : {a->cache, a->w_k, a->w_v, (const void*)a->k, (const void*)a->v, (const void*)a->k_rest, (const void*)a->v_rest})
        if (!aligned(x, 16)) return DCP_ERR_ALIGN;
    if (!multiples({a->c_P, a->c_S, a->wk_H, a->wk_N, a->wv_H, a->wv_N, a->k_B, a->k_S, a->k_H, a->v_B, a->v_S, a->v_H,
                    a->kr_B, a->kr_S, a->kr_H, a->vr_B, a->vr_S, a->vr_H}, 8) ||
        !aligned(a->block_table, 4) || !aligned(a->kv_len, 4) || !aligned(a->places, 4))
        return DCP_ERR_ALIGN;
    const int ec = esize_of(a->cache_dtype);
    const int64_t named = a->max_pages * a->page_size, keys = a->max_keys < named ? a->max_keys : named;
    k.cache = (const char*)a->cache;
    k.c_P = a->c_P * ec; k.c_S = a->c_S * ec;
    k.table = a->block_table; k.kv = a->kv_len;
    k.t_B = a->t_B;
    k.wk = (const char*)a->w_k; k.wv = (const char*)a->w_v;
    k.wk_H = a->wk_H * 2; k.wk_N = a->wk_N * 2; k.wv_H = a->wv_H * 2; k.wv_N = a->wv_N * 2;
    k.ko = (char*)a->k; k.vo = (char*)a->v;
    k.ko_B = a->k_B * 2; k.ko_S = a->k_S * 2; k.ko_H = a->k_H * 2;
    k.vo_B = a->v_B * 2; k.vo_S = a->v_S * 2; k.vo_H = a->v_H * 2;
    k.kr = (char*)a->k_rest; k.vr = (char*)a->v_rest;
    k.kr_B = a->kr_B * 2; k.kr_S = a->kr_S * 2; k.kr_H = a->kr_H * 2;
    k.vr_B = a->vr_B * 2; k.vr_S = a->vr_S * 2; k.vr_H = a->vr_H * 2;
    k.places = a->places;
    k.pl_B = a->p_B;
    k.B = (int32_t)a->B; k.H = (int32_t)a->H;
    k.Dn = (int32_t)a->Dn; k.Dr = (int32_t)a->Dr; k.Dv = (int32_t)a->Dv; k.Dc = (int32_t)a->Dc;
    k.most = (int32_t)a->max_keys; k.keys = (int32_t)keys; k.pages = (int32_t)a->num_pages;
    k.fpage = dcp::make_fastdiv((uint32_t)a->page_size);
    k.fper = dcp::make_fastdiv((uint32_t)(a->Dn + a->Dv));
    k.ks = (float)a->k_scale;
    return DCP_OK;
}
int run_expand(const dcpa_expand_args* a, const ExpandArgs& k, void* stream) {
    return status(launch_expand(k, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, (hipStream_t)stream));
}

// The two calls that attention in the expanded form consists of: the expansion `make`, and attention over caches of one
// key to a page.
// The scale k_scale = f 2^e, 1 <= f < 2, is shared out: 2^e into the expansion, f to the scores and the outputs.  So what is
// written is within a factor of 2 of the keys and values themselves, however small or large the scale of a cache, and
// stays within fp16 where they do (a cache of rows near 448 with a scale of 2^-10 holds keys whose products with
// the weights pass 65504 by themselves); and the columns of the rope, which have no second part, stay exact: an 8-bit
// number, a multiple of 2^-9 up to 448, times 2^-15 to 2^7 is an fp16 one (16-bit ones lose what lies below 2^-24
// times 1 / f; they are not made larger).
int expanded_form(const dcpa_expand_args* e, const dcpa_attn_args* a, dcpa_expand_args& make, dcpa_attn_args& over, Rest& kr,
                  Rest& vr) {
    if (int st = check_expand(e)) return st;
    if (a->dtype != e->dtype) return DCP_ERR_DTYPE;
    if (a->B != e->B) return DCP_ERR_SHAPE;
    const int64_t n = e->max_keys;
    // from a key to the next, over all sequences
    if (e->B > 1 && n > 1 && (e->k_B != n * e->k_S || e->v_B != n * e->v_S ||
                              (e->k_rest && (e->kr_B != n * e->kr_S || e->vr_B != n * e->vr_S))))
        return DCP_ERR_STRIDE;
    auto apart = [&](int64_t b, int64_t s) { return n > 1 ? s : b; };
    kr = Rest{e->k_rest, apart(e->kr_B, e->kr_S), 0, e->kr_H};
    vr = Rest{e->v_rest, apart(e->vr_B, e->vr_S), 0, e->vr_H};
    make = *e;
    int power;
    frexp(e->k_scale, &power);
    const int least = -15, most = e->cache_dtype == DCP_FP8_E4M3 ? 7 : 0;
    make.k_scale = ldexp(1.0, power - 1 < least ? least : power - 1 > most ? most : power - 1);
    over = *a;
    over.k = e->k;
    over.k_P = apart(e->k_B, e->k_S);
    over.k_S = 0;
    over.k_H = e->k_H;
    // (no values at all, an empty buffer or a size query: NULL would say that they lie within the keys)
    static const char none alignas(16) = 0;
    over.v = e->v ? e->v : &none;
    over.v_P = apart(e->v_B, e->v_S);
    over.v_S = 0;
    over.v_H = e->v_H;
    over.block_table = e->places;
    over.t_B = e->p_B;
    over.kv_len = e->kv_len;
    over.Hkv = e->H;
    over.Dk = e->Dn + e->Dr;
    over.Dv = e->Dv;
    over.num_pages = e->B * n;
    over.page_size = 1;
    over.max_pages = n;
    over.cache_dtype = e->dtype;
    over.k_scale = over.v_scale = e->k_scale / make.k_scale;
    return DCP_OK;
}

// The weights' plan; as check_attn, no more workgroups than a launch may have.
int check_mass(const dcpa_attn_args* a, Batch& m, MassPlan& pl) {
    if (int st = check_batch(a, m)) return st;
    pl = plan_mass(m, (int)a->Dk, key_pieces(a));
    return ((int64_t)pl.units + 7) * m.Hkv > kMaxGrid ? DCP_ERR_SHAPE : DCP_OK;
}

}  // namespace

extern "C" {

const char* dcpa_status_str(int st) {
    switch (st) {
        case DCP_OK: return "DCP_OK";
        case DCP_ERR_NULL: return "DCP_ERR_NULL: a required pointer is NULL";
        case DCP_ERR_SHAPE: return "DCP_ERR_SHAPE: invalid or too large extent";
        case DCP_ERR_HEADS_NOT_DIVISIBLE: return "DCP_ERR_HEADS_NOT_DIVISIBLE: Hq is not a multiple of Hkv";
        case DCP_ERR_DTYPE: return "DCP_ERR_DTYPE: unsupported dtype";
        case DCP_ERR_LSE_BASE: return "DCP_ERR_LSE_BASE: lse_base is neither DCP_LSE_BASE_E nor DCP_LSE_BASE_2";
        case DCP_ERR_STRIDE: return "DCP_ERR_STRIDE: negative or too large stride";
        case DCP_ERR_ALIGN: return "DCP_ERR_ALIGN: a pointer or row stride is not aligned as documented";
        case DCP_ERR_LAUNCH: return "DCP_ERR_LAUNCH: HIP kernel launch failed";
        case DCPA_ERR_WORKSPACE: return "DCPA_ERR_WORKSPACE: workspace too small, missing or not 16-byte aligned";
        case DCPA_ERR_VALUE: return "DCPA_ERR_VALUE: a scale, eps or count outside its range";
        default: return "unknown dcpattn status";
    }
}

int64_t dcpa_paged_attn_workspace(const dcpa_attn_args* a) {
    if (a == nullptr) return DCP_ERR_NULL;
    Batch m;
    if (int st = check_attn(a, m)) return st;
    if (a->B == 0 || a->T == 0) return 0;
    return plan_of(a, m).ws_bytes;
}

int dcpa_paged_attn(const dcpa_attn_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    AttnArgs k;
    AttnPlan pl;
    bool any;
    if (int st = prepare_attn(a, k, pl, any)) return st;
    return any ? run_attn(a, k, pl, stream) : DCP_OK;
}

int64_t dcpa_prefix_attn_workspace(const dcpa_attn_args* a, int64_t n_groups) {
    if (a == nullptr) return DCP_ERR_NULL;
    Batch m;
    AttnPlan pl;
    if (int st = check_prefix(a, n_groups, m, pl)) return st;
    return a->B == 0 || a->T == 0 ? 0 : pl.ws_bytes;
}

int dcpa_prefix_attn(const dcpa_attn_args* a, const int32_t* cu_group, const int32_t* shared_len, int64_t n_groups,
                     void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    GroupArgs k;
    AttnPlan pl;
    if (int st = check_prefix(a, n_groups, k.m, pl)) return st;
    if (a->B == 0 || a->T == 0) return DCP_OK;
    if (int st = check_inputs(a)) return st;
    if (n_groups > 0 && (!cu_group || !shared_len)) return DCP_ERR_NULL;
    if (!aligned(cu_group, 4) || !aligned(shared_len, 4)) return DCP_ERR_ALIGN;
    if (int st = check_outputs(a)) return st;
    if (!sharing_pays(k.m, n_groups)) {
        if (int st = fill_attn(a, pl, k)) return st;
        return run_attn(a, k, pl, stream);
    }
    if (int st = fill_attn(a, pl, k, prefix_list_bytes(pl.units, n_groups + a->B))) return st;
    k.list = (PrefixUnit*)a->workspace;
    k.entries = (PrefixEntry*)(k.list + pl.units);
    k.cug = cu_group;
    k.same = shared_len;
    k.groups = (int32_t)n_groups;
    k.own_rows = pl.by_keys ? 32 : pl.rows;
    return status(launch_prefix(k, pl.latent, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, a->wide_weights != 0,
                                (hipStream_t)stream));
}

int64_t dcpa_pair_attn_workspace(const dcpa_attn_args* a) {
    if (a == nullptr) return DCP_ERR_NULL;
    Batch m;
    AttnPlan pl;
    if (int st = check_pairs(a, m, pl)) return st;
    return a->B == 0 || a->T == 0 ? 0 : pl.ws_bytes;
}

int dcpa_pair_attn(const dcpa_attn_args* a, const void* k_rest, int64_t kr_P, int64_t kr_S, int64_t kr_H, int64_t Dr,
                   const void* v_rest, int64_t vr_P, int64_t vr_S, int64_t vr_H, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    PairArgs k;
    AttnPlan pl;
    bool any;
    if (int st = prepare_pairs(a, Rest{k_rest, kr_P, kr_S, kr_H}, Dr, Rest{v_rest, vr_P, vr_S, vr_H}, k, pl, any)) return st;
    return any ? run_pairs(a, k, pl, stream) : DCP_OK;
}

int64_t dcpa_attn_mass_workspace(const dcpa_attn_args* a) {
    if (a == nullptr) return DCP_ERR_NULL;
    Batch m;
    MassPlan pl;
    if (int st = check_mass(a, m, pl)) return st;
    return a->B == 0 || a->T == 0 ? 0 : pl.ws_bytes;
}

int dcpa_attn_mass(const dcpa_attn_args* a, float* mass, int64_t m_P, int64_t m_S, int64_t m_H, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    MassArgs k;
    MassPlan pl;
    if (int st = check_mass(a, k.m, pl)) return st;
    if (!strides_ok({m_P, m_S, m_H}) || !span_ok({{a->num_pages, m_P}, {a->page_size, m_S}, {a->Hkv, m_H}}, 4))
        return DCP_ERR_STRIDE;
    if (a->B == 0 || a->T == 0) return DCP_OK;
    if (int st = check_inputs(a)) return st;
    if (!a->lse || (a->num_pages > 0 && !mass)) return DCP_ERR_NULL;
    if (!aligned(mass, 4)) return DCP_ERR_ALIGN;
    if (pl.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < pl.ws_bytes || !aligned(a->workspace, 16)))
        return DCPA_ERR_WORKSPACE;
    const int ec = esize_of(a->cache_dtype);
    k.q = (const char*)a->q;
    k.q_T = a->q_T * 2; k.q_H = a->q_H * 2;
    k.k = (const char*)a->k;
    k.k_P = a->k_P * ec; k.k_S = a->k_S * ec; k.k_H = a->k_H * ec;
    k.lse = a->lse;
    k.l_T = a->l_T; k.l_H = a->l_H;
    k.mass = mass;
    k.m_P = m_P; k.m_S = m_S; k.m_H = m_H;
    k.ws = pl.ws_bytes > 0 ? (float*)a->workspace : nullptr;
    k.Dk = (int32_t)a->Dk;
    k.slots = pl.slots;
    k.share = pl.share;
    k.units = pl.units;
    k.c = (float)(a->scale * a->k_scale * 1.4426950408889634);
    k.lmul = a->lse_base == DCP_LSE_BASE_E ? kLog2e : 1.0f;
    return status(launch_mass(k, pl.few, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, (hipStream_t)stream));
}

int dcpa_qk_norm_rope_append(const dcpa_rope_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    if (a->dtype != DCP_F16 && a->dtype != DCP_BF16) return DCP_ERR_DTYPE;
    if (a->cache_dtype != a->dtype && a->cache_dtype != DCP_FP8_E4M3) return DCP_ERR_DTYPE;
    const bool has_v = a->v != nullptr;
    if (a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq > (1 << 16) || a->Hkv > (1 << 16) || a->T > kMaxRows ||
        a->T * (a->Hq + 2 * a->Hkv) > kMaxRows)
        return DCP_ERR_SHAPE;
    auto cols = [](int64_t d) { return d >= 8 && d % 8 == 0 && d <= 1024; };
    if (!cols(a->D) || (has_v && !cols(a->Dv))) return DCP_ERR_SHAPE;
    if (a->q_norm < 0 || a->q_norm % 8 != 0 || a->q_norm > a->D || a->k_norm < 0 || a->k_norm % 8 != 0 ||
        a->k_norm > a->D)
        return DCP_ERR_SHAPE;
    if (a->rot < 0 || a->rot % 8 != 0 || a->rope_off < 0 || a->rope_off % 8 != 0 || a->rope_off > a->D ||
        a->rot > a->D - a->rope_off)
        return DCP_ERR_SHAPE;
    if (a->positions_max < 1 || a->positions_max >= (int64_t(1) << 31) || !cache_shape_ok(a->num_pages, a->page_size, 0))
        return DCP_ERR_SHAPE;
    if (!(a->eps >= 0.0) || a->eps > 3.0e38 || !positive(a->k_scale) || !positive(a->v_scale) ||
        !positive(1.0 / a->k_scale) || !positive(1.0 / a->v_scale))
        return DCPA_ERR_VALUE;
    if (!strides_ok({a->q_T, a->q_H, a->k_T, a->k_H, a->v_T, a->v_H, a->cs_P, a->qo_T, a->qo_H, a->kc_P, a->kc_S,
                     a->kc_H, a->vc_P, a->vc_S, a->vc_H, a->m_P, a->m_S, a->m_H}))
        return DCP_ERR_STRIDE;
    const int ec = esize_of(a->cache_dtype);
    if (!span_ok({{a->T, a->q_T}, {a->Hq, a->q_H}, {a->D, 1}}, 2) ||
        !span_ok({{a->T, a->qo_T}, {a->Hq, a->qo_H}, {a->D, 1}}, 2) ||
        !span_ok({{a->T, a->k_T}, {a->Hkv, a->k_H}, {a->D, 1}}, 2) ||
        !span_ok({{a->T, a->v_T}, {a->Hkv, a->v_H}, {a->Dv, 1}}, 2) ||
        !span_ok({{a->num_pages, a->kc_P}, {a->page_size, a->kc_S}, {a->Hkv, a->kc_H}, {a->D, 1}}, ec) ||
        !span_ok({{a->num_pages, a->vc_P}, {a->page_size, a->vc_S}, {a->Hkv, a->vc_H}, {a->Dv, 1}}, ec) ||
        !span_ok({{a->positions_max, a->cs_P}, {a->rot, 1}}, 4) ||
        !span_ok({{a->num_pages, a->m_P}, {a->page_size, a->m_S}, {a->Hkv, a->m_H}}, 4))
        return DCP_ERR_STRIDE;
    if (a->T == 0) return DCP_OK;
    if (a->q_out == a->q && ((a->T > 1 && a->qo_T != a->q_T) || (a->Hq > 1 && a->qo_H != a->q_H))) return DCP_ERR_STRIDE;
    if (!a->q || !a->k || !a->q_out || !a->slots || (a->rot > 0 && (!a->positions || !a->cos_sin)) ||
        (a->q_norm > 0 && !a->q_weight) || (a->k_norm > 0 && !a->k_weight) ||
        (a->num_pages > 0 && (!a->k_cache || (has_v && !a->v_cache))))
        return DCP_ERR_NULL;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->q_out, 16) ||
        !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16) || (a->rot > 0 && (!aligned(a->cos_sin, 16) || a->cs_P % 4 != 0)) ||
        !multiples({a->q_T, a->q_H, a->k_T, a->k_H, a->qo_T, a->qo_H, a->kc_P, a->kc_S, a->kc_H}, 8) ||
        (has_v && !multiples({a->v_T, a->v_H, a->vc_P, a->vc_S, a->vc_H}, 8)) || !aligned(a->k_cache, 8 * ec) ||
        !aligned(a->v_cache, 8 * ec) || !aligned(a->mass, 4) || !aligned(a->positions, 4) || !aligned(a->slots, 8))
        return DCP_ERR_ALIGN;
    RopeArgs k;
    k.q = (const char*)a->q; k.k = (const char*)a->k; k.v = (const char*)a->v;
    k.q_T = a->q_T * 2; k.q_H = a->q_H * 2; k.k_T = a->k_T * 2; k.k_H = a->k_H * 2;
    k.v_T = a->v_T * 2; k.v_H = a->v_H * 2;
    k.wq = (const char*)a->q_weight; k.wk = (const char*)a->k_weight;
    k.pos = a->positions;
    k.cs = a->cos_sin;
    k.cs_P = a->cs_P;
    k.slots = a->slots;
    k.qo = (char*)a->q_out; k.kc = (char*)a->k_cache; k.vc = (char*)a->v_cache;
    k.qo_T = a->qo_T * 2; k.qo_H = a->qo_H * 2;
    k.kc_P = a->kc_P * ec; k.kc_S = a->kc_S * ec; k.kc_H = a->kc_H * ec;
    k.vc_P = a->vc_P * ec; k.vc_S = a->vc_S * ec; k.vc_H = a->vc_H * ec;
    k.mass = a->mass;
    k.m_P = a->m_P; k.m_S = a->m_S; k.m_H = a->m_H;
    k.T = (int32_t)a->T; k.Hq = (int32_t)a->Hq; k.Hkv = (int32_t)a->Hkv; k.D = (int32_t)a->D; k.Dv = (int32_t)a->Dv;
    k.nq = (int32_t)a->q_norm; k.nk = (int32_t)a->k_norm; k.off = (int32_t)a->rope_off; k.rot = (int32_t)a->rot;
    k.pairs = a->interleaved != 0;
    k.positions = (int32_t)a->positions_max;
    k.page_size = (int32_t)a->page_size;
    k.slots_max = a->num_pages * a->page_size;
    k.fheads = dcp::make_fastdiv((uint32_t)(a->Hq + a->Hkv * (has_v ? 2 : 1)));
    k.eps = (float)a->eps;
    k.ik = (float)(1.0 / a->k_scale);
    k.iv = (float)(1.0 / a->v_scale);
    return status(launch_rope(k, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, (hipStream_t)stream));
}

int dcpa_cache_evict(const dcpa_evict_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    if (a->esize != 1 && a->esize != 2 && a->esize != 4) return DCP_ERR_DTYPE;
    if (a->B < 0 || a->Hkv < 1 || a->Hkv > (1 << 16) || a->B > (int64_t(1) << 20) || a->B * a->Hkv > (int64_t(1) << 21) ||
        a->Dk < 1 || a->Dk > 4096 || (a->v && (a->Dv < 1 || a->Dv > 4096)) ||
        !cache_shape_ok(a->num_pages, a->page_size, a->max_pages) ||
        !cache_shape_ok(a->num_pages, a->page_size, a->dst_pages))
        return DCP_ERR_SHAPE;
    if (a->budget < 1 || a->n_sink < 0 || a->n_recent < 0 || a->n_sink > a->budget ||
        a->n_recent > a->budget - a->n_sink || a->budget > a->dst_pages * a->page_size)
        return DCPA_ERR_VALUE;
    // 2^31 work-items of a launch: 1024 to a sequence and head above, up to 32 to a row here
    if (a->B * a->Hkv * a->budget > kMaxGrid * 32) return DCP_ERR_SHAPE;
    if (!strides_ok({a->m_P, a->m_S, a->m_H, a->k_P, a->k_S, a->k_H, a->v_P, a->v_S, a->v_H, a->t_B, a->d_B, a->kp_B,
                     a->kp_H}))
        return DCP_ERR_STRIDE;
    const int64_t e = a->esize;
    if (!span_ok({{a->num_pages, a->m_P}, {a->page_size, a->m_S}, {a->Hkv, a->m_H}}, 4) ||
        !span_ok({{a->num_pages, a->k_P}, {a->page_size, a->k_S}, {a->Hkv, a->k_H}, {a->Dk, 1}}, e) ||
        !span_ok({{a->num_pages, a->v_P}, {a->page_size, a->v_S}, {a->Hkv, a->v_H}, {a->v ? a->Dv : 1, 1}}, e) ||
        !span_ok({{a->B, a->t_B}, {a->max_pages, 1}}, 4) || !span_ok({{a->B, a->d_B}, {a->dst_pages, 1}}, 4) ||
        !span_ok({{a->B, a->kp_B}, {a->Hkv, a->kp_H}, {a->budget, 1}}, 4))
        return DCP_ERR_STRIDE;
    if (a->B == 0) return DCP_OK;
    if (!a->kv_len || !a->new_len || !a->kept || !a->dst_table || (a->max_pages > 0 && !a->block_table) ||
        (a->num_pages > 0 && (!a->mass || !a->k)))
        return DCP_ERR_NULL;
    auto rows = [&](int64_t n) {
        return aligned(a->k, n) && multiples({a->Dk * e, a->k_P * e, a->k_S * e, a->k_H * e}, n) &&
               (!a->v || (aligned(a->v, n) && multiples({a->Dv * e, a->v_P * e, a->v_S * e, a->v_H * e}, n)));
    };
    if (!rows(8) || !aligned(a->mass, 4) || !aligned(a->kv_len, 4) || !aligned(a->new_len, 4) || !aligned(a->kept, 4) ||
        !aligned(a->block_table, 4) || !aligned(a->dst_table, 4))
        return DCP_ERR_ALIGN;
    // new lengths over the old ones of other sequences would be read for them
    const uintptr_t l0 = (uintptr_t)a->kv_len, l1 = (uintptr_t)a->new_len, bytes = (uintptr_t)a->B * 4;
    if (l0 != l1 && (l0 < l1 ? l1 - l0 : l0 - l1) < bytes) return DCPA_ERR_VALUE;
    EvictArgs k;
    k.mass = (char*)a->mass;
    k.m_P = a->m_P; k.m_S = a->m_S; k.m_H = a->m_H;
    k.k = (char*)a->k; k.v = (char*)a->v;
    k.k_P = a->k_P * e; k.k_S = a->k_S * e; k.k_H = a->k_H * e;
    k.v_P = a->v_P * e; k.v_S = a->v_S * e; k.v_H = a->v_H * e;
    k.table = a->block_table; k.kv = a->kv_len; k.dst = a->dst_table;
    k.t_B = a->t_B; k.d_B = a->d_B;
    k.new_len = a->new_len; k.kept = a->kept;
    k.kp_B = a->kp_B; k.kp_H = a->kp_H;
    k.B = (int32_t)a->B; k.Hkv = (int32_t)a->Hkv;
    k.k_bytes = (int32_t)(a->Dk * e); k.v_bytes = (int32_t)(a->v ? a->Dv * e : 0);
    k.pages = (int32_t)a->num_pages; k.page_size = (int32_t)a->page_size;
    k.max_keys = (int32_t)(a->max_pages * a->page_size);
    k.budget = (int32_t)a->budget; k.sink = (int32_t)a->n_sink; k.recent = (int32_t)a->n_recent;
    k.wide = rows(16);
    k.fpage = dcp::make_fastdiv((uint32_t)a->page_size);
    k.fHkv = dcp::make_fastdiv((uint32_t)a->Hkv);
    k.fbudget = dcp::make_fastdiv((uint32_t)a->budget);
    return status(launch_evict(k, (hipStream_t)stream));
}

int dcpa_batch_plan(const dcpa_plan_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    if (a->B < 0 || a->B > (int64_t(1) << 20) || a->T < 0 || a->T > kMaxRows || a->free_max < 0 ||
        a->free_max >= (int64_t(1) << 31) || !cache_shape_ok(0, a->page_size, a->max_pages) ||
        !ranks_ok(a->N, a->rank, a->interleave))
        return DCP_ERR_SHAPE;
    if (!strides_ok({a->t_B}) || !span_ok({{a->B, a->t_B}, {a->max_pages, 1}}, 4)) return DCP_ERR_STRIDE;
    // (rows of the table that overlap would be written by two sequences)
    if (a->B > 1 && a->t_B < a->max_pages) return DCP_ERR_STRIDE;
    if (!a->free_count || !a->free_count_out || !a->cu_q || (a->free_max > 0 && !a->free_pages) ||
        (a->B > 0 && (!a->new_len || !a->seq_len || !a->kv_len || !a->seq_out || !a->kv_out ||
                      (a->max_pages > 0 && !a->block_table))) ||
        (a->T > 0 && (!a->positions || !a->sequence || !a->slots)))
        return DCP_ERR_NULL;
    for (const void* x : {(const void*)a->new_len, (const void*)a->seq_len, (const void*)a->kv_len,
                          (const void*)a->keep_pages, (const void*)a->block_table, (const void*)a->free_pages,
                          (const void*)a->free_count, (const void*)a->free_count_out, (const void*)a->seq_out,
                          (const void*)a->kv_out, (const void*)a->cu_q, (const void*)a->positions, (const void*)a->sequence})
        if (!aligned(x, 4)) return DCP_ERR_ALIGN;
    if (!aligned(a->slots, 8)) return DCP_ERR_ALIGN;
    // a length written over another sequence's that is still to be read
    for (const int32_t* out : {a->seq_out, a->kv_out})
        for (const int32_t* in : {a->new_len, a->seq_len, a->kv_len, a->keep_pages})
            if (in && in != out && apart((uintptr_t)in, (uintptr_t)out) < (uintptr_t)a->B * 4) return DCPA_ERR_VALUE;
    if (a->B > 0 && apart((uintptr_t)a->seq_out, (uintptr_t)a->kv_out) < (uintptr_t)a->B * 4) return DCPA_ERR_VALUE;
    PlanArgs k;
    k.new_len = a->new_len; k.seq = a->seq_len; k.kv = a->kv_len; k.keep = a->keep_pages;
    k.table = a->block_table;
    k.t_B = a->t_B;
    k.free = a->free_pages; k.count = a->free_count;
    k.count_out = a->free_count_out; k.seq_out = a->seq_out; k.kv_out = a->kv_out; k.cu = a->cu_q;
    k.positions = a->positions; k.sequence = a->sequence;
    k.slots = a->slots;
    k.B = (int32_t)a->B; k.T = (int32_t)a->T; k.width = (int32_t)a->max_pages;
    k.page_size = (int32_t)a->page_size; k.free_max = (int32_t)a->free_max;
    k.N = (int32_t)a->N; k.rank = (int32_t)a->rank; k.inter = (int32_t)a->interleave;
    k.fpage = dcp::make_fastdiv((uint32_t)k.page_size);
    k.fblock = dcp::make_fastdiv((uint32_t)(k.N * k.inter));
    return status(launch_plan(k, (hipStream_t)stream));
}

int dcpa_project(const dcpa_project_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    if (a->dtype != DCP_F16 && a->dtype != DCP_BF16) return DCP_ERR_DTYPE;
    auto cols = [](int64_t d) { return d >= 8 && d % 8 == 0 && d <= 1024; };
    if (a->T < 0 || a->T > kMaxRows || a->H < 1 || a->H > (1 << 16) || a->T * a->H > kMaxRows || !cols(a->N) ||
        !cols(a->K) || (a->copy != 0 && !cols(a->copy)) || project_tiles(a->T, a->H, a->N) >= kMaxRows)
        return DCP_ERR_SHAPE;
    const bool turned = a->w_N == 1;
    if (!strides_ok({a->x_T, a->x_H, a->w_H, a->w_N, a->w_K, a->y_T, a->y_H}) || (!turned && a->w_K != 1) ||
        !span_ok({{a->T, a->x_T}, {a->H, a->x_H}, {a->K + a->copy, 1}}, 2) ||
        !span_ok({{a->T, a->y_T}, {a->H, a->y_H}, {a->N + a->copy, 1}}, 2) ||
        !span_ok({{a->H, a->w_H}, {a->N, a->w_N}, {a->K, a->w_K}}, 2))
        return DCP_ERR_STRIDE;
    if (a->T == 0) return DCP_OK;
    if (!a->x || !a->w || !a->y) return DCP_ERR_NULL;
    if (!aligned(a->x, 16) || !aligned(a->w, 16) || !aligned(a->y, 16) ||
        !multiples({a->x_T, a->x_H, a->w_H, turned ? a->w_K : a->w_N, a->y_T, a->y_H}, 8))
        return DCP_ERR_ALIGN;
    ProjectArgs k;
    k.x = (const char*)a->x; k.w = (const char*)a->w; k.y = (char*)a->y;
    k.x_T = a->x_T * 2; k.x_H = a->x_H * 2;
    k.w_H = a->w_H * 2; k.w_N = a->w_N * 2; k.w_K = a->w_K * 2;
    k.y_T = a->y_T * 2; k.y_H = a->y_H * 2;
    k.T = (int32_t)a->T; k.H = (int32_t)a->H; k.N = (int32_t)a->N; k.K = (int32_t)a->K; k.copy = (int32_t)a->copy;
    k.fH = dcp::make_fastdiv((uint32_t)a->H);
    return status(launch_project(k, turned, a->dtype == DCP_BF16, (hipStream_t)stream));
}

int dcpa_latent_expand(const dcpa_expand_args* a, void* stream) {
    if (a == nullptr) return DCP_ERR_NULL;
    ExpandArgs k;
    bool any;
    if (int st = prepare_expand(a, k, any)) return st;
    return any ? run_expand(a, k, stream) : DCP_OK;
}

int64_t dcpa_latent_attn_workspace(const dcpa_expand_args* e, const dcpa_attn_args* a) {
    if (e == nullptr || a == nullptr) return DCP_ERR_NULL;
    dcpa_expand_args make;
    dcpa_attn_args over;
    Rest kr, vr;
    if (int st = expanded_form(e, a, make, over, kr, vr)) return st;
    return e->k_rest ? dcpa_pair_attn_workspace(&over) : dcpa_paged_attn_workspace(&over);
}

int dcpa_latent_attn(const dcpa_expand_args* e, const dcpa_attn_args* a, void* stream) {
    if (e == nullptr || a == nullptr) return DCP_ERR_NULL;
    dcpa_expand_args make;
    dcpa_attn_args over;
    Rest kr, vr;
    if (int st = expanded_form(e, a, make, over, kr, vr)) return st;
    ExpandArgs x;
    PairArgs k;
    AttnPlan pl;
    bool keys, rows;
    if (int st = prepare_expand(&make, x, keys)) return st;
    if (keys && !e->places) return DCP_ERR_NULL;
    const bool parts = e->k_rest != nullptr;
    if (int st = parts ? prepare_pairs(&over, kr, e->Dn, vr, k, pl, rows) : prepare_attn(&over, k, pl, rows)) return st;
    // (every check is made: from here on work is enqueued)
    if (keys)
        if (int st = run_expand(&make, x, stream)) return st;
    if (!rows) return DCP_OK;
    return parts ? run_pairs(&over, k, pl, stream) : run_attn(&over, k, pl, stream);
}

}  // extern "C"
