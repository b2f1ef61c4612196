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
    if (a->N < 1 || a->N > (1 << 20) || a->rank < 0 || a->rank >= a->N || a->interleave < 1 ||
        a->interleave > (1 << 20) || a->N * a->interleave > (int64_t(1) << 30))
        return DCP_ERR_SHAPE;
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
AttnPlan plan_of(const dcpa_attn_args* a, const Batch& m) {
    const bool values = a->cache_dtype != DCP_FP8_E4M3 ||
                        (a->Dv % 16 == 0 && (!a->v || multiples({a->v_P, a->v_S, a->v_H}, 16)));
    return plan_attn(m, (int)a->Dk, (int)a->Dv, key_pieces(a) && values);
}

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

int check_attn(const dcpa_attn_args* a, Batch& m) {
    if (int st = check_batch(a, m)) return st;
    const bool shared = a->v == nullptr;
    if (a->Dv < 8 || a->Dv % 8 != 0 || a->Dv > 512) return DCP_ERR_SHAPE;
    if (shared ? a->Dv > a->Dk : a->Dk > 256 || a->Dv > 256) return DCP_ERR_SHAPE;
    if (!strides_ok({a->v_P, a->v_S, a->v_H, a->o_T, a->o_H})) return DCP_ERR_STRIDE;
    if (!span_ok({{a->num_pages, a->v_P}, {a->page_size, a->v_S}, {a->Hkv, a->v_H}, {a->Dv, 1}},
                 esize_of(a->cache_dtype)) ||
        !span_ok({{a->T, a->o_T}, {a->Hq, a->o_H}, {a->Dv, 1}}, 2))
        return DCP_ERR_STRIDE;
    const AttnPlan pl = plan_of(a, m);
    if (((int64_t)pl.units + 7) * m.Hkv > kMaxGrid || (pl.slots > 0 && a->T * a->Hq / 4 >= kMaxGrid)) return DCP_ERR_SHAPE;
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
    if (int st = check_attn(a, k.m)) return st;
    if (a->B == 0 || a->T == 0) return DCP_OK;
    if (int st = check_inputs(a)) return st;
    if (!a->out) return DCP_ERR_NULL;
    const int ec = esize_of(a->cache_dtype);
    if (!aligned(a->v, 16) || (a->v && !multiples({a->v_P, a->v_S, a->v_H}, 8)) || !aligned(a->out, 4) ||
        !multiples({a->o_T, a->o_H}, 2))
        return DCP_ERR_ALIGN;
    const AttnPlan pl = plan_of(a, k.m);
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
    k.ws_o = (float*)a->workspace;
    k.ws_l = k.ws_o == nullptr ? nullptr : k.ws_o + (int64_t)pl.units * k.m.Hkv * pl.rows * a->Dv;
    k.c = (float)(a->scale * a->k_scale * 1.4426950408889634);
    // (in the latent layout the values are the keys' own columns)
    k.vs = (float)(a->v ? a->v_scale : a->k_scale);
    k.lmul = a->lse_base == DCP_LSE_BASE_E ? kLn2 : 1.0f;
    return status(launch_attn(k, pl, a->dtype == DCP_BF16, a->cache_dtype == DCP_FP8_E4M3, a->wide_weights != 0,
                              (hipStream_t)stream));
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

}  // extern "C"
