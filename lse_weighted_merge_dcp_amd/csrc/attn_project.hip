// attn_project.hip -- the projections on both sides of latent attention, head
// by head, and the keys and values of all heads from cached latent rows.
//
// project_rows: y[t, h] = x[t, h] W[h], rows of tokens against one head's
// weights.  Bound by the weights' bytes where tokens are few, by the rows' where
// they are many (a weight of 128 x 512 makes 512 outputs of 128 inputs: 205
// operations a byte, and the matrix instructions do 220).
// expand_rows: cached rows against the weights of all heads side by side.
#include "attn_product.hpp"

namespace dcpa {

namespace {

// ---------------------------------------------------------------------------
// project_rows
// ---------------------------------------------------------------------------
template <typename E, int MT, int NT, int ST, bool TURNED>
__global__ __launch_bounds__(256, 2) void project_rows(ProjectArgs p) {
    using P = Product<E, MT, NT, 2, 2, ST, TURNED, false>;
    __shared__ __attribute__((aligned(1024))) char lds[P::LDS];
    // the column tiles of a unit (one head's row tile) follow each other on one XCD, which the heads keep
    const uint32_t id = blockIdx.x, turn = fdiv(id >> 3, p.fnt);
    const int nt = (int)((id >> 3) - turn * p.fnt.d);
    const int64_t unit = (int64_t)turn * 8 + (id & 7);
    if (unit >= (int64_t)p.mt * p.H) return;
    const int m = (int)fdiv((uint32_t)unit, p.fH), head = (int)((uint32_t)unit - (uint32_t)m * p.fH.d);
    const int row0 = m * MT, col0 = nt * NT;
    P t(lds);
    const char* x = p.x + (int64_t)head * p.x_H;
    const char* w = p.w + (int64_t)head * p.w_H;
#pragma unroll
    for (int i = 0; i < P::NX; ++i) t.xat[i] = (uint64_t)(x + (int64_t)min(row0 + t.x_row(i), p.T - 1) * p.x_T);
    bool n_here = true;
    if constexpr (TURNED) {
        n_here = col0 + t.wc * 8 < p.N;
#pragma unroll
        for (int i = 0; i < P::NW; ++i) t.wat[i] = (uint64_t)(w + (int64_t)t.w_row(i) * p.w_K + (col0 + t.wc * 8) * 2);
    } else {
#pragma unroll
        for (int i = 0; i < P::NW; ++i) t.wat[i] = (uint64_t)(w + (int64_t)min(col0 + t.w_row(i), p.N - 1) * p.w_N);
    }
    t.run(p.K, p.w_K, n_here);
    char* y = p.y + (int64_t)head * p.y_H;
    t.template store<false>(1.0f, [&](int row, int col, u32x4 v, u32x4) {
        if (row0 + row < p.T && col0 + col < p.N)
            *(u32x4*)(y + (int64_t)(row0 + row) * p.y_T + (col0 + col) * 2) = v;
    });
    if (nt == 0 && p.copy > 0) {
        const int pieces = p.copy / 8;
        for (int i = threadIdx.x; i < MT * pieces; i += 256) {
            const int row = row0 + i / pieces, c = i % pieces;
            if (row < p.T)
                *(u32x4*)(y + (int64_t)row * p.y_T + (p.N + c * 8) * 2) = *(const u32x4*)(x + (int64_t)row * p.x_T + (p.K + c * 8) * 2);
        }
    }
}

// ---------------------------------------------------------------------------
// expand_rows: a workgroup takes 256 keys of a sequence and 256 of the H (Dn + Dv)
// weight rows.
// ---------------------------------------------------------------------------
template <typename E, bool X8, bool REST> __global__ __launch_bounds__(512, 2) void expand_rows(ExpandArgs p) {
    using P = Product<E, 256, 256, 2, 4, 2, false, X8>;
    __shared__ __attribute__((aligned(1024))) char lds[P::LDS];
    const int nt = (int)(blockIdx.x % (uint32_t)p.nt), rest = (int)(blockIdx.x / (uint32_t)p.nt);
    const int b = rest / p.mt, row0 = (rest - b * p.mt) * 256, col0 = nt * 256;
    // (a length may be more than the table has pages for: those keys are not there)
    const int counted = min(max(p.kv[b], 0), p.most), kv = min(counted, p.keys);
    auto place_of = [&](int j, bool there) {
        if (nt == 0 && p.places != nullptr && j < counted) p.places[(int64_t)b * p.pl_B + j] = there ? b * p.most + j : -1;
    };
    if (row0 >= kv) {
        if (threadIdx.x < 256) place_of(row0 + (int)threadIdx.x, false);
        return;
    }
    constexpr int ES = X8 ? 1 : 2;
    const int per = p.Dn + p.Dv, cols = per * p.H;
    const int32_t* table = p.table + (int64_t)b * p.t_B;
    P t(lds);
    auto page_of = [&](int j, int& place) {
        const uint32_t at = fdiv((uint32_t)j, p.fpage);
        place = j - (int)(at * p.fpage.d);
        return table[at];
    };
#pragma unroll
    for (int i = 0; i < P::NX; ++i) {
        int place;
        const int page = page_of(min(row0 + t.x_row(i), kv - 1), place);
        const bool there = (uint32_t)page < (uint32_t)p.pages;
        // (the row of zeros is as long as the widest cached row)
        t.xat[i] = at_or_zeros(there, (uint64_t)p.cache + times64((uint32_t)page, p.c_P) + times64((uint32_t)place, p.c_S));
    }
#pragma unroll
    for (int i = 0; i < P::NW; ++i) {
        const uint32_t n = (uint32_t)min(col0 + t.w_row(i), cols - 1), h = fdiv(n, p.fper);
        const int d = (int)(n - h * (uint32_t)per);
        t.wat[i] = d < p.Dn ? (uint64_t)(p.wk + (int64_t)h * p.wk_H + (int64_t)d * p.wk_N)
                            : (uint64_t)(p.wv + (int64_t)h * p.wv_H + (int64_t)(d - p.Dn) * p.wv_N);
    }
    t.run(p.Dc, 0, true);
    meet();
    // which of the tile's keys are there
    uint8_t* there_s = (uint8_t*)lds;
    if (threadIdx.x < 256) {
        const int j = row0 + (int)threadIdx.x;
        int place;
        bool there = false;
        if (j < kv) there = (uint32_t)page_of(j, place) < (uint32_t)p.pages;
        there_s[threadIdx.x] = there;
        place_of(j, there);
    }
    meet();
    char* ko = p.ko + (int64_t)b * p.ko_B;
    char* vo = p.vo + (int64_t)b * p.vo_B;
    auto put = [&](int row, int col, u32x4 v, u32x4 rest) {
        const int j = row0 + row;
        const uint32_t n = (uint32_t)(col0 + col), h = fdiv(n, p.fper);
        const int d = (int)(n - h * (uint32_t)per);
        if ((int)n >= cols || !there_s[row]) return;
        char* at = d < p.Dn ? ko + (int64_t)j * p.ko_S + (int64_t)h * p.ko_H + d * 2
                            : vo + (int64_t)j * p.vo_S + (int64_t)h * p.vo_H + (d - p.Dn) * 2;
        *(u32x4*)at = v;
        if constexpr (REST) {
            at = d < p.Dn ? p.kr + (int64_t)b * p.kr_B + (int64_t)j * p.kr_S + (int64_t)h * p.kr_H + d * 2
                          : p.vr + (int64_t)b * p.vr_B + (int64_t)j * p.vr_S + (int64_t)h * p.vr_H + (d - p.Dn) * 2;
            *(u32x4*)at = rest;
        }
    };
    t.template store<REST>(p.ks, put);
    // the columns that all heads share, for the heads whose first weight row is this tile's
    if (p.Dr > 0) {
        const int h0 = (col0 + per - 1) / per, h1 = min((min(col0 + 256, cols) + per - 1) / per, p.H), pieces = p.Dr / 8;
        for (int i = threadIdx.x; i < 256 * pieces; i += 512) {
            const int row = i / pieces, c = i % pieces, j = row0 + row;
            if (!there_s[row]) continue;
            int place;
            const int page = page_of(j, place);
            const char* from = p.cache + (int64_t)page * p.c_P + (int64_t)place * p.c_S + (p.Dc + c * 8) * ES;
            u32x4 v;
            if constexpr (X8) {
                v = widen8<E>(*(const u32x2*)from);
                uint32_t s[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] = Mat<E>::pack2(Mat<E>::low(v[k]) * p.ks, Mat<E>::high(v[k]) * p.ks);
                v = u32x4{s[0], s[1], s[2], s[3]};
            } else {
                v = *(const u32x4*)from;
                if (p.ks != 1.0f) {
                    uint32_t s[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[k] = Mat<E>::pack2(Mat<E>::low(v[k]) * p.ks, Mat<E>::high(v[k]) * p.ks);
                    v = u32x4{s[0], s[1], s[2], s[3]};
                }
            }
            for (int h = h0; h < h1; ++h)
                *(u32x4*)(ko + (int64_t)j * p.ko_S + (int64_t)h * p.ko_H + (p.Dn + c * 8) * 2) = v;
        }
    }
}

template <typename E, int MT, int NT, int ST> hipError_t project(const ProjectArgs& arg, bool turned, hipStream_t stream) {
    ProjectArgs a = arg;
    a.mt = (a.T + MT - 1) / MT;
    const int nt = (a.N + NT - 1) / NT;
    a.fnt = dcp::make_fastdiv((uint32_t)nt);
    const dim3 grid((uint32_t)(((int64_t)a.mt * a.H + 7) / 8 * 8 * nt)), block(256);
    return turned ? launch(project_rows<E, MT, NT, ST, true>, grid, block, stream, a)
                  : launch(project_rows<E, MT, NT, ST, false>, grid, block, stream, a);
}

// Rows of a tile.
bool few_rows(int64_t T) { return T <= 128; }
int64_t tiles_of(int64_t n, int64_t each) { return (n + each - 1) / each; }

}  // namespace

int64_t project_workgroups(int64_t T, int64_t H, int64_t N) {
    const int64_t each = few_rows(T) ? 64 : 128;
    return (tiles_of(T, each) * H + 7) / 8 * 8 * tiles_of(N, each);
}
int64_t expand_workgroups(int64_t B, int64_t most, int64_t H, int64_t per) {
    return B * tiles_of(most, 256) * tiles_of(H * per, 256);
}

hipError_t launch_project(const ProjectArgs& a, bool turned, bool bf16, hipStream_t stream) {
    auto run = [&](auto e) {
        using E = decltype(e);
        return few_rows(a.T) ? project<E, 64, 64, 4>(a, turned, stream) : project<E, 128, 128, 2>(a, turned, stream);
    };
    return bf16 ? run(BF16T{}) : run(F16T{});
}

hipError_t launch_expand(const ExpandArgs& arg, bool bf16, bool x8, hipStream_t stream) {
    ExpandArgs a = arg;
    a.mt = (a.most + 255) / 256;
    a.nt = (int32_t)(((int64_t)a.H * (a.Dn + a.Dv) + 255) / 256);
    const dim3 grid((uint32_t)((int64_t)a.B * a.mt * a.nt)), block(512);
    auto run = [&](auto e) {
        using E = decltype(e);
        if (a.kr != nullptr)
            return x8 ? launch(expand_rows<E, true, true>, grid, block, stream, a) : launch(expand_rows<E, false, true>, grid, block, stream, a);
        return x8 ? launch(expand_rows<E, true, false>, grid, block, stream, a) : launch(expand_rows<E, false, false>, grid, block, stream, a);
    };
    return bf16 ? run(BF16T{}) : run(F16T{});
}

}  // namespace dcpa
