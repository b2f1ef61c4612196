// attn_project.hip -- the projections on both sides of latent attention, head
// by head, and the keys and values of all heads from cached latent rows.
//
// project_rows: y[t, h] = x[t, h] W[h], rows of tokens against one head's weights.
// Bound by bytes: the weights' where tokens are few (64 tokens, 128 heads of 128 x
// 512: 9.2 us for queries, 7.5 for values, of which the 27 MB take 4.5 and a launch the
// rest), the rows' where they are many (a weight of 128 x 512 makes 512 outputs of
// 128 inputs: 205 operations a byte, and the matrix instructions do 220).  4096
// tokens' queries take 223 us, 3.7 TB/s; without their stores 117, so stores and the
// rest still come one after the other; 2001 tokens' values of 96 heads 55 us, 4.7 TB/s
// (42 over the same rows again and again: the Infinity Cache holds part of them).
// expand_rows: cached rows against the weights of all heads side by side.  Bound by
// products and stores, which come one after the other as the waves of a CU's one
// workgroup go in step.  In the products a step of 256 x 256 x 64 takes 2048 clocks of
// matrix instructions, and as many of LDS accesses for the fragments (1536) and the next
// operands (512).  16384 rows, 128 heads of 128 + 64 / 128 columns: 731 to 755 us, 0.74
// PFLOP/s (390 us without loads and stores, 515 without stores; tiles of 128 x 256 by two
// workgroups to a CU 860 us, steps of 32 columns 827, one workgroup to a tile 814).
#include "attn_product.hpp"

namespace dcpa {

namespace {

// ---------------------------------------------------------------------------
// project_rows: a workgroup takes p.each tiles in the order (rows, head, columns).
// ---------------------------------------------------------------------------
template <typename E, int MT, int NT, int ST, bool TURNED, bool FAR>
__global__ __launch_bounds__(256, 2) void project_rows(ProjectArgs p) {
    using P = Product<E, MT, NT, 64, 2, 2, ST, TURNED, false>;
    __shared__ __attribute__((aligned(1024))) char lds[P::LDS];
    P c(lds);
    const int first = (int)blockIdx.x * p.each, tiles = min(p.each, p.tiles - first);
    if (tiles <= 0) return;
    struct Tile {
        int row0, head, col0;
    };
    auto tile = [&](int t) {
        const uint32_t id = (uint32_t)(first + t), unit = fdiv(id, p.fnt), m = fdiv(unit, p.fH);
        return Tile{(int)m * MT, (int)(unit - m * p.fH.d), (int)(id - unit * p.fnt.d) * NT};
    };
    auto aim = [&](int t) {
        const Tile a = tile(t);
        const char* x = p.x + (int64_t)a.head * p.x_H;
        const char* w = p.w + (int64_t)a.head * p.w_H;
#pragma unroll
        for (int i = 0; i < P::NX; ++i) c.xat[i] = (uint64_t)(x + (int64_t)min(a.row0 + c.x_row(i), p.T - 1) * p.x_T);
        if constexpr (TURNED) {
            c.n_here = a.col0 + c.wc * 8 < p.N;
#pragma unroll
            for (int i = 0; i < P::NW; ++i) c.wat[i] = (uint64_t)(w + (int64_t)c.w_row(i) * p.w_K + (a.col0 + c.wc * 8) * 2);
        } else {
#pragma unroll
            for (int i = 0; i < P::NW; ++i) c.wat[i] = (uint64_t)(w + (int64_t)min(a.col0 + c.w_row(i), p.N - 1) * p.w_N);
        }
    };
    c.template run<P::STORES>(tiles, p.K, p.w_K, aim, [&](int t) {
        const Tile a = tile(t);
        const int col = a.col0 + c.out_col();
        char* y = p.y + (int64_t)a.head * p.y_H;
        char* to = y + (int64_t)a.row0 * p.y_T + col * 2;
        const bool whole = a.row0 + MT <= p.T && a.col0 + NT <= p.N;
        if (whole) c.template store<false, FAR>(1.0f, to, p.y_T, nullptr, 0, [](int) { return true; });
        else c.template store<false, FAR>(1.0f, to, p.y_T, nullptr, 0, [&](int row) { return a.row0 + row < p.T && col < p.N; });
        const bool copies = p.copy > 0 && a.col0 == 0;
        if (copies) {
            const char* x = p.x + (int64_t)a.head * p.x_H;
            const int pieces = p.copy / 8;
            for (int i = threadIdx.x; i < MT * pieces; i += 256) {
                const int row = a.row0 + i / pieces, k = i % pieces;
                if (row < p.T)
                    *(u32x4*)(y + (int64_t)row * p.y_T + (p.N + k * 8) * 2) = *(const u32x4*)(x + (int64_t)row * p.x_T + (p.K + k * 8) * 2);
            }
        }
        return whole && !copies;
    });
}

// ---------------------------------------------------------------------------
// expand_rows: a workgroup takes 256 or 128 keys of a sequence and p.each tiles of 256 of
// the H (Dn + Dv) weight rows.
// ---------------------------------------------------------------------------
// (128 keys where the roundings' rests are written too: their way out takes the registers of the other 128)
constexpr int NT = 256;
constexpr int expand_rows_of(bool rest) { return rest ? 128 : 256; }
constexpr int kChip = 256, kMostRounds = 4;     // workgroups that run at once; rounds of them, at most, where columns are cut
template <typename E, bool X8, bool REST, bool FAR> __global__ __launch_bounds__(512, 2) void expand_rows(ExpandArgs p) {
    constexpr int MT = expand_rows_of(REST);
    using P = Product<E, MT, NT, 64, 2, 4, 2, false, X8>;
    constexpr int ES = X8 ? 1 : 2, NR = MT * 8 / 512;      // NR: the thread's pieces of the columns that all heads share, at most
    __shared__ __attribute__((aligned(1024))) char lds[P::LDS];
    P c(lds);
    // Row tiles that there are keys for, and into how many ranges the columns are cut for each: of 64 numbers the one
    // with which the longest workgroup (rounds of the chip times its tiles, and a third of one to start) ends first.
    // Row tiles 8 apart go to one XCD with all their ranges, so that its L2 serves most of what they read.
    int rows = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64)
        rows += b0 + c.lane < p.B ? (min(max(p.kv[b0 + c.lane], 0), p.most) + MT - 1) / MT : 0;
    rows = fold_wave(rows, 0, [](int x, int y) { return x + y; });
    const int apart = rows >= 8 ? (rows + 7) / 8 * 8 : max(rows, 1);
    int ranges;
    {
        const int r = c.lane + 1, each = (p.nt + r - 1) / r, rounds = (apart * r + kChip - 1) / kChip;
        const bool fits = r == 1 || (r <= p.nt && apart * r <= kMostRounds * kChip);
        const int price = fits ? (int)min((int64_t)rounds * (3 * each + 1), (int64_t)1 << 24) * 64 + c.lane : 0x7fffffff;
        ranges = (fold_wave(price, 0x7fffffff, [](int x, int y) { return min(x, y); }) & 63) + 1;
    }
    const int range = (int)blockIdx.x / apart, m = (int)blockIdx.x - range * apart;
    if (m >= rows || range >= ranges) return;
    const int each = (p.nt + ranges - 1) / ranges, nt0 = range * each, tiles = min(each, p.nt - nt0);
    if (tiles <= 0) return;
    int b = 0, mt = m;
    for (int b0 = 0, base = 0; b0 < p.B; b0 += 64) {
        const int mine = b0 + c.lane < p.B ? (min(max(p.kv[b0 + c.lane], 0), p.most) + MT - 1) / MT : 0;
        const int ends = base + scan_incl(mine);
        const uint64_t past = __ballot(ends > m);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            b = b0 + at;
            mt = m - (__builtin_amdgcn_readlane(ends, at) - __builtin_amdgcn_readlane(mine, at));
            break;
        }
        base = __builtin_amdgcn_readlane(ends, 63);
    }
    const int row0 = mt * MT;
    // (a length may be more than the table has pages for: those keys are not there)
    const int counted = min(max(p.kv[b], 0), p.most), kv = min(counted, p.keys);
    auto name = [&](int j, bool there) {
        if (nt0 == 0 && p.places != nullptr && j < counted) p.places[(int64_t)b * p.pl_B + j] = there ? b * p.most + j : -1;
    };
    if (row0 >= kv) {
        if ((int)threadIdx.x < MT) name(row0 + (int)threadIdx.x, false);
        return;
    }
    const int per = p.Dn + p.Dv, cols = per * p.H;
    const int32_t* table = p.table + (int64_t)b * p.t_B;
    const char* base = p.cache;
    // where cached row j lies (an address of zeros where its page is missing; the row of zeros is as long as the
    // widest cached row)
    auto row_at = [&](int j, bool& there) {
        const uint32_t at = fdiv((uint32_t)j, p.fpage), place = (uint32_t)j - at * p.fpage.d;
        const int page = table[at];
        there = (uint32_t)page < (uint32_t)p.pages;
        return at_or_zeros(there, (uint64_t)base + times64((uint32_t)page, p.c_P) + times64(place, p.c_S));
    };
#pragma unroll
    for (int i = 0; i < P::NX; ++i) {
        bool there;
        c.xat[i] = row_at(min(row0 + c.x_row(i), kv - 1), there);
    }
    // which rows of the tile are there: bit r of here[r / 64]
    uint64_t here[MT / 64];
    bool all_here = true;
#pragma unroll
    for (int i = 0; i < MT / 64; ++i) {
        const int j = row0 + i * 64 + c.lane;
        bool there = false;
        if (j < kv) row_at(j, there);
        here[i] = __ballot(there);
        all_here &= here[i] == ~0ull;
        if (c.wave == 0) name(j, there);
    }
    auto is_here = [&](int row) { return (here[row >> 6] >> (row & 63) & 1) != 0; };
    // the columns that all heads share, held for all of them where they are few
    const int pieces = p.Dr / 8;
    const bool held = pieces <= NR * 512 / MT;
    u32x4 rope[NR];
    auto shared_piece = [&](int row, int k) {
        bool there;
        const char* from = (const char*)row_at(row0 + row, there) + (p.Dc + k * 8) * ES;
        u32x4 v;
        if constexpr (X8) v = widen8<E>(*(const u32x2*)from);
        else v = *(const u32x4*)from;
        if (p.ks != 1.0f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = Mat<E>::pack2(Mat<E>::low(v[e]) * p.ks, Mat<E>::high(v[e]) * p.ks);
        }
        return v;
    };
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int n = i * 512 + c.tid;
        rope[i] = u32x4{0, 0, 0, 0};
        if (held && n < MT * pieces && is_here(n / pieces)) rope[i] = shared_piece(n / pieces, n % pieces);
    }
    // (a whole tile of one head makes as many stores in every wave)
    const bool plain = all_here && per == NT && pieces == NR * 512 / MT;
    auto aim = [&](int t) {
#pragma unroll
        for (int i = 0; i < P::NW; ++i) {
            const uint32_t n = (uint32_t)min((nt0 + t) * NT + c.w_row(i), cols - 1), h = fdiv(n, p.fper);
            const int d = (int)(n - h * (uint32_t)per);
            c.wat[i] = d < p.Dn ? (uint64_t)(p.wk + (int64_t)h * p.wk_H + (int64_t)d * p.wk_N)
                                : (uint64_t)(p.wv + (int64_t)h * p.wv_H + (int64_t)(d - p.Dn) * p.wv_N);
        }
    };
    c.template run<P::STORES * (REST ? 2 : 1) + NR>(tiles, p.Dc, 0, aim, [&](int t) {
        const int col0 = (nt0 + t) * NT;
        const uint32_t n = (uint32_t)(col0 + c.out_col()), h = fdiv(n, p.fper);
        const int d = (int)(n - h * (uint32_t)per);
        const bool key = d < p.Dn, in = (int)n < cols;
        char* to = key ? p.ko + (int64_t)b * p.ko_B + (int64_t)row0 * p.ko_S + (int64_t)h * p.ko_H + d * 2
                       : p.vo + (int64_t)b * p.vo_B + (int64_t)row0 * p.vo_S + (int64_t)h * p.vo_H + (d - p.Dn) * 2;
        char* rest = to;
        if constexpr (REST)
            rest = key ? p.kr + (int64_t)b * p.kr_B + (int64_t)row0 * p.kr_S + (int64_t)h * p.kr_H + d * 2
                       : p.vr + (int64_t)b * p.vr_B + (int64_t)row0 * p.vr_S + (int64_t)h * p.vr_H + (d - p.Dn) * 2;
        const int64_t to_S = key ? p.ko_S : p.vo_S, rest_S = key ? p.kr_S : p.vr_S;
        char* ko = p.ko + (int64_t)b * p.ko_B + (int64_t)row0 * p.ko_S + p.Dn * 2;
        if (plain) {
            c.template store<REST, FAR>(p.ks, to, to_S, rest, rest_S, [](int) { return true; });
#pragma unroll
            for (int i = 0; i < NR; ++i) *(u32x4*)(ko + (i * 64 + c.tid / 8) * p.ko_S + (int64_t)(nt0 + t) * p.ko_H + c.tid % 8 * 16) = rope[i];
            return true;
        }
        c.template store<REST, FAR>(p.ks, to, to_S, rest, rest_S, [&](int row) { return in && is_here(row); });
        // the shared columns, of the heads whose first weight row is this tile's
        const int h0 = (col0 + per - 1) / per, h1 = min((min(col0 + NT, cols) + per - 1) / per, p.H);
        if (held) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int n = i * 512 + c.tid;
                if (n < MT * pieces && is_here(n / pieces))
                    for (int e = h0; e < h1; ++e) *(u32x4*)(ko + n / pieces * p.ko_S + (int64_t)e * p.ko_H + n % pieces * 16) = rope[i];
            }
        } else {
            for (int i = c.tid; i < MT * pieces; i += 512) {
                const int row = i / pieces, k = i - row * pieces;
                if (!is_here(row)) continue;
                const u32x4 v = shared_piece(row, k);
                for (int e = h0; e < h1; ++e) *(u32x4*)(ko + row * p.ko_S + (int64_t)e * p.ko_H + k * 16) = v;
            }
        }
        return false;
    });
}

int64_t tiles_of(int64_t n, int64_t each) { return (n + each - 1) / each; }

// How many of `all` tiles a workgroup takes where `slots` run at once: the rounds of the longest, each with a tile's
// worth of start and end.
int64_t share_of(int64_t all, int64_t slots) {
    int64_t best = 1, price = tiles_of(all, slots) * 2;
    for (int64_t rounds = 1; rounds <= 4; ++rounds) {
        const int64_t each = tiles_of(all, slots * rounds), now = tiles_of(tiles_of(all, each), slots) * (each + 1);
        if (now < price) {
            price = now;
            best = each;
        }
    }
    return best;
}

// Results of an eighth of the Infinity Cache and more go out with the nontemporal hint.  In the expansion the size is
// that of the buffers (without the rests), since the host knows no lengths: a few keys in large ones take as long with
// the hint as without (300 keys of 128 heads 30 and 34 us, attention over them 66 and 69).
bool far_out(int64_t bytes) { return bytes >= (int64_t(1) << 25); }

// Tiles of 64 x 64 for few tokens, and where those of 128 x 128 leave half the chip without one; larger ones read
// rows and weights half as often.  (Values of 64 tokens, 128 heads 7.2 us in small tiles, 8.4 in large ones; of 128
// tokens 10.3 and 9.0, queries of 256 17.4 and 14.1; values of 256 and 512 tokens of 16 heads 7.0 and 8.4.)
bool few_rows(int64_t T, int64_t H, int64_t N) { return T <= 64 || tiles_of(T, 128) * H * tiles_of(N, 128) < 128; }

template <typename E, int MT, int NT, int ST> hipError_t project(const ProjectArgs& arg, bool turned, hipStream_t stream) {
    ProjectArgs a = arg;
    const int64_t nt = tiles_of(a.N, NT), all = tiles_of(a.T, MT) * a.H * nt;
    a.fnt = dcp::make_fastdiv((uint32_t)nt);
    a.tiles = (int32_t)all;
    a.each = (int32_t)share_of(all, 512);
    const dim3 grid((uint32_t)tiles_of(all, a.each)), block(256);
    const bool far = far_out((int64_t)a.T * a.H * a.N * 2);
    if (turned)
        return far ? launch(project_rows<E, MT, NT, ST, true, true>, grid, block, stream, a)
                   : launch(project_rows<E, MT, NT, ST, true, false>, grid, block, stream, a);
    return far ? launch(project_rows<E, MT, NT, ST, false, true>, grid, block, stream, a)
               : launch(project_rows<E, MT, NT, ST, false, false>, grid, block, stream, a);
}

}  // namespace

int64_t project_tiles(int64_t T, int64_t H, int64_t N) {
    const int64_t each = few_rows(T, H, N) ? 64 : 128;
    return tiles_of(T, each) * H * tiles_of(N, each);
}
int64_t expand_workgroups(int64_t B, int64_t most, bool rest) {
    // (row tiles 8 apart, or as many workgroups as columns are cut for; the kernel finds how many there are)
    const int64_t rows = (B * tiles_of(most, expand_rows_of(rest)) + 7) / 8 * 8;
    return rows > kMostRounds * kChip ? rows : kMostRounds * kChip;
}

hipError_t launch_project(const ProjectArgs& a, bool turned, bool bf16, hipStream_t stream) {
    auto run = [&](auto e) {
        using E = decltype(e);
        return few_rows(a.T, a.H, a.N) ? project<E, 64, 64, 4>(a, turned, stream) : project<E, 128, 128, 2>(a, turned, stream);
    };
    return bf16 ? run(BF16T{}) : run(F16T{});
}

hipError_t launch_expand(const ExpandArgs& arg, bool bf16, bool x8, hipStream_t stream) {
    ExpandArgs a = arg;
    a.nt = (int32_t)tiles_of((int64_t)a.H * (a.Dn + a.Dv), NT);
    const dim3 grid((uint32_t)expand_workgroups(a.B, a.most, a.kr != nullptr)), block(512);
    auto run = [&](auto e) {
        using E = decltype(e);
        auto with = [&](auto k8, auto far) {
            constexpr bool X8 = decltype(k8)::value, FAR = decltype(far)::value;
            return a.kr != nullptr ? launch(expand_rows<E, X8, true, FAR>, grid, block, stream, a)
                                   : launch(expand_rows<E, X8, false, FAR>, grid, block, stream, a);
        };
        constexpr std::true_type yes{};
        constexpr std::false_type no{};
        if (far_out((int64_t)a.B * a.most * a.H * (a.Dn + a.Dr + a.Dv) * 2)) return x8 ? with(yes, yes) : with(no, yes);
        return x8 ? with(yes, no) : with(no, no);
    };
    return bf16 ? run(BF16T{}) : run(F16T{});
}

}  // namespace dcpa
