// attn_prefix.hpp -- attention of a batch whose sequences share the first keys
// of their caches, group by group.
//
// The rows of all sequences of a group stand together, so against the shared
// keys they are one long sequence: its row tiles take the shared keys once for
// 128 rows of whichever sequences, and every sequence's own tiles take the keys
// behind them.  Both are units of one launch, of the code that single sequences
// run (attn_rows.hpp, attn_latent.hpp, attn_keys.hpp for a sequence's own keys where
// rows are few), which differs only in how a workgroup finds its share and in what
// a row sees: a list that a kernel of one workgroup has made.  A row's parts are
// joined by a third kernel.
//
// The shared keys are bound by matrix instructions as soon as a group has more than
// some 64 rows of a key head, the sequences' own keys by their bytes, so the two fill
// each other's gaps.  64 sequences behind 32768 keys (8192 on this rank), 64 / 8 heads
// of 128: 73 to 78 us, 56 of them the units (floor 24: 148 MB), the rest the list and
// the join; 215 where each sequence reads all of its keys.  Few shared keys do not pay
// for the list: 4 sequences behind 1000 (250 here) take 22 us, by themselves 16; nor do
// sequences of many rows for their parts (sharing_pays()).
#pragma once
#include "attn_common.hpp"

namespace dcpa {

// A workgroup's share: rows of one sequence against its own keys, or rows of a
// group against the keys that its sequences share.
struct GroupUnit : Unit {
    int begin;      // first key
    int end;        // one behind the last shared key (group)
    int b0, b1;     // the group's sequences (none: a sequence's own keys)
    bool even;      // every row of the group sees all shared keys
};
template <int STEP> __device__ __forceinline__ GroupUnit unit_of(const GroupArgs& p, int, int id) {
    const PrefixUnit x = p.list[id];
    GroupUnit u;
    u.s = Seq{x.first, x.n, x.kv, x.len};
    u.b = x.b;
    u.tile = x.tile;
    u.split = x.split;
    u.splits = x.splits;
    u.chunk = x.chunk;
    u.slot = id - x.split;
    u.ok = x.n > 0;
    u.begin = x.begin;
    u.end = x.end;
    u.b0 = x.b0;
    u.b1 = x.b1;
    u.even = x.even != 0;
    return u;
}
__device__ __forceinline__ int first_key(const GroupUnit& u) { return u.begin; }
__device__ __forceinline__ int last_key(const GroupArgs& p, const GroupUnit& u, int last_row) {
    return u.b1 > u.b0 ? u.end : visible(p.m, u.s, (int)fdiv((uint32_t)last_row, p.m.fG));
}
__device__ __forceinline__ int sees(const GroupArgs& p, const GroupUnit& u, int token) {
    if (u.b1 == u.b0) return visible(p.m, u.s, token);
    if (u.even) return u.end;
    // the last sequence that starts at the token's row or before it
    const int t = u.s.first + token;
    int lo = u.b0, hi = u.b1 - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (min(max(p.m.cu[mid], 0), p.m.T) <= t) lo = mid;
        else hi = mid - 1;
    }
    const Seq s = load_seq(p.m, lo);
    return min(visible(p.m, s, t - s.first), u.end);
}
// (rows of several sequences are in no order)
__device__ __forceinline__ int least_seen(const GroupUnit&, int vis) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) vis = min(vis, __shfl_xor(vis, d, 64));
    return __builtin_amdgcn_readfirstlane(vis);
}
__device__ __forceinline__ int most_seen(const GroupUnit&, int vis) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) vis = max(vis, __shfl_xor(vis, d, 64));
    return __builtin_amdgcn_readfirstlane(vis);
}

}  // namespace dcpa
