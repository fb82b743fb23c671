// prefix_units.cuh - what both kernels of the shared-prefix attention take from the caller's
// counts: a group's prefix or a sequence's own tokens, with lengths and bounds checked.
#pragma once

#include "cache_internal.h"

namespace locks {

constexpr int kTile = 128;                        // tokens per tile, rows per block
constexpr float kScaleLog2 = kInvSqrtD * kLog2e;  // raw score -> exponent of 2

struct Unit {
    int tokens, tiles, seq0, num_seqs;            // tiles per item
    bool bad;
};
// The largest group bound ahead of this lane's, given the largest one before the warp's
// (`bound`, at least 0), which moves on past the warp's own.
__device__ __forceinline__ int bound_before(int mine, int& bound) {
    const int lane = threadIdx.x & 31;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = max(upto, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, upto, 1);
    const int at = bound;
    bound = max(bound, __shfl_sync(0xffffffffu, upto, 31));
    return lane == 0 ? at : max(before, at);
}
// A group's prefix: sequences s..e, n tokens. Bounds may not fall: `before` is the largest one
// ahead (bound_before).
__device__ __forceinline__ Unit group_unit(const PrefixArgs& a, int s, int e, int n, int before) {
    const bool span = s >= before && e >= s && e <= a.batch;
    const bool len = n >= 0 && n <= static_cast<int64_t>(a.max_prefix_pages) * kPage;
    Unit r;
    r.seq0 = span ? s : 0;
    r.num_seqs = span ? e - s : 0;
    r.tokens = span && len ? n : 0;
    r.tiles = (r.tokens + kTile - 1) / kTile;
    r.bad = !span || !len;
    return r;
}
__device__ __forceinline__ Unit own_unit(const PrefixArgs& a, int b, int n) {
    const bool len = n >= 0 && n <= static_cast<int64_t>(a.max_pages) * kPage;
    Unit r;
    r.seq0 = b;
    r.num_seqs = 1;
    r.tokens = len ? n : 0;
    r.tiles = (r.tokens + kTile - 1) / kTile;
    r.bad = !len;
    return r;
}
}  // namespace locks
