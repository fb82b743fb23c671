// prefix_units.cuh - what the kernels of the shared-prefix attention share: the units taken
// from the caller's counts (a group's prefix or a sequence's own tokens, with lengths and
// bounds checked), the line of tiles that is cut into CTAs, and the joining of partials.
#pragma once

#include "cache_internal.h"

namespace locks {

constexpr int kTile = 128;                        // tokens per tile, rows per block
constexpr int kNarrow = 16;                       // rows of a piece that takes one query unit
constexpr float kScaleLog2 = kInvSqrtD * kLog2e;  // raw score -> exponent of 2

struct Unit {
    int tokens, tiles, seq0, num_seqs;            // tiles per item
    bool bad;
};
// Lists may be as long as 2^31 - 16 tokens: no sum before the division.
__device__ __forceinline__ int tiles_of(int tokens) { return tokens / kTile + (tokens % kTile != 0); }
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
    r.tiles = tiles_of(r.tokens);
    r.bad = !span || !len;
    return r;
}
__device__ __forceinline__ Unit own_unit(const PrefixArgs& a, int b, int n) {
    const bool len = n >= 0 && n <= static_cast<int64_t>(a.max_pages) * kPage;
    Unit r;
    r.seq0 = b;
    r.num_seqs = 1;
    r.tokens = len ? n : 0;
    r.tiles = tiles_of(r.tokens);
    r.bad = !len;
    return r;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }

// The line is counted in steps: one per tile, and ahead of an item's tiles what starting it
// costs, in tiles: its queries, its partials, a pipeline that fills. A wide item's queries
// wait for the ones before to be used up.
constexpr int kNarrowCost = 1, kWideCost = 6;
__device__ __forceinline__ int item_cost(int rows) { return rows > kNarrow ? kWideCost : kNarrowCost; }

__device__ __forceinline__ int blocks_of(int rows) { return (rows + kTile - 1) / kTile; }

// First step of CTA c of n on a line of `total` steps, and the CTA of a step. (32-bit division
// where it will do: a 64-bit one is a long routine, kept in one place.)
static __device__ __noinline__ int64_t divide64(int64_t x, int64_t y) { return x / y; }
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    if (x < (1ll << 32) && y < (1ll << 32)) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return divide64(x, y);
}
__device__ __forceinline__ int64_t cta_first(int64_t total, int c, int n) { return divide(total * c, n); }
__device__ __forceinline__ int cta_of(int64_t total, int64_t step, int n) {
    return static_cast<int>(divide((step + 1) * n - 1, total));
}
__device__ __forceinline__ int ctas_of(int64_t total, int grid) {
    return total < grid ? static_cast<int>(total) : grid;
}

// The partials of a prefix for query h of a group's kv head: one per CTA that holds tiles of
// its block of rows, a block of partial rows apart.
struct PrefixRows {
    int count;
    int64_t row;                    // of the first
};
__device__ __forceinline__ PrefixRows prefix_rows(const PrefixArgs& a, const PrefixSeq& s, int b, int kvh, int h,
                                                  int64_t total, int ctas) {
    PrefixRows r = {0, 0};
    if (s.pre_tiles > 0) {
        const int rows = s.pre_num_seqs * a.group, row_in = (b - s.pre_seq0) * a.group + h;
        const int64_t item = static_cast<int64_t>(kvh) * blocks_of(rows) + row_in / kTile;
        const int cost = item_cost(rows);
        const int64_t t = s.pre_step0 + item * (s.pre_tiles + cost) + cost;
        const int first = cta_of(total, t, ctas);
        r.count = cta_of(total, t + s.pre_tiles - 1, ctas) - first + 1;
        r.row = static_cast<int64_t>(s.pre_row0) + kvh * rows + row_in + static_cast<int64_t>(first) * kTile;
    }
    return r;
}

// Adds partials i0 .. i0 + kBatch of `count` to a row's maximum, sum and accumulator (four dims
// a lane). All loads of a batch are in flight together.
template <int kBatch, class PartRow>
__device__ __forceinline__ void join_partials(const PrefixArgs& a, const PartRow& part_row, int i0, int count, float& m,
                                              float& l, float4& o) {
    const int lane = threadIdx.x & 31;
    const int here = min(kBatch, count - i0);
    const int64_t at = part_row(i0 + min(lane, here - 1));       // a partial a lane
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t r = shfl64(at, k);
        if (k < here) v[k] = *reinterpret_cast<const float4*>(a.part_o + r * kD + lane * 4);
    }
    // either softmax group's maximum and sum; the accumulator goes by the larger maximum
    float4 ml = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    if (lane < here) ml = *reinterpret_cast<const float4*>(a.part_ml + at * 2);
    const float mine = fmaxf(ml.x, ml.z);
    float top = mine;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float to = fmaxf(m, top), base = to == -INFINITY ? 0.f : to;
    const float f = fast_exp2((m - base) * kScaleLog2);
    const float wgt = lane < here ? fast_exp2((mine - base) * kScaleLog2) : 0.f;
    float sum = lane < here ? fast_exp2((ml.x - base) * kScaleLog2) * ml.y +
                                  fast_exp2((ml.z - base) * kScaleLog2) * ml.w
                            : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * f + sum;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    m = to;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wgt, k);
        if (k < here) o.x += wk * v[k].x, o.y += wk * v[k].y, o.z += wk * v[k].z, o.w += wk * v[k].w;
    }
}

}  // namespace locks
