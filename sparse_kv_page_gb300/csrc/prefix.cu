// prefix.cu - decode attention of a batch whose sequences share prefixes
// (locks_prefix_attention).
//
// The queries of all sequences of a group meet the group's prefix as rows of one matrix,
// so each prefix key and value is read once for up to 128 (sequence, query head) rows of
// a kv head: S = Q K^T / sqrt(128), running maximum m and sum l per row,
// O = sum exp(S - m) V. A sequence's own tokens are the same product with the g rows of
// its GQA group. Parts of one softmax meet in a second launch by
//   m = max m_i, l = sum l_i e^(m_i - m), O = sum O_i e^(m_i - m), out = O / l.
//
// Work: "units" (a group's prefix, a sequence's own tokens), each an item per kv head and
// block of 128 rows, each item a run of tiles of 128 tokens. All tiles of the call form one
// line, split evenly over one CTA per SM whatever the items are; an item cut by a CTA
// boundary gives one partial (m, l, O) per piece. The line is found on the device from the
// token counts, so a captured graph follows them.
//
// CTA (12 warps): warp 0 loads, warp 1 issues the products, warps 4-7 and 8-11 are two
// softmax groups that take alternate tiles, each with its own running maximum, sum and
// accumulator, so neither waits for the other. Tensor memory: scores of the two groups
// (2 x 128 columns; the bf16 weights overwrite them) and their accumulators (2 x 128).
// Shared memory: Q as a bf16 high and low part (64 KB; fp32 queries keep 16 significant
// bits) and a ring of five 32 KB slots, each a K or a V tile: eight pages of two 64-dim
// halves, one 2 KB TMA box each.
//
// Bound: per 128 x 128 tile the products take 128 * 128 * 128 * (2 + 1) multiply-adds (high
// and low scores, then the values), 1536 cycles at the SM's 4096 a cycle; its 64 KB take
// about 2800 cycles at an SM's share of HBM. Up to 128 rows HBM bounds it, above that the
// tensor cores.
#include <cudaTypedefs.h>

#include <climits>
#include <cstring>

#include "cache_internal.h"
#include "tcgen05.cuh"

namespace locks {
namespace {

constexpr int kTile = 128;                        // tokens per tile, rows per block
constexpr int kTilePages = kTile / kPage;
constexpr int kHalfBytes = kTile * 128;           // 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kBoxBytes = kPage * 128;
constexpr int kSlots = 5;
constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 128;              // per group
constexpr float kScaleLog2 = kInvSqrtD * kLog2e;  // raw score -> exponent of 2
constexpr float kRescale = 8.f / kScaleLog2;      // a running maximum may lag by 2^8

struct Control {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t scores[2];                           // a group's score tile is in tensor memory
    uint64_t weights[2];                          // ... its weights are, and its V rows are ready
    uint64_t queries;                             // Q of the piece is in shared memory
    uint64_t done;                                // every product of the piece has completed
    uint64_t joined;                              // both groups' (m, l) of the piece are in ml
    uint64_t drained;                             // its accumulators and ml have been read
    uint32_t tmem;
    int abort;
    float2 ml[2][kTile];
};
constexpr int kSmemBytes = 2 * kTileBytes + kSlots * kTileBytes + static_cast<int>(sizeof(Control));
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

// Tensor-memory columns.
__host__ __device__ constexpr uint32_t score_col(int x) { return x * 128; }
__host__ __device__ constexpr uint32_t acc_col(int x) { return 256 + x * 128; }

// A wait that gives up after the limit, or once another warp of the CTA has.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Control* ctl, const DeviceStatus& st) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*static_cast<volatile int*>(&ctl->abort)) return false;
            if (global_timer_ns() - t0 > st.wait_limit_ns) {
                *static_cast<volatile int*>(&ctl->abort) = 1;
                report_error(st, LOCKS_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// ----------------------------------------------------------------- the line of tiles

__device__ __forceinline__ int blocks_of(int rows) { return (rows + kTile - 1) / kTile; }

struct Unit {
    int tiles, seq0, num_seqs;      // tiles per item
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
// Group u's prefix. Bounds may not fall: `before` is the largest one ahead (bound_before).
__device__ __forceinline__ Unit group_unit(const PrefixArgs& a, int u, int before) {
    const int s = a.group_start[u], e = a.group_start[u + 1], n = a.prefix_tokens[u];
    const bool span = s >= before && e >= s && e <= a.batch;
    const bool len = n >= 0 && n <= static_cast<int64_t>(a.max_prefix_pages) * kPage;
    Unit r;
    r.seq0 = span ? s : 0;
    r.num_seqs = span ? e - s : 0;
    r.tiles = span && len ? (n + kTile - 1) / kTile : 0;
    r.bad = !span || !len;
    return r;
}
__device__ __forceinline__ Unit own_unit(const PrefixArgs& a, int b) {
    const int n = a.seq_tokens[b];
    const bool len = n >= 0 && n <= static_cast<int64_t>(a.max_pages) * kPage;
    Unit r;
    r.seq0 = b;
    r.num_seqs = 1;
    r.tiles = len ? (n + kTile - 1) / kTile : 0;
    r.bad = !len;
    return r;
}
__device__ __forceinline__ int unit_tokens(const PrefixArgs& a, int u) {
    return u < a.num_groups ? a.prefix_tokens[u] : a.seq_tokens[u - a.num_groups];
}
__device__ __forceinline__ int64_t unit_tiles(const PrefixArgs& a, const Unit& u) {
    return static_cast<int64_t>(u.tiles) * blocks_of(u.num_seqs * (a.hq / a.hkv)) * a.hkv;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }

// 32 units, one a lane, with their places on the line. Whole warps call everything here.
struct Chunk {
    Unit u;
    int64_t tile0, count;           // the unit's first tile and its tiles
    int row0;                       // its first partial row
};
struct Cursor {                     // what lies before a chunk
    int64_t tiles;
    int rows, bound;
};
__device__ __forceinline__ Chunk load_chunk(const PrefixArgs& a, int first, Cursor& at) {
    const int lane = threadIdx.x & 31, u = first + lane;
    const int units = a.num_groups + a.batch;
    Chunk c;
    c.u = Unit{0, 0, 0, false};
    if (first < a.num_groups) {
        const int before = bound_before(u < a.num_groups ? a.group_start[u] : 0, at.bound);
        if (u < a.num_groups) c.u = group_unit(a, u, before);
    }
    if (u >= a.num_groups && u < units) c.u = own_unit(a, u - a.num_groups);
    c.count = unit_tiles(a, c.u);
    const int rows = c.u.num_seqs * a.hq;
    int64_t ts = c.count;
    int rs = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ty = __shfl_up_sync(0xffffffffu, ts, o);
        const int ry = __shfl_up_sync(0xffffffffu, rs, o);
        if (lane >= o) ts += ty, rs += ry;
    }
    c.tile0 = at.tiles + ts - c.count;
    c.row0 = at.rows + rs - rows;
    at.tiles += shfl64(ts, 31);
    at.rows += __shfl_sync(0xffffffffu, rs, 31);
    return c;
}

// First tile of CTA c of n on a line of `total` tiles, and the CTA of a tile.
__host__ __device__ __forceinline__ int64_t cta_first(int64_t total, int c, int n) { return total * c / n; }
__host__ __device__ __forceinline__ int cta_of(int64_t total, int64_t tile, int n) {
    return static_cast<int>(((tile + 1) * n - 1) / total);
}
__host__ __device__ __forceinline__ int ctas_of(int64_t total, int grid) {
    return total < grid ? static_cast<int>(total) : grid;
}

struct Piece {                      // a run of tiles of one item
    const int32_t* table;
    int tokens, kvh, seq0, row0;    // row r of the block: sequence seq0 + (row0 + r) / g, head kvh * g + (row0 + r) % g
    int rows, tile0, tiles;
    int64_t part;                   // its first partial row
};

struct Walk {
    int64_t t, t_end;
    Cursor at;
    int first;                      // of the chunk in hand
    Chunk c;
};

// Positions the walk at this CTA's first tile; false if it has none.
__device__ __forceinline__ bool walk_begin(const PrefixArgs& a, Walk& w) {
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    int bound = 0;
    for (int u0 = 0; u0 < a.num_groups; u0 += 32) {
        const int u = u0 + lane;
        const int before = bound_before(u < a.num_groups ? a.group_start[u] : 0, bound);
        if (u < a.num_groups) sum += unit_tiles(a, group_unit(a, u, before));
    }
#pragma unroll 4
    for (int b = lane; b < a.batch; b += 32) sum += unit_tiles(a, own_unit(a, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int n = ctas_of(sum, gridDim.x), cta = blockIdx.x;
    if (cta >= n) return false;
    w.t = cta_first(sum, cta, n);
    w.t_end = cta_first(sum, cta + 1, n);
    w.at = Cursor{0, 0, 0};
    w.first = 0;
    w.c = load_chunk(a, 0, w.at);
    return true;
}

__device__ __forceinline__ bool walk_next(const PrefixArgs& a, Walk& w, Piece& p) {
    if (w.t >= w.t_end) return false;
    const int g = a.hq / a.hkv;
    while (w.t >= w.at.tiles) {     // ends: t < t_end <= tiles of the line
        w.first += 32;
        w.c = load_chunk(a, w.first, w.at);
    }
    const unsigned in = __ballot_sync(0xffffffffu, w.c.tile0 <= w.t && w.t < w.c.tile0 + w.c.count);
    const int at = __ffs(in) - 1;   // exactly one
    const int tiles = __shfl_sync(0xffffffffu, w.c.u.tiles, at);
    const int seq0 = __shfl_sync(0xffffffffu, w.c.u.seq0, at);
    const int rows = __shfl_sync(0xffffffffu, w.c.u.num_seqs, at) * g;
    const int part0 = __shfl_sync(0xffffffffu, w.c.row0, at);
    const int64_t off = w.t - shfl64(w.c.tile0, at);
    const int u = w.first + at, blocks = blocks_of(rows);
    const int item = static_cast<int>(off / tiles);
    const int rb = item % blocks;
    p.kvh = item / blocks;
    p.tile0 = static_cast<int>(off - static_cast<int64_t>(item) * tiles);
    p.tiles = static_cast<int>(min(static_cast<int64_t>(tiles - p.tile0), w.t_end - w.t));
    p.table = u < a.num_groups ? a.prefix_table + static_cast<int64_t>(u) * a.max_prefix_pages
                               : a.page_table + static_cast<int64_t>(u - a.num_groups) * a.max_pages;
    p.tokens = unit_tokens(a, u);
    p.seq0 = seq0;
    p.row0 = rb * kTile;
    p.rows = min(kTile, rows - p.row0);
    p.part = static_cast<int64_t>(part0) + p.kvh * rows + p.row0 + static_cast<int64_t>(blockIdx.x) * kTile;
    w.t += p.tiles;
    return true;
}

// A piece of n tiles passes through the ring as K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1), the
// order in which the products use it.
__device__ __forceinline__ void ring_entry(int j, int n, bool& is_v, int& tile) {
    if (j < 2 && j < n) {
        is_v = false;
        tile = j;
    } else if (j == 2 * n - 1) {
        is_v = true;
        tile = n - 1;
    } else {
        is_v = (j & 1) == 0;
        tile = is_v ? (j - 2) / 2 : (j + 1) / 2;
    }
}

// ----------------------------------------------------------------------- the loads

__device__ __forceinline__ void run_loads(const PrefixArgs& a, uint8_t* ring, Control* ctl, Walk& w) {
    const int lane = threadIdx.x & 31;
    uint32_t seq = 0;
    bool ok = true;
    Piece p;
    while (ok && walk_next(a, w, p)) {
        // page ids of four tiles at a time, a page a lane: those of the K tile in hand, and
        // the four before for V, which runs at most two tiles behind
        int ids = 0, ids_before = 0, batch = -1;
        const int pages = (p.tokens + kPage - 1) / kPage;
        for (int j = 0; ok && j < 2 * p.tiles; ++j) {
            bool is_v;
            int tile;
            ring_entry(j, p.tiles, is_v, tile);
            if (!is_v && (tile >> 2) != batch) {
                batch = tile >> 2;
                ids_before = ids;
                const int page = (p.tile0 + batch * 4) * kTilePages + lane;
                ids = page < pages ? p.table[page] : 0;
                if (ids < 0 || ids >= a.num_phys) {
                    report_error(a.st, LOCKS_ERR_BAD_INDEX);
                    ids = 0;
                }
            }
            const int from = (tile & 3) * kTilePages + (lane & 7);
            const int id_now = __shfl_sync(0xffffffffu, ids, from);
            const int id_before = __shfl_sync(0xffffffffu, ids_before, from);
            const int id = (tile >> 2) == batch ? id_now : id_before;
            const int slot = seq % kSlots;
            const uint32_t parity = ((seq / kSlots) & 1) ^ 1;
            ok = wait_or_abort(&ctl->empty[slot], parity, ctl, a.st);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int live = min(kTilePages, pages - (p.tile0 + tile) * kTilePages);
            if (lane == 0) mbar_arrive_expect_tx(&ctl->full[slot], live * 2 * kBoxBytes);
            __syncwarp();
            if (lane < 2 * kTilePages && (lane & 7) < live) {
                const int half = lane >> 3;
                tma_load_2d(ring + slot * kTileBytes + half * kHalfBytes + (lane & 7) * kBoxBytes,
                            is_v ? &a.tm_v : &a.tm_k, half * 64, (id * a.hkv + p.kvh) * kPage, &ctl->full[slot]);
            }
            __syncwarp();
            ++seq;
        }
    }
    if (!ok) {
        // giving up: the loads in flight write to this CTA's shared memory, so wait for them
        for (uint32_t s = seq > kSlots ? seq - kSlots : 0; s < seq; ++s)
            mbar_wait_bounded(&ctl->full[s % kSlots], (s / kSlots) & 1, a.st.wait_limit_ns);
    }
}

// -------------------------------------------------------------------- the products

template <bool kSplitQ>
__device__ __forceinline__ void run_products(const PrefixArgs& a, uint32_t q_addr, uint32_t ring_addr, Control* ctl,
                                             Walk& w) {
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = ctl->tmem;
    constexpr uint32_t kScores = bf16_idesc(kTile, kTile, false), kValues = bf16_idesc(kTile, kD, true);
    uint32_t seq = 0, pieces = 0, ready[2] = {0, 0};
    bool ok = true;
    Piece p;
    while (ok && walk_next(a, w, p)) {
        if (lane == 0) {
            auto scores = [&](int x) {            // S_x = Q K^T of the ring's next tile
                const int slot = seq % kSlots;
                if (!wait_or_abort(&ctl->full[slot], (seq / kSlots) & 1, ctl, a.st)) return false;
                tc_fence_after_sync();
                const uint32_t k_addr = ring_addr + slot * kTileBytes;
#pragma unroll
                for (int part = 0; part < (kSplitQ ? 2 : 1); ++part)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = (k >> 2) * kHalfBytes + (k & 3) * 32;
                        mma_ss(tmem + score_col(x), sw128_desc(q_addr + part * kTileBytes + off, 16, 1024),
                               sw128_desc(k_addr + off, 16, 1024), kScores, part + k > 0);
                    }
                mma_commit(&ctl->empty[slot]);
                mma_commit(&ctl->scores[x]);
                ++seq;
                return true;
            };
            ok = wait_or_abort(&ctl->queries, pieces & 1, ctl, a.st);
            if (ok) {
                tc_fence_after_sync();
                ok = scores(0);
            }
            if (ok && p.tiles > 1) ok = scores(1);
            if (ok && pieces > 0) ok = wait_or_abort(&ctl->drained, (pieces - 1) & 1, ctl, a.st);
            for (int i = 0; ok && i < p.tiles; ++i) {
                const int x = i & 1, slot = seq % kSlots;
                ok = wait_or_abort(&ctl->weights[x], ready[x]++ & 1, ctl, a.st) &&
                     wait_or_abort(&ctl->full[slot], (seq / kSlots) & 1, ctl, a.st);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t v_addr = ring_addr + slot * kTileBytes;
#pragma unroll
                for (int k = 0; k < 8; ++k)       // 16 tokens: one page
                    mma_ts(tmem + acc_col(x), tmem + score_col(x) + 8 * k,
                           sw128_desc(v_addr + k * kBoxBytes, kHalfBytes, 1024), kValues, i >= 2 || k > 0);
                mma_commit(&ctl->empty[slot]);
                ++seq;
                if (i + 2 < p.tiles) ok = scores(x);
            }
            mma_commit(&ctl->done);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++pieces;
    }
    // Products may still read shared memory after a wait ran out: their end, bounded.
    if (!ok && lane == 0) mbar_wait_bounded(&ctl->done, (pieces - 1) & 1, a.st.wait_limit_ns);
    __syncwarp();
}

// --------------------------------------------------------------------- the softmax

// Rows of the piece's queries as bf16 high parts (and low parts behind them) in the
// 128-byte swizzle. Rows past p.rows keep what they held: no other row sees them.
template <bool kSplitQ>
__device__ __forceinline__ void write_queries(const PrefixArgs& a, const Piece& p, uint8_t* q_s, int tid) {
    const int g = a.hq / a.hkv;
    for (int i = tid; i < p.rows * 16; i += 2 * kSoftmaxThreads) {
        const int r = i >> 4, c = i & 15;
        const int row = p.row0 + r;
        const int64_t src = (static_cast<int64_t>(p.seq0 + row / g) * a.hq + p.kvh * g + row % g) * kD + c * 8;
        uint8_t* dst = q_s + (c >> 3) * kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        if (kSplitQ) {
            const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + src);
            const float4 u = s[0], v = s[1];
            const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
                lo[e] = pack_bf16x2(x[2 * e] - __uint_as_float(hi[e] << 16),
                                    x[2 * e + 1] - __uint_as_float(hi[e] & 0xffff0000u));
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + kTileBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + src);
        }
    }
}

template <bool kSplitQ>
__device__ __forceinline__ void run_softmax(const PrefixArgs& a, uint8_t* q_s, uint8_t* ring, Control* ctl, Walk& w) {
    const int tid = threadIdx.x - 128;            // 0..255
    const int x = tid >> 7, row = tid & 127;      // softmax group, row of the block (= tensor-memory lane)
    const uint32_t lane_base = ctl->tmem + (static_cast<uint32_t>((tid >> 5) & 3) << 21);
    const int warp_row = row & ~31;
    uint32_t seq = 0, pieces = 0, tiles = 0;
    bool ok = true;
    Piece p;
    while (ok && walk_next(a, w, p)) {
        write_queries<kSplitQ>(a, p, q_s, tid);
        fence_proxy_async_smem();
        mbar_arrive(&ctl->queries);
        const bool busy = warp_row < p.rows;      // some row of this warp is real
        float m = -INFINITY, l = 0.f;
        for (int i = x; i < p.tiles; i += 2) {
            ok = wait_or_abort(&ctl->scores[x], tiles++ & 1, ctl, a.st);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const int valid = min(kTile, p.tokens - (p.tile0 + i) * kTile);
            if (busy) {
                // first pass: the rows' maxima; the scores are read again below (they would take
                // 128 registers in between)
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    tmem_load(r, lane_base + score_col(x) + c * 32);
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        mx[e & 1] = fmaxf(mx[e & 1], c * 32 + e < valid ? __uint_as_float(r[e]) : -INFINITY);
                    top = fmaxf(top, fmaxf(mx[0], mx[1]));
                }
                if (i < 2) {
                    m = top;
                } else if (__any_sync(0xffffffffu, row < p.rows && top > m + kRescale)) {
                    // some row's maximum grew enough to matter: bring its sums over (the other
                    // rows' stay, so that no row's rounding depends on its neighbours)
                    const float to = top > m + kRescale ? top : m;
                    const float f = to == m ? 1.f : fast_exp2((m - to) * kScaleLog2);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_load(r, lane_base + acc_col(x) + c * 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                        tmem_store(lane_base + acc_col(x) + c * 32, r);
                    }
                    l *= f;
                    m = to;
                }
                const float base = m == -INFINITY ? 0.f : m * kScaleLog2;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                // 32 scores become 16 columns of weights, which lie in columns already read
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32], w16[16];
                    tmem_load(r, lane_base + score_col(x) + c * 32);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float u = fast_exp2(fmaf(__uint_as_float(r[2 * e]), kScaleLog2, -base));
                        float v = fast_exp2(fmaf(__uint_as_float(r[2 * e + 1]), kScaleLog2, -base));
                        if (c * 32 + 2 * e >= valid) u = 0.f;
                        if (c * 32 + 2 * e + 1 >= valid) v = 0.f;
                        sum[e & 3] += u + v;
                        w16[e] = pack_bf16x2(u, v);
                    }
                    tmem_store(lane_base + score_col(x) + c * 16, w16);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_store();
            }
            if (valid < kTile) {
                // rows of V past the end weigh 0, but 0 * NaN would still reach the sum
                const uint32_t at = seq + 2 * p.tiles - 1;
                ok = wait_or_abort(&ctl->full[at % kSlots], (at / kSlots) & 1, ctl, a.st);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (row >= valid) {
                    uint8_t* v_row = ring + (at % kSlots) * kTileBytes + row * 128;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(v_row + (c >> 3) * kHalfBytes + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            mbar_arrive(&ctl->weights[x]);
        }
        if (!ok) break;
        seq += 2 * p.tiles;
        ok = wait_or_abort(&ctl->done, pieces & 1, ctl, a.st);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        // the two groups' parts of a row: group x writes its 64 dims of both
        ctl->ml[x][row] = make_float2(m, l);
        mbar_arrive(&ctl->joined);
        ok = wait_or_abort(&ctl->joined, pieces & 1, ctl, a.st);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (busy) {
            const float2 o0 = ctl->ml[0][row], o1 = ctl->ml[1][row];
            const float top = fmaxf(o0.x, o1.x), at = top == -INFINITY ? 0.f : top;
            const float f0 = fast_exp2((o0.x - at) * kScaleLog2);
            const float f1 = p.tiles > 1 ? fast_exp2((o1.x - at) * kScaleLog2) : 0.f;
            float* dst = a.part_o + (p.part + row) * kD + x * 64;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                uint32_t r0[32], r1[32];
                tmem_load(r0, lane_base + acc_col(0) + x * 64 + c * 32);
                if (p.tiles > 1) {
                    tmem_load(r1, lane_base + acc_col(1) + x * 64 + c * 32);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r1[e] = 0;
                }
                if (row < p.rows) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4 o;
                        o.x = __uint_as_float(r0[e]) * f0 + __uint_as_float(r1[e]) * f1;
                        o.y = __uint_as_float(r0[e + 1]) * f0 + __uint_as_float(r1[e + 1]) * f1;
                        o.z = __uint_as_float(r0[e + 2]) * f0 + __uint_as_float(r1[e + 2]) * f1;
                        o.w = __uint_as_float(r0[e + 3]) * f0 + __uint_as_float(r1[e + 3]) * f1;
                        *reinterpret_cast<float4*>(dst + c * 32 + e) = o;
                    }
                }
            }
            if (x == 0 && row < p.rows)
                a.part_ml[p.part + row] = make_float2(top, o0.y * f0 + (p.tiles > 1 ? o1.y * f1 : 0.f));
        }
        // the next piece's values, and so its (m, l), wait for this
        tc_fence_before_sync();
        mbar_arrive(&ctl->drained);
        ++pieces;
    }
}

// Writes where every unit lies for the second launch, and reports bad lengths and bounds.
__device__ __forceinline__ void write_plan(const PrefixArgs& a) {
    const int lane = threadIdx.x & 31, units = a.num_groups + a.batch;
    Cursor at{0, 0, 0};
    for (int first = 0; first < units; first += 32) {
        const Chunk c = load_chunk(a, first, at);
        const int u = first + lane;
        if (u < units) {
            a.units[u] = PrefixUnit{c.tile0, c.row0, c.u.tiles, c.u.seq0, c.u.num_seqs};
            if (c.u.bad) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        }
    }
    if (lane == 0) *a.total = at.tiles;
}

template <bool kSplitQ>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(1024) uint8_t q_s[];   // swizzle atoms: 1024-byte aligned
    uint8_t* ring = q_s + 2 * kTileBytes;
    Control* ctl = reinterpret_cast<Control*>(ring + kSlots * kTileBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&ctl->scores[x], 1);
            mbar_init(&ctl->weights[x], kSoftmaxThreads);
        }
        mbar_init(&ctl->queries, 2 * kSoftmaxThreads);
        mbar_init(&ctl->done, 1);
        mbar_init(&ctl->joined, 2 * kSoftmaxThreads);
        mbar_init(&ctl->drained, 2 * kSoftmaxThreads);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&ctl->tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 2) {
        if (blockIdx.x == 0) write_plan(a);
    } else if (warp != 3) {
        Walk w;
        if (walk_begin(a, w)) {
            if (warp == 0) run_loads(a, ring, ctl, w);
            else if (warp == 1) run_products<kSplitQ>(a, smem_u32(q_s), smem_u32(ring), ctl, w);
            else run_softmax<kSplitQ>(a, q_s, ring, ctl, w);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_free(ctl->tmem, 512);
}

// ------------------------------------------------------------------------ the join

constexpr int kJoinWarps = 4;

// Grid: batch * hkv CTAs; a warp takes every kJoinWarps-th head of the GQA group.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ PrefixArgs a, int grid) {
    __shared__ int group_s;
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x / a.hkv, kvh = blockIdx.x % a.hkv;
    const int lane = threadIdx.x & 31, g = a.hq / a.hkv;
    if (threadIdx.x == 0) group_s = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.num_groups; i += kJoinWarps * 32) {
        const PrefixUnit u = a.units[i];
        if (b >= u.seq0 && b < u.seq0 + u.num_seqs) group_s = i;
    }
    __syncthreads();
    const int64_t total = *a.total;
    const int n = ctas_of(total, grid);
    PrefixUnit pre = {0, 0, 0, 0, 0};
    if (group_s >= 0) pre = a.units[group_s];
    const int rows = pre.num_seqs * g;                      // of the group, per kv head
    const PrefixUnit own = a.units[a.num_groups + b];
    int first_o = 0, count_o = 0;                           // CTAs with a piece of the own tokens
    if (own.tiles > 0) {
        const int64_t t = own.tile0 + static_cast<int64_t>(kvh) * own.tiles;
        first_o = cta_of(total, t, n);
        count_o = cta_of(total, t + own.tiles - 1, n) - first_o + 1;
    }
    for (int h = threadIdx.x >> 5; h < g; h += kJoinWarps) {
        int first_p = 0, count_p = 0;                       // ... and of the prefix, for this row's block
        const int row_in = (b - pre.seq0) * g + h;
        if (pre.tiles > 0) {
            const int64_t item = static_cast<int64_t>(kvh) * blocks_of(rows) + row_in / kTile;
            const int64_t t = pre.tile0 + item * pre.tiles;
            first_p = cta_of(total, t, n);
            count_p = cta_of(total, t + pre.tiles - 1, n) - first_p + 1;
        }
        const int count = count_p + count_o;
        const int64_t row_p = static_cast<int64_t>(pre.row0) + kvh * rows + row_in;
        const int64_t row_o = static_cast<int64_t>(own.row0) + kvh * g + h;
        auto part_row = [&](int i) {
            return i < count_p ? row_p + static_cast<int64_t>(first_p + i) * kTile
                               : row_o + static_cast<int64_t>(first_o + i - count_p) * kTile;
        };
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < count; i0 += 32) {            // 32 pieces at a time, one a lane
            const int i = i0 + lane;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (i < count) ml = a.part_ml[part_row(i)];
            float top = ml.x;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float to = fmaxf(m, top), base = to == -INFINITY ? 0.f : to;
            const float f = fast_exp2((m - base) * kScaleLog2);
            const float wgt = i < count ? fast_exp2((ml.x - base) * kScaleLog2) : 0.f;
            float sum = wgt * ml.y;
            if (i >= count) sum = 0.f;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * f + sum;
            o.x *= f, o.y *= f, o.z *= f, o.w *= f;
            m = to;
            const int here = min(32, count - i0);
#pragma unroll 8
            for (int k = 0; k < here; ++k) {
                const float wk = __shfl_sync(0xffffffffu, wgt, k);
                const float4 v = *reinterpret_cast<const float4*>(a.part_o + part_row(i0 + k) * kD + lane * 4);
                o.x += wk * v.x, o.y += wk * v.y, o.z += wk * v.z, o.w += wk * v.w;
            }
        }
        const float inv = count > 0 ? 1.f / l : 0.f;
        const int64_t row = static_cast<int64_t>(b) * a.hq + kvh * g + h;
        *reinterpret_cast<uint2*>(a.out + row * kD + lane * 4) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (a.lse && lane == 0) a.lse[row] = count > 0 ? fmaf(m, kInvSqrtD, logf(l)) : -INFINITY;
    }
}

PFN_cuTensorMapEncodeTiled_v12000 tiled_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A cache [num_phys][hkv][16][128] as num_phys * hkv * 16 rows, in 64 x 16 boxes.
cudaError_t cache_map(CUtensorMap* map, const uint16_t* base, int64_t rows) {
    const auto fn = tiled_encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kPage)};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(base), dims, strides, box,
                          steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kSplitQ>
cudaError_t launch_prefix_t(const PrefixArgs& a, int grid, cudaStream_t stream) {
    cudaError_t e = ensure_kernel_attrs<prefix_kernel<kSplitQ>>(kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, prefix_kernel<kSplitQ>, a)) != cudaSuccess) return e;
    cfg.gridDim = dim3(a.batch * a.hkv, 1, 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, join_kernel, a, grid)) != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

PrefixLayout prefix_layout(int batch, int hq, int num_groups) {
    // Partial rows: every unit has its own (the groups' are disjoint sequences, so at most
    // batch * hq, and as many for the own tokens), and each CTA boundary moves on by a block.
    const size_t rows = 2 * static_cast<size_t>(batch) * hq + static_cast<size_t>(kMaxPrefixCtas + 1) * kTile;
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    PrefixLayout w;
    w.units = 512;
    w.ml = w.units + up((static_cast<size_t>(num_groups) + batch) * sizeof(PrefixUnit));
    w.o = w.ml + up(rows * sizeof(float2));
    w.bytes = w.o + rows * kD * sizeof(float);
    return w;
}

cudaError_t launch_prefix(const PrefixArgs& args, int num_sms, cudaStream_t stream) {
    PrefixArgs a = args;
    std::memset(&a.tm_k, 0, sizeof(a.tm_k));
    std::memset(&a.tm_v, 0, sizeof(a.tm_v));
    const int64_t rows = static_cast<int64_t>(a.num_phys) * a.hkv * kPage;   // TMA row coordinates are int32
    if (rows > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cache_map(&a.tm_k, a.k_cache, rows);
    if (e == cudaSuccess) e = cache_map(&a.tm_v, a.v_cache, rows);
    if (e != cudaSuccess) return e;
    const int grid = num_sms < kMaxPrefixCtas ? num_sms : kMaxPrefixCtas;
    return a.q_type == LOCKS_FP32 ? launch_prefix_t<true>(a, grid, stream) : launch_prefix_t<false>(a, grid, stream);
}

}  // namespace locks
