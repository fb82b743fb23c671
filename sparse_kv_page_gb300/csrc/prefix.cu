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
// token counts, so a captured graph follows them. Short lists, and those of few sequences, take
// one launch of prefix_pages.cu in place of this; own lists of few pages are left to the second
// launch there, and the line holds the prefixes alone.
//
// CTA (16 warps): warp 14 finds the CTA's pieces and announces them to the others, warp 0
// loads K and warp 3 V, warp 1 issues the products with K, warp 2 those with V, warps 4-7 and
// 8-11 are two softmax groups, the other three bring the queries. The CTA's
// tiles are one stream, whatever pieces they belong to: the scores of tile t + 1 are formed
// while the groups weigh tile t, group x its 64 tokens x * 64.., each with a running maximum,
// sum and accumulator of its own, so neither waits for the other; the two are joined into the
// piece's one partial as they are read, while the next piece's scores are formed.
// The roles are apart because each would hold up another: issuing a product or a load box
// blocks until it is taken (one warp for both products took 3600 cycles a tile, one for all
// 32 boxes 2400), and every role finding its own pieces spilled. The code is kept small: behind
// a saturated HBM an instruction fetch from L2 takes microseconds.
// Tensor memory: two score tiles (2 x 128 columns; the weights, a bf16 high and low part each,
// overwrite them) and the groups' accumulators (2 x 128). Shared memory: the queries as a bf16 high part and, for
// fp32, a low part (32 KB each; 16 significant bits together), and a ring of 32 KB slots,
// each a K or a V tile: eight pages of two 64-dim halves, one 2 KB TMA box each.
// Pieces of up to 16 rows (a sequence's own tokens, small groups) take an eighth of the
// query space each, so their queries come ahead of time; the products read 128 rows all the
// same, and what the rows behind a piece's own hold reaches no row but theirs.
//
// The weights meet the values as two bf16 parts too (16 significant bits): as one, their
// rounding would be as large in the output as the output's own, and put its error against 64
// bits at 1.4 times that. One part / two, us: fp32 queries 128K tokens x 16 sequences 91 / 104,
// 1M x 8 (32/2 heads) 170 / 195; bf16 queries 24K x 4 x 32 91.5 / 94.6, 64K x 64 94.7 / 98.2.
// Bound: per 128 x 128 tile the products take 128 * 128 * 128 * (2 + 2) multiply-adds (high
// and low scores, then the values with high and low weights; bf16 queries have no low scores),
// 2048 cycles at the SM's 4096 a cycle; its 64 KB take about 2800 cycles at an SM's share of
// HBM. Each block of 128 rows streams its prefix for itself.
#include <cudaTypedefs.h>

#include <climits>
#include <cstring>

#include "cache_internal.h"
#include "prefix_units.cuh"
#include "tcgen05.cuh"

namespace locks {
namespace {

constexpr int kTilePages = kTile / kPage;
constexpr int kHalfBytes = kTile * 128;           // 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kBoxBytes = kPage * 128;
constexpr int kGroupTokens = kTile / 2;           // of a tile, per softmax group
constexpr int kQueryUnits = kTile / kNarrow;
constexpr int kThreads = 512;
constexpr int kQueryThreads = 96;
constexpr int kPieces = 8;                        // pieces announced ahead
constexpr int kPieceReaders = 15;                 // warps that follow them
constexpr float kRescale = 8.f / kScaleLog2;      // a running maximum may lag by 2^8

// Ring slots: what the queries leave of shared memory.
template <bool kSplitQ>
constexpr int kSlots = kSplitQ ? 5 : 6;
template <bool kSplitQ>
constexpr int kQueryBytes = (kSplitQ ? 2 : 1) * kTileBytes;

struct Piece {                      // a run of tiles of one item
    const int32_t* table;
    int tokens, kvh, seq0, row0;    // row r of the block: sequence seq0 + (row0 + r) / g, head kvh * g + (row0 + r) % g
    int rows, tile0, tiles;         // no tiles: the end
    int64_t part;                   // its first partial row
    uint32_t n;                     // pieces of this CTA before it
    bool once;                      // no other block of rows reads its K and V

    __device__ __forceinline__ bool wide() const { return rows > kNarrow; }
    // of its queries in shared memory
    __device__ __forceinline__ int query_offset() const { return wide() ? 0 : (n % kQueryUnits) * (kNarrow * 128); }
    // tokens of its tile i
    __device__ __forceinline__ int valid(int i) const { return min(kTile, tokens - (tile0 + i) * kTile); }
};

struct Control {
    uint64_t full[6], empty[6];
    uint64_t scores[2];                           // a score tile is in tensor memory
    uint64_t weights[2][2];                       // [group][score tile] its weights are
    uint64_t values[2];                           // [score tile] their products with V have completed
    uint64_t p_full[kPieces], p_free[kPieces];    // a piece is announced; every role has read it
    uint64_t q_full[kQueryUnits];                 // a piece's queries are in shared memory
    uint64_t q_first;                             // ... what the softmax groups bring of the first
    uint64_t q_free[kQueryUnits];                 // its last scores have been formed
    uint64_t last[2];                             // every product with K (with V) of the CTA has completed
    uint64_t joined;                              // both groups' maxima of a piece are in m
    uint32_t tmem;
    int abort;
    uint32_t issued[2];                           // tiles whose K (V) loads were issued
    float m[2][2][kTile];                         // [piece n % 2][group]: see run_softmax
    Piece pieces[kPieces];
};
template <bool kSplitQ>
constexpr int kSmemBytes = kQueryBytes<kSplitQ> + kSlots<kSplitQ> * kTileBytes + static_cast<int>(sizeof(Control));
static_assert(kSmemBytes<true> <= 227 * 1024 && kSmemBytes<false> <= 227 * 1024, "shared memory of one CTA");

// Tensor-memory columns: score tile b, accumulator of group x.
__host__ __device__ constexpr uint32_t score_col(int b) { return b * 128; }
__host__ __device__ constexpr uint32_t acc_col(int x) { return 256 + x * 128; }
constexpr uint32_t kLowWeights = kGroupTokens / 2;   // a group's weights: high parts, then low parts

// A wait that gives up after the limit, or once another warp of the CTA has. Out of line: the
// roles' code together is larger than the nearer instruction caches, and behind a saturated
// HBM a fetch from L2 takes microseconds.
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status,
                                       uint64_t limit_ns) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort = 1;
            if (status) atomicCAS(status, 0, LOCKS_ERR_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Control* ctl, const DeviceStatus& st) {
    if (mbar_try_wait(bar, parity)) return true;
    return slow_wait(smem_u32(bar), parity, &ctl->abort, st.word, st.wait_limit_ns);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Control* ctl, const DeviceStatus& st) {
    const bool ok = wait_or_abort(bar, parity, ctl, st);
    return __all_sync(0xffffffffu, ok) != 0;
}

// What a role that gave up still has in flight: loads and products that were issued end by
// themselves, so this wait is not cut short by a small limit.
constexpr uint64_t kDrainNs = 500000000ull;

// The next piece of the CTA, as warp 14 announced it; false after the last. Whole warps.
__device__ __forceinline__ bool next_piece(Control* ctl, uint32_t& n, Piece& p, const DeviceStatus& st) {
    const int slot = n % kPieces;
    if (!warp_wait(&ctl->p_full[slot], (n / kPieces) & 1, ctl, st)) return false;
    p = ctl->pieces[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->p_free[slot]);
    ++n;
    return p.tiles > 0;
}

// ----------------------------------------------------------------- the line of tiles

// Steps of a unit on the line: an item's cost goes before its tiles.
__device__ __forceinline__ int64_t unit_steps(const PrefixArgs& a, const Unit& u) {
    const int rows = u.num_seqs * (a.group);
    return u.tiles == 0 ? 0 : static_cast<int64_t>(u.tiles + item_cost(rows)) * blocks_of(rows) * a.hkv;
}

// Units on the line: the groups' prefixes and, unless the second launch attends to them, the
// sequences' own tokens.
__device__ __forceinline__ int line_units(const PrefixArgs& a) { return a.num_groups + (a.own_apart ? 0 : a.batch); }

// 32 units, one a lane, with their places on the line. Whole warps call everything here.
struct Chunk {
    Unit u;
    int64_t step0, count;           // the unit's first step and its steps
    int row0;                       // its first partial row
};
struct Cursor {                     // what lies before a chunk
    int64_t steps;
    int rows, bound;
};
__device__ __noinline__ Chunk load_chunk(const PrefixArgs& a, int first, Cursor& at) {
    const int lane = threadIdx.x & 31, u = first + lane;
    const int units = line_units(a);
    Chunk c;
    c.u = Unit{0, 0, 0, 0, false};
    const bool own = u >= a.num_groups && u < units;
    const int own_tokens = own ? a.seq_tokens[u - a.num_groups] : 0;
    if (first < a.num_groups) {
        const bool group = u < a.num_groups;
        const int start = group ? a.group_start[u] : 0, end = group ? a.group_start[u + 1] : 0;
        const int tokens = group ? a.prefix_tokens[u] : 0;
        const int before = bound_before(start, at.bound);
        if (group) c.u = group_unit(a, start, end, tokens, before);
    }
    if (own) c.u = own_unit(a, u - a.num_groups, own_tokens);
    c.count = unit_steps(a, c.u);
    const int rows = c.u.num_seqs * a.hq;
    int64_t ts = c.count;
    int rs = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ty = __shfl_up_sync(0xffffffffu, ts, o);
        const int ry = __shfl_up_sync(0xffffffffu, rs, o);
        if (lane >= o) ts += ty, rs += ry;
    }
    c.step0 = at.steps + ts - c.count;
    c.row0 = at.rows + rs - rows;
    at.steps += shfl64(ts, 31);
    at.rows += __shfl_sync(0xffffffffu, rs, 31);
    return c;
}

struct Walk {
    int64_t t, t_end;
    Cursor at;
    int first;                      // of the chunk in hand
    uint32_t pieces;                // so far
    Chunk c;
};

// Positions the walk at this CTA's first step; false if it has none. Calls of up to 32 units
// know the whole line from their first chunk.
__device__ __forceinline__ bool walk_begin(const PrefixArgs& a, Walk& w) {
    const int lane = threadIdx.x & 31;
    w.at = Cursor{0, 0, 0};
    w.first = 0;
    w.pieces = 0;
    w.c = load_chunk(a, 0, w.at);
    int64_t sum = 0;
    int bound = w.at.bound;
#pragma unroll 1
    for (int u0 = 32; u0 < a.num_groups; u0 += 32) {
        const int u = u0 + lane;
        const int start = u < a.num_groups ? a.group_start[u] : 0;
        const int before = bound_before(start, bound);
        if (u < a.num_groups)
            sum += unit_steps(a, group_unit(a, start, a.group_start[u + 1], a.prefix_tokens[u], before));
    }
#pragma unroll 1
    for (int b = max(32 - a.num_groups, 0) + lane; b < line_units(a) - a.num_groups; b += 32) sum += unit_steps(a, own_unit(a, b, a.seq_tokens[b]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum += w.at.steps;
    const int n = ctas_of(sum, gridDim.x), cta = blockIdx.x;
    if (cta >= n) return false;
    w.t = cta_first(sum, cta, n);
    w.t_end = cta_first(sum, cta + 1, n);
    return true;
}

__device__ __forceinline__ bool walk_next(const PrefixArgs& a, Walk& w, Piece& p) {
    const int g = a.group;
    int at, tiles, rows, cost, step;
    int64_t item;
    for (;;) {
        if (w.t >= w.t_end) return false;
        while (w.t >= w.at.steps) { // ends: t < t_end <= steps of the line
            w.first += 32;
            w.c = load_chunk(a, w.first, w.at);
        }
        const unsigned in = __ballot_sync(0xffffffffu, w.c.step0 <= w.t && w.t < w.c.step0 + w.c.count);
        at = __ffs(in) - 1;         // exactly one
        tiles = __shfl_sync(0xffffffffu, w.c.u.tiles, at);
        rows = __shfl_sync(0xffffffffu, w.c.u.num_seqs, at) * g;
        cost = item_cost(rows);
        const int64_t off = w.t - shfl64(w.c.step0, at);
        item = divide(off, tiles + cost);
        step = static_cast<int>(off - item * (tiles + cost));
        if (step >= cost) break;
        w.t += cost - step;         // the item's first tile, if it is this CTA's
    }
    const int seq0 = __shfl_sync(0xffffffffu, w.c.u.seq0, at);
    const int part0 = __shfl_sync(0xffffffffu, w.c.row0, at);
    const int u = w.first + at, blocks = blocks_of(rows);
    const int rb = static_cast<int>(item) % blocks;
    p.kvh = static_cast<int>(item) / blocks;
    p.tile0 = step - cost;
    p.tiles = static_cast<int>(min(static_cast<int64_t>(tiles - p.tile0), w.t_end - w.t));
    p.table = u < a.num_groups ? a.prefix_table + static_cast<int64_t>(u) * a.max_prefix_pages
                               : a.page_table + static_cast<int64_t>(u - a.num_groups) * a.max_pages;
    p.tokens = __shfl_sync(0xffffffffu, w.c.u.tokens, at);
    p.seq0 = seq0;
    p.row0 = rb * kTile;
    p.rows = min(kTile, rows - p.row0);
    p.part = static_cast<int64_t>(part0) + p.kvh * rows + p.row0 + static_cast<int64_t>(blockIdx.x) * kTile;
    p.n = w.pieces++;
    p.once = blocks == 1;
    w.t += p.tiles;
    return true;
}

// The order of the ring: K of tile t + 1 comes before V of tile t. (The entry of the K that
// would follow the last tile stays empty.)
__device__ __forceinline__ uint32_t k_entry(uint32_t t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ uint32_t v_entry(uint32_t t) { return 2 * t + 2; }

// ----------------------------------------------------------------------- the loads

// The loads of K (kValues false) or of V, a warp each: a box takes about 75 cycles to issue,
// so one warp for the 32 boxes of a tile would bound the supply.
// With an odd ring the two take turns in a slot, and a wait for one use's end by its parity would
// take the end of the use two before for it; so that one has to be seen before. Entry e's loader
// last waited for entry e - 7. Where e is K of tile t, that is V of tile t - 5, whose products
// followed that tile's scores, and e - 10, its K, was handed back ahead of the scores. Where e
// is V of tile t, it is K of tile t - 2, whose scores followed the products of tile t - 4,
// issued after e - 10, V of tile t - 5, had been handed back.
template <bool kSplitQ, bool kValues>
__device__ __forceinline__ void run_loads(const PrefixArgs& a, uint8_t* ring, Control* ctl) {
    constexpr uint32_t kN = kSlots<kSplitQ>;
    const int lane = threadIdx.x & 31;
    const uint64_t first_out = policy_evict_first(), normal = policy_evict_normal();
    uint32_t t = 0, pieces = 0;                   // tiles and pieces so far
    bool ok = true;
    Piece p;
    while (ok && next_piece(ctl, pieces, p, a.st)) {
        const int pages = (p.tokens + kPage - 1) / kPage;
        int ids = 0;                              // of four tiles, a page a lane
        for (int i = 0; i < p.tiles; ++i) {
            if ((i & 3) == 0) {
                const int page = (p.tile0 + i) * kTilePages + lane;
                ids = page < pages ? p.table[page] : 0;
                if (ids < 0 || ids >= a.num_phys) {
                    report_error(a.st, LOCKS_ERR_BAD_INDEX);
                    ids = 0;
                }
            }
            // lanes 0-7 load the pages' first halves, lanes 8-15 the second
            const int id = __shfl_sync(0xffffffffu, ids, (i & 3) * kTilePages + (lane & 7));
            const int live = min(kTilePages, pages - (p.tile0 + i) * kTilePages);
            const uint32_t seq = kValues ? v_entry(t) : k_entry(t), slot = seq % kN;
            ok = wait_or_abort(&ctl->empty[slot], ((seq / kN) & 1) ^ 1, ctl, a.st);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl->full[slot], live * 2 * kBoxBytes);
            __syncwarp();
            if (lane < 2 * kTilePages && (lane & 7) < live) {
                const int half = lane >> 3;
                tma_load_2d_hint(ring + slot * kTileBytes + half * kHalfBytes + (lane & 7) * kBoxBytes,
                                 kValues ? &a.tm_v : &a.tm_k, half * 64, (id * a.hkv + p.kvh) * kPage,
                                 &ctl->full[slot], p.once ? first_out : normal);
            }
            __syncwarp();
            ++t;
        }
    }
    if (lane == 0) ctl->issued[kValues] = t;
}

// After a role has given up, wherever it did: the loads in flight write to this CTA's shared
// memory, which has to stay until they have landed. A warp, once every role has ended: lane s
// waits for the last entry that was loaded into slot s (what was there before was used up, so
// it had landed; entries of a slot follow one another without a gap, so entry e is its phase
// e / kN). The last entry of a slot is among the last kN tiles of K or of V.
template <bool kSplitQ>
__device__ __noinline__ void drain_loads(Control* ctl) {
    constexpr int kN = kSlots<kSplitQ>;
    const int slot = threadIdx.x & 31;
    int last = -1;
    for (int back = 1; back <= kN; ++back) {
        const int k = static_cast<int>(ctl->issued[0]) - back, v = static_cast<int>(ctl->issued[1]) - back;
        if (k >= 0 && static_cast<int>(k_entry(k) % kN) == slot) last = max(last, static_cast<int>(k_entry(k)));
        if (v >= 0 && static_cast<int>(v_entry(v) % kN) == slot) last = max(last, static_cast<int>(v_entry(v)));
    }
    if (slot < kN && last >= 0) mbar_wait_bounded(&ctl->full[slot], (last / kN) & 1, kDrainNs);
}

// --------------------------------------------------------------------- the queries

// Rows first, first + step, ... of a piece's queries as bf16 high parts (and low parts behind
// them) in the 128-byte swizzle: a narrow piece in unit p.n % 8 (16 rows), a wide one from the
// first unit on. Rows past the piece's keep what they held. Sixteen threads a row, a 16-byte
// chunk each (thread % 16), four rows in flight.
template <bool kSplitQ>
__device__ __noinline__ void write_queries(const void* queries, int hq, int g, int kvh, int seq0, int row0, int rows,
                                           uint8_t* dst, int first, int step) {
    constexpr int kInFlight = 4;
    constexpr int kWords = kSplitQ ? 2 : 1;                 // 16-byte loads a chunk
    const int c = threadIdx.x & 15;
    const float per_g = 1.f / g;                            // rows stay below 2^20: (row + 1/2) / g is exact enough
    dst += (c >> 3) * kHalfBytes;
#pragma unroll 1
    for (int r = first; r < rows; r += kInFlight * step) {
        uint4 in[kInFlight][kWords];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int row = row0 + r + u * step;
            const int seq = static_cast<int>((static_cast<float>(row) + 0.5f) * per_g), h = row - seq * g;
            const int64_t src = (static_cast<int64_t>(seq0 + seq) * hq + kvh * g + h) * kD + c * 8;
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(queries) + src * (kSplitQ ? 4 : 2));
            if (r + u * step < rows) {
#pragma unroll
                for (int k = 0; k < kWords; ++k) in[u][k] = s[k];
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int at = r + u * step;
            if (at >= rows) continue;
            uint8_t* to = dst + at * 128 + (((c & 7) ^ (at & 7)) << 4);
            if (kSplitQ) {
                const uint4 v0 = in[u][0], v1 = in[u][kWords - 1];
                const float x[8] = {__uint_as_float(v0.x), __uint_as_float(v0.y), __uint_as_float(v0.z),
                                    __uint_as_float(v0.w), __uint_as_float(v1.x), __uint_as_float(v1.y),
                                    __uint_as_float(v1.z), __uint_as_float(v1.w)};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
                    lo[e] = pack_bf16x2(x[2 * e] - __uint_as_float(hi[e] << 16),
                                        x[2 * e + 1] - __uint_as_float(hi[e] & 0xffff0000u));
                }
                *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(to + kTileBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            } else {
                *reinterpret_cast<uint4*>(to) = in[u][0];
            }
        }
    }
    fence_proxy_async_smem();
}

// The first piece's queries are brought by the softmax groups too, which have nothing else to
// do yet: by the three query warps alone 128 rows take 6 us, longer than the ring lasts.
constexpr int kFirstRows = (kQueryThreads + 256) / 16;      // rows that all of them take at once

template <bool kSplitQ>
__device__ __forceinline__ void run_queries(const PrefixArgs& a, uint8_t* q_s, Control* ctl) {
    // warps 12, 13 and 15
    const int tid = threadIdx.x < 14 * 32 ? threadIdx.x - 12 * 32 : threadIdx.x - 13 * 32;
    uint32_t pieces = 0;
    uint32_t freed = 0;                           // pieces whose scores are known to be formed
    uint32_t after_wide = 0;                      // 1 + the last wide piece
    Piece p;
    while (next_piece(ctl, pieces, p, a.st)) {
        // a narrow piece follows its unit's last user and any wide piece; a wide one, all
        const uint32_t need = p.wide() ? p.n : max(after_wide, p.n >= kQueryUnits ? p.n - kQueryUnits + 1 : 0u);
        for (; freed < need; ++freed)
            if (!warp_wait(&ctl->q_free[freed % kQueryUnits], (freed / kQueryUnits) & 1, ctl, a.st)) return;
        write_queries<kSplitQ>(a.q, a.hq, a.group, p.kvh, p.seq0, p.row0, p.rows, q_s + p.query_offset(), tid >> 4,
                               p.n == 0 ? kFirstRows : kQueryThreads / 16);
        mbar_arrive(&ctl->q_full[p.n % kQueryUnits]);
        if (p.wide()) after_wide = p.n + 1;
    }
}

// -------------------------------------------------------------------- the products

// In both the whole warp keeps step and its first lane issues.

// Whatever the warp issued reads shared and tensor memory: sees its end.
__device__ __forceinline__ void end_products(uint64_t* bar) {
    if ((threadIdx.x & 31) == 0) {
        mma_commit(bar);
        mbar_wait_bounded(bar, 0, kDrainNs);
    }
    __syncwarp();
}

// S = Q K^T, over each tile's live pages alone.
template <bool kSplitQ>
__device__ __forceinline__ void run_scores(const PrefixArgs& a, uint32_t q_addr, uint32_t ring_addr, Control* ctl) {
    constexpr uint32_t kN = kSlots<kSplitQ>;
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = ctl->tmem;
    uint32_t t = 0, pieces = 0;                   // tiles and pieces so far
    bool ok = true;
    Piece p;
    while (ok && next_piece(ctl, pieces, p, a.st)) {
        ok = warp_wait(&ctl->q_full[p.n % kQueryUnits], (p.n / kQueryUnits) & 1, ctl, a.st);
        const uint32_t q_at = q_addr + p.query_offset();
        if (p.n == 0) ok = ok && warp_wait(&ctl->q_first, 0, ctl, a.st);
        for (int i = 0; ok && i < p.tiles; ++i, ++t) {
            const uint32_t seq = k_entry(t), slot = seq % kN, b = t & 1;
            // the weights of tile t - 2 lie where these scores go
            if (t >= 2) ok = warp_wait(&ctl->values[b], ((t >> 1) - 1) & 1, ctl, a.st);
            ok = ok && warp_wait(&ctl->full[slot], (seq / kN) & 1, ctl, a.st);
            if (!ok) break;
            tc_fence_after_sync();
            if (lane == 0) {
                const uint32_t idesc = bf16_idesc(kTile, (p.valid(i) + kPage - 1) / kPage * kPage, false);
                const uint32_t k_addr = ring_addr + slot * kTileBytes;
                const uint64_t q_desc = sw128_desc(q_at, 16, 1024), k_desc = sw128_desc(k_addr, 16, 1024);
#pragma unroll
                for (int part = 0; part < (kSplitQ ? 2 : 1); ++part)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
                        mma_ss(tmem + score_col(b), q_desc + (part * (kTileBytes >> 4) + off), k_desc + off, idesc,
                               part + k > 0);
                    }
                mma_commit(&ctl->empty[slot]);          // first: see run_loads
                mma_commit(&ctl->scores[b]);
                if (i == p.tiles - 1) mma_commit(&ctl->q_free[p.n % kQueryUnits]);
            }
        }
    }
    end_products(&ctl->last[0]);
}

// O_x += P_x V, over each tile's live pages alone.
template <bool kSplitQ>
__device__ __forceinline__ void run_values(const PrefixArgs& a, uint8_t* ring, Control* ctl) {
    constexpr uint32_t kN = kSlots<kSplitQ>;
    constexpr uint32_t kValues = bf16_idesc(kTile, kD, true);
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = ctl->tmem;
    uint32_t t = 0, pieces = 0;                   // tiles and pieces so far
    bool ok = true;
    Piece p;
    while (ok && next_piece(ctl, pieces, p, a.st)) {
        for (int i = 0; ok && i < p.tiles; ++i, ++t) {
            const uint32_t seq = v_entry(t), slot = seq % kN, b = t & 1;
            const int valid = p.valid(i), live = (valid + kPage - 1) / kPage;
            ok = warp_wait(&ctl->full[slot], (seq / kN) & 1, ctl, a.st);
            if (!ok) break;
            if (valid % kPage != 0) {
                // rows of the last page past the end weigh 0, but 0 * NaN would still reach the sums
                uint8_t* rows = ring + slot * kTileBytes + valid * 128;
                for (int j = lane; j < (live * kPage - valid) * 16; j += 32)
                    *reinterpret_cast<uint4*>(rows + (j & 8) * (kHalfBytes / 8) + (j >> 4) * 128 + (j & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            const uint32_t v_addr = smem_u32(ring) + slot * kTileBytes;
            // both groups read both accumulators of the piece before
            if (i == 0) ok = warp_wait(&ctl->weights[1][b], (t >> 1) & 1, ctl, a.st);
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                ok = ok && warp_wait(&ctl->weights[x][b], (t >> 1) & 1, ctl, a.st);
                if (!ok) break;
                tc_fence_after_sync();
                if (lane == 0) {
                    const uint64_t v = sw128_desc(v_addr + x * (kTilePages / 2) * kBoxBytes, kHalfBytes, 1024);
                    const uint32_t w = tmem + score_col(b) + x * kGroupTokens;
                    const auto page = [&](int k) {                // 16 tokens
                        mma_ts(tmem + acc_col(x), w + 8 * k, v + k * (kBoxBytes >> 4), kValues, i > 0 || k > 0);
                        mma_ts(tmem + acc_col(x), w + kLowWeights + 8 * k, v + k * (kBoxBytes >> 4), kValues, true);
                    };
                    if (live == kTilePages) {
#pragma unroll
                        for (int k = 0; k < kTilePages / 2; ++k) page(k);
                    } else {
#pragma unroll 1
                        for (int k = 0; k < min(kTilePages / 2, live - x * (kTilePages / 2)); ++k) page(k);
                    }
                }
            }
            if (ok && lane == 0) {
                mma_commit(&ctl->values[b]);
                mma_commit(&ctl->empty[slot]);
            }
        }
    }
    end_products(&ctl->last[1]);
}

// --------------------------------------------------------------------- the softmax

// The softmax groups' share of the first piece's queries. (The piece stays announced until they
// have read it for themselves.)
template <bool kSplitQ>
__device__ __forceinline__ void help_queries(const PrefixArgs& a, uint8_t* q_s, Control* ctl) {
    if (!warp_wait(&ctl->p_full[0], 0, ctl, a.st)) return;
    const Piece& p = ctl->pieces[0];
    if (p.tiles > 0)
        write_queries<kSplitQ>(a.q, a.hq, a.group, p.kvh, p.seq0, p.row0, p.rows, q_s + p.query_offset(),
                               kQueryThreads / 16 + ((threadIdx.x - 128) >> 4), kFirstRows);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->q_first);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t bits2(float2 v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 d;\n\tfma.rn.f32x2 d, %2, %3, %4;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "l"(bits2(a)), "l"(bits2(make_float2(b, b))), "l"(bits2(c)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 d;\n\tadd.rn.f32x2 d, %2, %3;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "l"(bits2(a)), "l"(bits2(b)));
    return r;
}

__device__ __forceinline__ void run_softmax(const PrefixArgs& a, Control* ctl) {
    const int tid = threadIdx.x - 128;            // 0..255
    const int x = tid >> 7, row = tid & 127;      // softmax group, row of the block (= tensor-memory lane)
    const int lane = tid & 31;
    const uint32_t lane_base = ctl->tmem + (static_cast<uint32_t>((tid >> 5) & 3) << 21);
    const uint32_t acc = lane_base + acc_col(x);  // of this group
    uint32_t t = 0, pieces = 0;                   // tiles and pieces so far
    Piece p;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, ctl, a.st); };
    while (next_piece(ctl, pieces, p, a.st)) {
        const bool busy = (row & ~31) < p.rows;   // some row of this warp is real
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < p.tiles; ++i, ++t) {
            const int b = t & 1;
            const int valid = p.valid(i) - x * kGroupTokens;      // tokens of this group; may be none
            if (!wait(&ctl->scores[b], (t >> 1) & 1)) return;
            tc_fence_after_sync();
            if (busy && valid > 0) {
                const uint32_t tile = lane_base + score_col(b) + x * kGroupTokens;
                float s[kGroupTokens];
                {
                    uint32_t r[kGroupTokens];
                    tmem_load(r, tile);
#pragma unroll
                    for (int e = 0; e < kGroupTokens; ++e) s[e] = __uint_as_float(r[e]);
                }
                if (valid < kGroupTokens) {
#pragma unroll
                    for (int e = 0; e < kGroupTokens; ++e) s[e] = e < valid ? s[e] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int e = 4; e < kGroupTokens; ++e) mx[e & 3] = fmaxf(mx[e & 3], s[e]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (i == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, row < p.rows && top > m + kRescale)) {
                    // some row's maximum grew enough to matter: bring its sums over (the other
                    // rows' stay, so that no row's rounding depends on its neighbours), once the
                    // values of the tile before are in
                    const float to = top > m + kRescale ? top : m;
                    const float f = to == m ? 1.f : fast_exp2((m - to) * kScaleLog2);
                    if (!wait(&ctl->values[b ^ 1], ((t - 1) >> 1) & 1)) return;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_load(r, acc + c * 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                        tmem_store(acc + c * 32, r);
                    }
                    l *= f;
                    m = to;
                }
                const float base = m == -INFINITY ? 0.f : m * kScaleLog2;
                float2 sum[4] = {};
#pragma unroll
                for (int c = 0; c < kGroupTokens; c += 32) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 u =
                            fma2(make_float2(s[c + 2 * e], s[c + 2 * e + 1]), kScaleLog2, make_float2(-base, -base));
                        const float2 w = make_float2(fast_exp2(u.x), fast_exp2(u.y));
                        sum[e & 3] = add2(sum[e & 3], w);
                        hi[e] = pack_bf16x2(w.x, w.y);
                        const float2 rest = fma2(
                            make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xffff0000u)), -1.f, w);
                        lo[e] = pack_bf16x2(rest.x, rest.y);
                    }
                    tmem_store(tile + c / 2, hi);
                    tmem_store(tile + kLowWeights + c / 2, lo);
                }
                const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += all.x + all.y;
                tmem_wait_store();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->weights[x][b]);
        }
        // the piece's partial, once its last products are in: group x brings 64 dims of both
        // groups' sums to the larger maximum. Pieces take turns with two copies of the maxima: a
        // group may be done with the next piece's weights while the other has yet to read this
        // one's, but the copy is written again only after `joined` of the piece between, where
        // the other arrives after its read.
        float(&tops)[2][kTile] = ctl->m[p.n & 1];
        tops[x][row] = m;
        const int64_t at = p.part + row;
        if (row < p.rows) a.part_ml[at * 2 + x] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->joined);
        if (!wait(&ctl->values[(t - 1) & 1], ((t - 1) >> 1) & 1)) return;
        if (!wait(&ctl->joined, p.n & 1)) return;
        tc_fence_after_sync();
        if (busy) {
            const float m0 = tops[0][row], m1 = tops[1][row], top = fmaxf(m0, m1);
            const float base = top == -INFINITY ? 0.f : top;
            const float f0 = fast_exp2((m0 - base) * kScaleLog2), f1 = fast_exp2((m1 - base) * kScaleLog2);
            const bool second = p.tiles > 1 || p.valid(0) > kGroupTokens;     // else group 1 holds nothing
            float* dst = a.part_o + at * kD + x * kGroupTokens;
#pragma unroll 1
            for (int c = 0; c < kGroupTokens; c += 16) {
                uint32_t r[16], r1[16];
                tmem_load(r, lane_base + acc_col(0) + x * 64 + c);
                tmem_load(r1, lane_base + acc_col(1) + x * 64 + c);
                if (row < p.rows) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        r[e] = __float_as_uint(__uint_as_float(r[e]) * f0 +
                                               (second ? __uint_as_float(r1[e]) * f1 : 0.f));
                    store_v8(dst + c, &r[0]);
                    store_v8(dst + c + 8, &r[8]);
                }
            }
            // the next piece's products overwrite the accumulators once both groups' weights have arrived
            tc_fence_before_sync();
        }
    }
}

// Announces the CTA's pieces, and their end.
template <bool kSplitQ>
__device__ __forceinline__ void run_pieces(const PrefixArgs& a, Control* ctl) {
    const int lane = threadIdx.x & 31;
    Walk w;
    Piece p;
    const uint64_t keep = policy_evict_last();
    bool more = walk_begin(a, w);
    for (uint32_t n = 0;; ++n) {
        more = more && walk_next(a, w, p);
        const int slot = n % kPieces;
        if (n >= kPieces && !warp_wait(&ctl->p_free[slot], ((n / kPieces) & 1) ^ 1, ctl, a.st)) return;
        if (lane == 0) {
            if (!more) p.tiles = 0;
            ctl->pieces[slot] = p;
            mbar_arrive(&ctl->p_full[slot]);
        }
        if (more && n > 0) {
            // its queries (g rows of each sequence, side by side) into L2, to stay: behind a
            // saturated HBM a load takes several us, and a wide piece's come in three rounds
            const int g = a.group, bytes = g * kD * (kSplitQ ? 4 : 2);
            for (int s = p.row0 / g + lane; s * g < p.row0 + p.rows; s += 32)
                prefetch_l2_kept(static_cast<const uint8_t*>(a.q) +
                                     (static_cast<int64_t>(p.seq0 + s) * a.hkv + p.kvh) * bytes,
                                 bytes, keep);
        }
        __syncwarp();
        if (!more) return;
    }
}

// Writes where every sequence's tiles lie for the second launch, and reports bad lengths and
// bounds. One warp.
__device__ __forceinline__ void write_plan(const PrefixArgs& a) {
    const int lane = threadIdx.x & 31, units = line_units(a);
    for (int b = lane; b < a.batch; b += 32) a.seqs[b].pre_tiles = 0;
    __syncwarp();
    Cursor at{0, 0, 0};
    for (int first = 0; first < units; first += 32) {
        const Chunk c = load_chunk(a, first, at);
        const int u = first + lane;
        if (u < units && c.u.bad) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        if (u >= a.num_groups && u < units) {
            PrefixSeq& s = a.seqs[u - a.num_groups];
            s.own_step0 = c.step0;
            s.own_row0 = c.row0;
            s.own_tiles = c.u.tiles;
        }
        for (unsigned left = __ballot_sync(0xffffffffu, u < a.num_groups && c.u.tiles > 0); left; left &= left - 1) {
            const int from = __ffs(left) - 1;               // a group: all lanes write its sequences
            const int64_t step0 = shfl64(c.step0, from);
            const int row0 = __shfl_sync(0xffffffffu, c.row0, from);
            const int tiles = __shfl_sync(0xffffffffu, c.u.tiles, from);
            const int seq0 = __shfl_sync(0xffffffffu, c.u.seq0, from);
            const int num = __shfl_sync(0xffffffffu, c.u.num_seqs, from);
            for (int i = lane; i < num; i += 32) {
                PrefixSeq& s = a.seqs[seq0 + i];
                s.pre_step0 = step0;
                s.pre_row0 = row0;
                s.pre_tiles = tiles;
                s.pre_seq0 = seq0;
                s.pre_num_seqs = num;
            }
        }
    }
    if (lane == 0) *a.total = at.steps;
}

template <bool kSplitQ>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(1024) uint8_t q_s[];   // swizzle atoms: 1024-byte aligned
    uint8_t* ring = q_s + kQueryBytes<kSplitQ>;
    Control* ctl = reinterpret_cast<Control*>(ring + kSlots<kSplitQ> * kTileBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots<kSplitQ>; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->scores[b], 1);
            mbar_init(&ctl->values[b], 1);
            for (int x = 0; x < 2; ++x) mbar_init(&ctl->weights[x][b], 4);   // a warp each
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&ctl->p_full[i], 1);
            mbar_init(&ctl->p_free[i], kPieceReaders);
        }
        for (int i = 0; i < kQueryUnits; ++i) {
            mbar_init(&ctl->q_full[i], kQueryThreads);
            mbar_init(&ctl->q_free[i], 1);
        }
        mbar_init(&ctl->q_first, 8);                        // a warp each
        mbar_init(&ctl->joined, 8);                         // a warp each
        mbar_init(&ctl->last[0], 1);
        mbar_init(&ctl->last[1], 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&ctl->tmem, 512);
    if (warp == 0 && (threadIdx.x & 31) == 0) prefetch_tensor_map(&a.tm_k);
    if (warp == 3 && (threadIdx.x & 31) == 0) prefetch_tensor_map(&a.tm_v);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) run_loads<kSplitQ, false>(a, ring, ctl);
    else if (warp == 1) run_scores<kSplitQ>(a, smem_u32(q_s), smem_u32(ring), ctl);
    else if (warp == 2) run_values<kSplitQ>(a, ring, ctl);
    else if (warp == 3) run_loads<kSplitQ, true>(a, ring, ctl);
    else if (warp < 12) {
        help_queries<kSplitQ>(a, q_s, ctl);
        run_softmax(a, ctl);
    }
    else if (warp != 14) run_queries<kSplitQ>(a, q_s, ctl);
    else {
        run_pieces<kSplitQ>(a, ctl);
        if (blockIdx.x == 0) write_plan(a);               // off the way: the others still work
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0 && ctl->abort) drain_loads<kSplitQ>(ctl);
    if (warp == 1) tmem_free(ctl->tmem, 512);
}

// ------------------------------------------------------------------------ the join

// kWarps warps join the partials of one (sequence, query head): each takes every kWarps-th
// batch, whose partials are in flight together (8 of them, 16 where a row has a CTA to itself),
// and they meet in shared memory. The time is the latency of a few dependent loads.
constexpr int kJoinThreads = 256;


template <int kWarps>
__global__ void __launch_bounds__(kJoinThreads, kWarps == 8 ? 2 : 4)
    join_kernel(const __grid_constant__ PrefixArgs a, int grid) {
    constexpr int kJoinBatch = kWarps == 8 ? 16 : 8;
    constexpr int kRowsPerCta = kJoinThreads / 32 / kWarps;
    __shared__ float2 ml_s[kJoinThreads / 32];
    __shared__ float4 o_s[kJoinThreads / 32][32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = a.group;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + warp / kWarps;
    const bool live = row < static_cast<int64_t>(a.batch) * a.hq;
    const int b = live ? static_cast<int>(row / a.hq) : 0, head = static_cast<int>(row % a.hq);
    const int kvh = head / g, h = head % g;
    const int64_t total = *a.total;
    const PrefixSeq s = a.seqs[b];
    const int n = ctas_of(total, grid);
    int first_o = 0, count_o = 0;                           // CTAs with a piece of the own tokens
    if (s.own_tiles > 0) {
        const int cost = item_cost(g);
        const int64_t t = s.own_step0 + static_cast<int64_t>(kvh) * (s.own_tiles + cost) + cost;
        first_o = cta_of(total, t, n);
        count_o = cta_of(total, t + s.own_tiles - 1, n) - first_o + 1;
    }
    const PrefixRows p = prefix_rows(a, s, b, kvh, h, total, n);
    const int count = live ? p.count + count_o : 0;
    const int64_t row_o = static_cast<int64_t>(s.own_row0) + kvh * g + h;
    auto part_row = [&](int i) {
        return i < p.count ? p.row + static_cast<int64_t>(i) * kTile
                           : row_o + static_cast<int64_t>(first_o + i - p.count) * kTile;
    };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = (warp % kWarps) * kJoinBatch; i0 < count; i0 += kWarps * kJoinBatch)
        join_partials<kJoinBatch>(a, part_row, i0, count, m, l, o);
    if (kWarps > 1) {
        if (lane == 0) ml_s[warp] = make_float2(m, l);
        o_s[warp][lane] = o;
        __syncthreads();
        if (warp % kWarps != 0) return;                     // else: ml_s[warp] on are the row's
        m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml_s[warp + w].x);
        const float base = m == -INFINITY ? 0.f : m;
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2((ml_s[warp + w].x - base) * kScaleLog2);
            const float4 v = o_s[warp + w][lane];
            l += f * ml_s[warp + w].y;
            o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
        }
    }
    if (!live) return;
    const float inv = count > 0 ? 1.f / l : 0.f;
    *reinterpret_cast<uint2*>(a.out + row * kD + lane * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[row] = count > 0 ? fmaf(m, kInvSqrtD, logf(l)) : -INFINITY;
}

template <bool kSplitQ>
cudaError_t launch_prefix_t(const PrefixArgs& a, int grid, cudaStream_t stream) {
    cudaError_t e = ensure_kernel_attrs<prefix_kernel<kSplitQ>>(kSmemBytes<kSplitQ>);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes<kSplitQ>;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, prefix_kernel<kSplitQ>, a)) != cudaSuccess) return e;
    if (a.own_apart) return launch_own(a, grid, stream);
    // The fewer rows, the more pieces each has: a prefix row of n blocks of 128 in all has about
    // grid / n. A CTA per row up to two rows an SM, half a CTA up to sixteen, a warp beyond. The
    // whole call, CTA / half CTA a row: 256 rows (1M x 8 sequences) 170.2 / 174.8 us, 2048 rows
    // (64K x 64) 114.3 / 100.1.
    const int64_t rows = static_cast<int64_t>(a.batch) * a.hq;
    const int warps = rows <= 2 * grid ? 8 : rows < 16 * grid ? 4 : 1, per_cta = kJoinThreads / 32 / warps;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta), 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    e = warps == 8   ? cudaLaunchKernelEx(&cfg, join_kernel<8>, a, grid)
        : warps == 4 ? cudaLaunchKernelEx(&cfg, join_kernel<4>, a, grid)
                     : cudaLaunchKernelEx(&cfg, join_kernel<1>, a, grid);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
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

}  // namespace

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

PrefixLayout prefix_layout(int batch, int hq) {
    // Partial rows: every unit has its own (the groups' are disjoint sequences, so at most
    // batch * hq, and as many for the own tokens), and each CTA boundary moves on by a block.
    const size_t rows = 2 * static_cast<size_t>(batch) * hq + static_cast<size_t>(kMaxPrefixCtas + 1) * kTile;
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    PrefixLayout w;
    w.seqs = 512;
    w.ml = w.seqs + up(static_cast<size_t>(batch) * sizeof(PrefixSeq));
    w.o = w.ml + up(rows * 2 * sizeof(float2));
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
    if (prefix_is_small(a, num_sms)) return launch_prefix_small(a, num_sms, stream);
    const int grid = num_sms < kMaxPrefixCtas ? num_sms : kMaxPrefixCtas;
    a.own_alone = list_by_pages(a, num_sms);
    if (a.own_alone) return launch_own(a, grid, stream);
    a.own_apart = own_by_pages(a, num_sms);
    return a.q_type == LOCKS_FP32 ? launch_prefix_t<true>(a, grid, stream) : launch_prefix_t<false>(a, grid, stream);
}

}  // namespace locks
