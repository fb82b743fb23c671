// pool.cu - the page pool's calls (locks_pool.h): copying, forking, taking, freeing and
// compacting pages.
//
// Which pages are free follows from the reference counts alone, so the calls that look for
// free pages (fork, take) or rank the used ones (compact) scan them in two launches: one counts
// them by blocks of the pool (and plans, in a block of its own, who needs how many pages), the
// next knows every page's rank from the blocks' counts and places it. For small pools one block does
// both. A call is short, a few MB at most, so what bounds it are the launches and the loads that wait
// for one another; each launch starts while the one before it runs. Measured: freeing pages of 3
// sequences and taking some for 29 others in a pool of 16K pages 7.9 us; of 48 x 8192 pages in a pool
// of 1M 18.3; forking 2 x 64 rows of 8188 pages and copying the last ones 13.8; compacting a pool of 2048
// pages, with the copies, 8.6.
#include <algorithm>

#include "pool_internal.h"

namespace locks {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kRound = 4 * kThreads;                  // pages, or entries of a row, that a block takes at a time
constexpr int kScanRows = 2048;                       // rows whose sums lie in shared memory

__device__ __forceinline__ bool in_table(int tokens, int max_pages) {
    return tokens >= 0 && tokens <= static_cast<int64_t>(max_pages) * kPage;
}
__device__ __forceinline__ int pages_of(int tokens) { return tokens / kPage + (tokens % kPage != 0); }

// Block i of the pool: pages first .. last, a multiple of kRound but for the pool's end.
struct Segment {
    int first, last;
};
__host__ __device__ inline int pool_blocks(int pages) {
    const int n = (pages + kRound - 1) / kRound;
    return n < kMaxPoolBlocks ? n : kMaxPoolBlocks;
}
__device__ __forceinline__ Segment segment_of(int pages, int i) {
    const int64_t blocks = max(1, pool_blocks(pages));
    const int64_t per = (pages + blocks * kRound - 1) / (blocks * kRound) * kRound;
    return {static_cast<int>(min(i * per, static_cast<int64_t>(pages))),
            static_cast<int>(min((i + 1) * per, static_cast<int64_t>(pages)))};
}
// Counts of pages at .. at + 3 (a lane's), those past `last` as if held by nobody and not free.
__device__ __forceinline__ int4 load4(const int32_t* refs, int at, int last) {
    if (at + 4 <= last) return __ldcg(reinterpret_cast<const int4*>(refs + at));
    int4 r;                                           // (at may be past the end altogether)
    r.x = at < last ? __ldcg(refs + at) : INT32_MIN;
    r.y = at + 1 < last ? __ldcg(refs + at + 1) : INT32_MIN;
    r.z = at + 2 < last ? __ldcg(refs + at + 2) : INT32_MIN;
    r.w = INT32_MIN;
    return r;
}
__device__ __forceinline__ void store4(int32_t* refs, int at, int last, const int4& r) {
    if (at + 4 <= last) {
        *reinterpret_cast<int4*>(refs + at) = r;
        return;
    }
    if (at < last) refs[at] = r.x;
    if (at + 1 < last) refs[at + 1] = r.y;
    if (at + 2 < last) refs[at + 2] = r.z;
}
// Bit k: page at + k is free / used (neither past the end, whose counts are INT32_MIN, below those a
// caller may have).
__device__ __forceinline__ unsigned free4(const int4& r) {
    const auto is = [](int x) { return x <= 0 && x != INT32_MIN; };
    return (is(r.x) ? 1u : 0u) | (is(r.y) ? 2u : 0u) | (is(r.z) ? 4u : 0u) | (is(r.w) ? 8u : 0u);
}
__device__ __forceinline__ unsigned used4(const int4& r) {
    return (r.x > 0 ? 1u : 0u) | (r.y > 0 ? 2u : 0u) | (r.z > 0 ? 4u : 0u) | (r.w > 0 ? 8u : 0u);
}
__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
__device__ __forceinline__ int warp_upto(int x) {     // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(kAll, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ int block_sum(int x, int* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = warp_sum(x);
    if (lane == 0) scratch[warp] = x;
    __syncthreads();
    x = warp_sum(scratch[lane]);
    __syncthreads();
    return x;
}

// Counts pages of a kind (free4 or used4) in block i of the pool, and copies the counts to refs_out
// on the way where that is another array. `flags`: keeps which they are, four pages a byte (the next
// launch may change the counts in place while it looks for the pages).
template <typename Kind>
__device__ __forceinline__ int count_block(const PoolArgs& a, int i, Kind kind, bool flags, int* scratch) {
    const Segment seg = segment_of(a.num_pages, i);
    const bool copy = a.refs_out != a.refs;
    int n = 0;
#pragma unroll 2
    for (int at = seg.first + 4 * threadIdx.x; at < seg.last; at += kRound) {
        const int4 r = load4(a.refs, at, seg.last);
        const unsigned bits = kind(r);
        n += __popc(bits);
        if (flags) a.flags[at / 4] = static_cast<uint8_t>(bits);
        if (copy) store4(a.refs_out, at, seg.last, r);
    }
    n = block_sum(n, scratch);
    if (threadIdx.x == 0) a.block_counts[i] = n;
    return n;
}

// How many of the kind are before block i of the pool, and in all.
__device__ __forceinline__ void join_counts(const PoolArgs& a, int i, int* scratch, int& before, int& total) {
    const int blocks = pool_blocks(a.num_pages), tid = threadIdx.x;
    const int n = tid < blocks ? __ldcg(a.block_counts + tid) : 0;
    before = block_sum(tid < i ? n : 0, scratch);
    total = block_sum(n, scratch);
}
static_assert(kMaxPoolBlocks <= kThreads, "a thread per block of the pool");

// Calls f(page, rank) for the pages in a segment that bits_at(page of a lane's four) flags, ranks counted
// from `rank`, up to rank `most`: neighbouring threads get neighbouring ranks, through `list`, so that
// what goes by the rank is written together (200K pages taken from 1M by each lane's own: 12.0 us,
// through the list 10.2). own(page, bits) is called before by the lane whose four pages those are.
template <typename Bits, typename Own, typename F>
__device__ __forceinline__ void walk_segment(const Segment& seg, int rank, int most, int* scratch, uint16_t* list, Bits bits_at,
                                             Own own, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int at0 = seg.first; at0 < seg.last && rank < most; at0 += kRound) {
        const int at = at0 + 4 * threadIdx.x;
        const unsigned bits = at < seg.last ? bits_at(at) : 0u;
        const int upto = warp_upto(__popc(bits));
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        const int sums = scratch[lane], all = warp_sum(sums), n = min(all, most - rank);
        int r = upto - __popc(bits) + warp_sum(lane < warp ? sums : 0);
        unsigned taken = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (bits >> k & 1u) {
                if (r < n) list[r] = static_cast<uint16_t>(4 * threadIdx.x + k), taken |= 1u << k;
                ++r;
            }
        if (taken) own(at, taken);
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) f(at0 + list[i], rank + i);
        rank += all;
        __syncthreads();
    }
}
__device__ __forceinline__ auto flags_at(const PoolArgs& a) {
    return [&a](int at) -> unsigned { return __ldcg(a.flags + at / 4); };
}

// Sums over the batch, by one block: calls put(b, sum of count(0..b), count(b), extra) for every row in
// turn of its thread, with the extra number that count(b, extra) gave; returns the sum of all. Sums stop
// at kMany, which no pool has: all the rows' needs together may pass 31 bits.
constexpr int kMany = (1 << 30) + 1;
__device__ __forceinline__ int add_up(int x, int y) {
    return static_cast<int>(min(static_cast<unsigned>(x) + static_cast<unsigned>(y), static_cast<unsigned>(kMany)));
}
__device__ __forceinline__ int add_upto(int x) {      // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(kAll, x, o);
        if ((threadIdx.x & 31) >= o) x = add_up(x, y);
    }
    return x;
}
template <typename Count, typename Put>
__device__ __forceinline__ int scan_rows(int batch, int* scratch, Count count, Put put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int extra = 0;
        const int mine = b < batch ? count(b, extra) : 0;
        int upto = add_upto(mine);
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        const int sums = add_upto(scratch[lane]);
        const int before = __shfl_sync(kAll, sums, max(warp - 1, 0));
        upto = add_up(upto, add_up(base, warp > 0 ? before : 0));
        if (b < batch) put(b, upto, mine, extra);
        base = add_up(base, __shfl_sync(kAll, sums, 31));
        __syncthreads();
    }
    return base;
}

// ------------------------------------------------------------------ small pools
//
// One block does a call on a small pool whole, in one launch: the counts stay in its registers, what
// the rows need in shared memory, and a warp takes a piece of a row. Measured (graphs of calls, us, one
// block / two or three launches; pool, rows x entries): taking 500, 8 x 31 4.1 / 5.4, 16000, 32 x 250 4.5 /
// 5.9; forking 500, 8 x 31 4.3 / 6.7, 8000, 32 x 125 7.0 / 7.2, 16000, 32 x 250 9.7 / 7.6; compacting 500,
// 8 x 31 3.8 / 6.5, 8000, 32 x 125 8.6 / 10.6. (Freeing into another array, 500 2.4 / 2.7, 16000 4.9 / 2.9,
// has two launches always.)
constexpr int kOneRounds = 4, kTakePages = kOneRounds * kRound, kForkPages = 2 * kRound, kOneBatch = kThreads;
constexpr int kMovePages = 2 * kRound;                // ids of 16 bits in shared memory
constexpr int kWarpPiece = 4 * 32, kOnePieces = 2 * kWarps;
__host__ __device__ inline int warp_pieces(int entries) { return entries > kWarpPiece ? (entries + kWarpPiece - 1) / kWarpPiece : 1; }

// Bits (free4 or used4) of a lane's pages, four of each round, and the counts copied on the way.
template <typename Kind>
__device__ __forceinline__ unsigned one_bits(const PoolArgs& a, Kind kind) {
    const bool copy = a.refs_out != a.refs;
    int4 r[kOneRounds];
    unsigned bits = 0u;
#pragma unroll
    for (int k = 0; k < kOneRounds; ++k) r[k] = load4(a.refs, k * kRound + 4 * threadIdx.x, a.num_pages);
#pragma unroll
    for (int k = 0; k < kOneRounds; ++k) {
        bits |= kind(r[k]) << (4 * k);
        if (copy) store4(a.refs_out, k * kRound + 4 * threadIdx.x, a.num_pages, r[k]);
    }
    return bits;
}
// f(row, first entry of this lane; its others are 32, 64 and 96 further on) for all pieces of all rows.
template <typename F>
__device__ __forceinline__ void each_piece(int rows, int entries, F f) {
    const int pieces = warp_pieces(entries);
    for (int x = threadIdx.x >> 5; x < rows * pieces; x += kWarps) f(x / pieces, (x % pieces) * kWarpPiece + (threadIdx.x & 31));
}

// ------------------------------------------------------------------ take

// A lane's four pages, of which `taken` get a holder. (Nobody else changes the counts meanwhile.)
__device__ __forceinline__ auto hold_taken(const PoolArgs& a) {
    return [&a](int at, unsigned taken) {
        int4 r = load4(a.refs, at, a.num_pages);
        if (taken & 1u) r.x = 1;
        if (taken & 2u) r.y = 1;
        if (taken & 4u) r.z = 1;
        if (taken & 8u) r.w = 1;
        store4(a.refs_out, at, a.num_pages, r);
    };
}
// Pages that row b needs; -1: its counts are wrong.
__device__ __forceinline__ int pages_needed(const PoolArgs& a, int b) {
    const int old = __ldcg(a.seq_tokens + b), now = __ldcg(a.new_tokens + b);
    if (!in_table(old, a.max_pages) || !in_table(now, a.max_pages) || now < old) return -1;
    return pages_of(now) - pages_of(old);
}

// First launch: free pages, by block of the pool; pages needed by rows 0..b, and what turns the rank
// of a free page into its place in the row.
__global__ void __launch_bounds__(kThreads) take_count_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps];
    grid_dependency_wait();
    allow_dependent_launch();
    if (blockIdx.x > 0) {
        count_block(a, blockIdx.x - 1, free4, true, scratch);
        return;
    }
    scan_rows(a.batch, scratch,
              [&](int b, int& old) {
                  const int need = pages_needed(a, b);
                  old = need > 0 ? pages_of(__ldcg(a.seq_tokens + b)) : 0;
                  return max(0, need);
              },
              [&](int b, int sum, int mine, int old) {
                  a.scan[b] = sum;
                  a.shift[b] = old - (sum - mine);
              });
}

__global__ void __launch_bounds__(kThreads) take_place_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps], near_upto[kScanRows], near_shift[kScanRows], served;
    __shared__ uint16_t list[kRound];
    const int tid = threadIdx.x, blocks = pool_blocks(a.num_pages), block = blockIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    int before, free;
    join_counts(a, block, scratch, before, free);
    // rows whose pages are all there: those before the first that lacks some
    int taken = a.batch > 0 ? __ldcg(a.scan + a.batch - 1) : 0;
    if (taken > free) {
        if (tid == 0) served = 0;
        __syncthreads();
        int mine = 0;
        for (int b = tid; b < a.batch; b += kThreads) {
            const int upto = __ldcg(a.scan + b);
            if (upto <= free) mine = max(mine, upto);
        }
        if (mine > 0) atomicMax(&served, mine);
        __syncthreads();
        taken = served;
    }
    if (block < blocks && before < taken) {
        const bool near = a.batch <= kScanRows;
        if (near) {
            for (int b = tid; b < a.batch; b += kThreads) near_upto[b] = __ldcg(a.scan + b), near_shift[b] = __ldcg(a.shift + b);
            __syncthreads();
        }
        const int* const upto = near ? near_upto : a.scan;
        const int* const shift = near ? near_shift : a.shift;
        int lo = 0;                                   // the first row whose sum passes r, which only grows
        walk_segment(segment_of(a.num_pages, block), before, taken, scratch, list, flags_at(a), hold_taken(a), [&](int page, int r) {
            if (upto[lo] <= r) {
                int hi = a.batch - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (upto[mid] > r) hi = mid;
                    else lo = mid + 1;
                }
            }
            a.page_table_out[static_cast<int64_t>(lo) * a.max_pages + shift[lo] + r] = page;
        });
    }
    for (int b = block * kThreads + tid; b < a.batch; b += gridDim.x * kThreads) {
        const int need = pages_needed(a, b);
        int tokens = __ldcg(a.seq_tokens + b);
        if (need < 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        else if (need > 0 && __ldcg(a.scan + b) > free) report_error(a.st, LOCKS_ERR_NO_PAGES);
        else tokens = __ldcg(a.new_tokens + b);
        a.seq_tokens_out[b] = tokens;
    }
    if (a.n_free && block == 0 && tid == 0) *a.n_free = free - taken;
}

__global__ void __launch_bounds__(kThreads, 1) take_one_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps], upto[kOneBatch], shift[kOneBatch], served;
    __shared__ uint16_t list[kRound];
    const int b = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    if (b == 0) served = 0;
    const unsigned bits = one_bits(a, free4);
    int need = 0;
    const int all = scan_rows(a.batch, scratch,
                              [&](int b, int& old) {
                                  need = pages_needed(a, b);
                                  old = need > 0 ? pages_of(__ldcg(a.seq_tokens + b)) : 0;
                                  return max(0, need);
                              },
                              [&](int b, int sum, int mine, int old) {
                                  upto[b] = sum;
                                  shift[b] = old - (sum - mine);
                              });
    const int free = block_sum(__popc(bits), scratch);
    int taken = all;
    if (all > free) {                                 // rows whose pages are all there
        if (b < a.batch && upto[b] <= free) atomicMax(&served, upto[b]);
        __syncthreads();
        taken = served;
    }
    int lo = 0;                                       // the first row whose sum passes r, which only grows
    walk_segment({0, a.num_pages}, 0, taken, scratch, list, [&](int at) { return bits >> (at / kRound * 4) & 15u; }, hold_taken(a), [&](int page, int r) {
        if (upto[lo] <= r) {
            int hi = a.batch - 1;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (upto[mid] > r) hi = mid;
                else lo = mid + 1;
            }
        }
        a.page_table_out[static_cast<int64_t>(lo) * a.max_pages + shift[lo] + r] = page;
    });
    if (b < a.batch) {
        int tokens = __ldcg(a.seq_tokens + b);
        if (need < 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        else if (need > 0 && upto[b] > free) report_error(a.st, LOCKS_ERR_NO_PAGES);
        else tokens = __ldcg(a.new_tokens + b);
        a.seq_tokens_out[b] = tokens;
    }
    if (a.n_free && b == 0) *a.n_free = free - taken;
}

// ------------------------------------------------------------------ fork

__device__ __forceinline__ int parent_of(const PoolArgs& a, int b) {
    const int p = __ldcg(a.parents + b);
    return p >= 0 && p < a.batch ? p : -1;
}
__device__ __forceinline__ int tokens_of(const PoolArgs& a, int b) {
    const int n = __ldcg(a.seq_tokens + b);
    return in_table(n, a.max_pages) ? n : 0;
}
// Row b continues a row whose last page another child keeps.
__device__ __forceinline__ bool needs_page(const PoolArgs& a, int b) {
    const int p = parent_of(a, b);
    return p >= 0 && tokens_of(a, p) % kPage != 0 && __ldcg(a.keeper + p) != b;
}

// First launch: free pages, by block of the pool; the rows' children and who needs a page.
__global__ void __launch_bounds__(kThreads) fork_count_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps];
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    if (blockIdx.x > 0) {
        count_block(a, blockIdx.x - 1, free4, true, scratch);
        return;
    }
    for (int b = tid; b < a.batch; b += kThreads) {
        a.children[b] = 0;
        a.keeper[b] = a.batch;
        const int n = __ldcg(a.seq_tokens + b), p = __ldcg(a.parents + b);
        if (!in_table(n, a.max_pages) || p < -1 || p >= a.batch) report_error(a.st, LOCKS_ERR_BAD_INDEX);
    }
    __syncthreads();
    for (int b = tid; b < a.batch; b += kThreads) {
        const int p = parent_of(a, b);
        if (p < 0) continue;
        atomicAdd(a.children + p, 1);
        atomicMin(a.keeper + p, b == p ? -1 : b);
    }
    __syncthreads();
    for (int b = tid; b < a.batch; b += kThreads)
        if (__ldcg(a.keeper + b) < 0) a.keeper[b] = b;
    __syncthreads();
    const int n = scan_rows(a.batch, scratch, [&](int b, int&) { return needs_page(a, b) ? 1 : 0; },
                            [&](int b, int upto, int mine, int) {
                                if (mine) a.fresh[upto - 1] = b;
                                a.scan[b] = upto;
                            });
    if (tid == 0) *a.needed = n;
}

// Second launch: the first blocks place the free pages; of the others each takes a piece of a row: the
// tables' rows, and what their holds change by.
__global__ void __launch_bounds__(kThreads) fork_place_kernel(const __grid_constant__ PoolArgs a, int pieces) {
    __shared__ int scratch[kWarps];
    __shared__ uint16_t list[kRound];
    const int tid = threadIdx.x, blocks = pool_blocks(a.num_pages);
    grid_dependency_wait();
    allow_dependent_launch();
    if (static_cast<int>(blockIdx.x) <= blocks) {     // (a block more, for a pool without pages)
        const int block = blockIdx.x;
        int before, free;
        join_counts(a, block, scratch, before, free);
        const int n = min(__ldcg(a.needed), free);
        if (block < blocks)
            walk_segment(segment_of(a.num_pages, block), before, n, scratch, list, flags_at(a), [](int, unsigned) {}, [&](int page, int r) {
                const int b = __ldcg(a.fresh + r), p = parent_of(a, b), at = tokens_of(a, p) / kPage;
                a.page_table_out[static_cast<int64_t>(b) * a.max_pages + at] = page;
                a.list_src[r] = __ldcg(a.page_table + static_cast<int64_t>(p) * a.max_pages + at);
                a.list_dst[r] = page;
                a.refs_out[page] = 1;                 // nobody's until now: the rows' blocks leave it alone
            });
        for (int b = block * kThreads + tid; b < a.batch; b += (blocks + 1) * kThreads) {
            const int p = parent_of(a, b);
            int tokens = p >= 0 ? tokens_of(a, p) : 0;
            if (needs_page(a, b) && __ldcg(a.scan + b) > free) {
                report_error(a.st, LOCKS_ERR_NO_PAGES);
                tokens = tokens / kPage * kPage;
            }
            a.seq_tokens_out[b] = tokens;
        }
        if (block == 0 && tid == 0) *a.n_list = n;
        return;
    }
    const int x = blockIdx.x - blocks - 1, b = x / pieces, j0 = (x % pieces) * kRound + tid;
    const int p = parent_of(a, b);
    const int64_t row = static_cast<int64_t>(b) * a.max_pages;
    if (p >= 0) {                                     // row b of the new table
        const int n = tokens_of(a, p), full = n / kPage;
        const int end = full + (n % kPage != 0 && __ldcg(a.keeper + p) == b ? 1 : 0);
        const int32_t* from = a.page_table + static_cast<int64_t>(p) * a.max_pages;
        int page[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kThreads;
            if (j < end) page[i] = __ldcg(from + j);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kThreads;
            if (j >= end) continue;
            a.page_table_out[row + j] = page[i];
            if (page[i] < 0 || page[i] >= a.num_pages) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        }
    }
    const int n = tokens_of(a, b), children = __ldcg(a.children + b);
    if (children == 1) return;                        // every page has as many holders as before
    const int end = children == 0 ? pages_of(n) : n / kPage;      // a last page is kept by one child
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kThreads;
        if (j >= end) continue;
        const int page = __ldcg(a.page_table + row + j);
        if (page >= 0 && page < a.num_pages) atomicAdd(a.refs_out + page, children - 1);
        else report_error(a.st, LOCKS_ERR_BAD_INDEX);
    }
}

__global__ void __launch_bounds__(kThreads, 1) fork_one_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps], tokens[kOneBatch], parent[kOneBatch], children[kOneBatch], keeper[kOneBatch], fresh[kOneBatch];
    __shared__ uint16_t list[kRound];
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    int p = -1;
    if (tid < a.batch) {
        const int n = __ldcg(a.seq_tokens + tid);
        p = __ldcg(a.parents + tid);
        if (!in_table(n, a.max_pages) || p < -1 || p >= a.batch) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        if (p < 0 || p >= a.batch) p = -1;
        tokens[tid] = in_table(n, a.max_pages) ? n : 0;
        parent[tid] = p;
        children[tid] = 0;
        keeper[tid] = a.batch;
    }
    const unsigned bits = one_bits(a, free4);
    __syncthreads();
    if (p >= 0) {
        atomicAdd(&children[p], 1);
        atomicMin(&keeper[p], tid == p ? -1 : tid);
    }
    __syncthreads();
    if (tid < a.batch && keeper[tid] < 0) keeper[tid] = tid;
    __syncthreads();
    const bool needs = p >= 0 && tokens[p] % kPage != 0 && keeper[p] != tid;
    int upto = 0;
    const int needed = scan_rows(a.batch, scratch, [&](int, int&) { return needs ? 1 : 0; },
                                 [&](int b, int sum, int mine, int) {
                                     upto = sum;
                                     if (mine) fresh[sum - 1] = b;
                                 });
    const int free = block_sum(__popc(bits), scratch), n = min(needed, free);
    walk_segment({0, a.num_pages}, 0, n, scratch, list, [&](int at) { return bits >> (at / kRound * 4) & 15u; }, [](int, unsigned) {}, [&](int page, int r) {
        const int b = fresh[r], from = parent[b], at = tokens[from] / kPage;
        a.page_table_out[static_cast<int64_t>(b) * a.max_pages + at] = page;
        a.list_src[r] = __ldcg(a.page_table + static_cast<int64_t>(from) * a.max_pages + at);
        a.list_dst[r] = page;
        a.refs_out[page] = 1;
    });
    if (tid < a.batch) {
        int m = p >= 0 ? tokens[p] : 0;
        if (needs && upto > free) {
            report_error(a.st, LOCKS_ERR_NO_PAGES);
            m = m / kPage * kPage;
        }
        a.seq_tokens_out[tid] = m;
    }
    if (tid == 0) *a.n_list = n;
    each_piece(a.batch, a.max_pages, [&](int b, int j0) {
        const int from = parent[b], m = tokens[b], c = children[b];
        const int64_t row = static_cast<int64_t>(b) * a.max_pages;
        const int32_t* const old = a.page_table + static_cast<int64_t>(from) * a.max_pages;
        const int copied = from < 0 ? 0 : tokens[from] / kPage + (tokens[from] % kPage != 0 && keeper[from] == b ? 1 : 0);
        const int held = c == 1 ? 0 : c == 0 ? pages_of(m) : m / kPage;
        int x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + 32 * i;
            x[i] = j < copied ? __ldcg(old + j) : 0;
            y[i] = j < held ? __ldcg(a.page_table + row + j) : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + 32 * i;
            if (j < copied) a.page_table_out[row + j] = x[i];
            if (j < held && y[i] >= 0 && y[i] < a.num_pages) atomicAdd(a.refs_out + y[i], c - 1);
            if ((j < copied && (x[i] < 0 || x[i] >= a.num_pages)) || (j < held && (y[i] < 0 || y[i] >= a.num_pages)))
                report_error(a.st, LOCKS_ERR_BAD_INDEX);
        }
    });
}

// ------------------------------------------------------------------ free

constexpr int kRowThreads = 256, kRowPiece = 4 * kRowThreads;
__global__ void __launch_bounds__(kRowThreads) copy_refs_kernel(const __grid_constant__ PoolArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) * 4;
    if (at < a.num_pages) store4(a.refs_out, static_cast<int>(at), a.num_pages, load4(a.refs, static_cast<int>(at), a.num_pages));
}

__global__ void __launch_bounds__(kRowThreads) free_kernel(const __grid_constant__ PoolArgs a, int pieces) {
    grid_dependency_wait();
    allow_dependent_launch();
    for (int64_t x = blockIdx.x; x < static_cast<int64_t>(a.rows) * pieces; x += gridDim.x) {
        const int r = static_cast<int>(x / pieces), j0 = static_cast<int>(x % pieces) * kRowPiece + threadIdx.x;
        int n = __ldcg(a.counts + r);
        if (n < 0 || n > a.stride) {
            if (j0 == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            continue;
        }
        int page[4], old[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = j0 + static_cast<int64_t>(i) * kRowThreads;
            page[i] = j < n ? __ldcg(a.lists + static_cast<int64_t>(r) * a.stride + j) : -1;
            if (j < n && (page[i] < 0 || page[i] >= a.num_pages)) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            if (page[i] >= a.num_pages) page[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) old[i] = page[i] >= 0 ? atomicSub(a.refs_out + page[i], 1) : 1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (old[i] <= 0) {                        // nobody's: put back
                atomicAdd(a.refs_out + page[i], 1);
                report_error(a.st, LOCKS_ERR_BAD_INDEX);
            }
    }
}

// ------------------------------------------------------------------ compact

__global__ void __launch_bounds__(kThreads) compact_count_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps];
    grid_dependency_wait();
    allow_dependent_launch();
    count_block(a, blockIdx.x, used4, false, scratch);
}

// How many pages are used, and how many of those lie below the id of that number: all others move.
// A pool of one block is counted here, which saves it a launch.
__device__ __forceinline__ void find_moves(const PoolArgs& a, int i, int* scratch, int& before, int& used, int& low) {
    const bool one = pool_blocks(a.num_pages) == 1;
    before = 0;
    if (one) used = count_block(a, 0, used4, false, scratch);
    else join_counts(a, i, scratch, before, used);
    low = used;
    if (used >= a.num_pages) return;
    const int64_t per = segment_of(a.num_pages, 0).last;
    const int edge = static_cast<int>(used / per);    // the block that `used` lies in
    int ahead = 0, n = 0;
    if (!one) join_counts(a, edge, scratch, ahead, n);
    n = 0;
    const Segment seg = segment_of(a.num_pages, edge);
    for (int at = seg.first + 4 * threadIdx.x; at < used; at += kRound) {
        const unsigned bits = used4(load4(a.refs, at, seg.last));
        n += __popc(bits & (at + 4 <= used ? 15u : (1u << (used - at)) - 1u));
    }
    low = ahead + block_sum(n, scratch);
}

// Second launch: the k-th hole below `used` and the k-th used page from there on. A page that moves
// has -1 - k for its new id until the third launch.
__global__ void __launch_bounds__(kThreads) compact_place_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int scratch[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependent_launch();
    int rank, used, low;
    find_moves(a, blockIdx.x, scratch, rank, used, low);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_list = used - low;
    const Segment seg = segment_of(a.num_pages, blockIdx.x);
#pragma unroll 1
    for (int at0 = seg.first; at0 < seg.last; at0 += kRound) {
        const int at = at0 + 4 * threadIdx.x;
        const int4 r = load4(a.refs, at, seg.last);
        const unsigned bits = used4(r);
        const int upto = warp_upto(__popc(bits));
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        const int sums = scratch[lane];
        int u = rank + upto - __popc(bits) + warp_sum(lane < warp ? sums : 0);     // used pages before at + k
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = at + k;
            const bool on = bits >> k & 1u;
            if (page < seg.last) {
                if (on && page >= used) a.list_src[u - low] = page;
                if (!on && page < used) a.list_dst[page - u] = page;
                a.new_page[page] = on && page >= used ? -1 - (u - low) : page;
                if (page >= used && (k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w) < 0) a.refs_out[page] = 0;
            }
            u += on;
        }
        rank += warp_sum(sums);
        __syncthreads();
    }
}

// Third launch: a block takes a piece of a row of the tables, and all of them the moves. (An entry
// of new_page that another block is just setting is as good before as after.)
__global__ void __launch_bounds__(kThreads) renumber_kernel(const __grid_constant__ PoolArgs a, int pieces) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int moves = __ldcg(a.n_list);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < moves;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int from = __ldcg(a.list_src + i), to = __ldcg(a.list_dst + i);
        a.new_page[from] = to;
        a.refs_out[to] = __ldcg(a.refs + from);
        a.refs_out[from] = 0;
    }
    const int b = blockIdx.x / pieces, j0 = (blockIdx.x % pieces) * kRound + threadIdx.x;
    if (b >= a.batch) return;
    const int n = __ldcg(a.seq_tokens + b);
    if (!in_table(n, a.max_pages)) {
        if (j0 == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        return;
    }
    const int end = pages_of(n);
    const int64_t row = static_cast<int64_t>(b) * a.max_pages;
    int x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kThreads;
        x[i] = j < end ? __ldcg(a.page_table + row + j) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kThreads;
        if (j >= end) continue;
        if (x[i] >= 0 && x[i] < a.num_pages) {
            x[i] = __ldcg(a.new_page + x[i]);
            if (x[i] < 0) x[i] = __ldcg(a.list_dst + (-1 - x[i]));
        } else {
            report_error(a.st, LOCKS_ERR_BAD_INDEX);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kThreads;
        if (j < end) a.page_table_out[row + j] = x[i];
    }
}

__global__ void __launch_bounds__(kThreads, 1) compact_one_kernel(const __grid_constant__ PoolArgs a) {
    constexpr int kRounds = kMovePages / kRound;
    constexpr unsigned kMoves = 0x8000u;              // an id that is still the number of a move
    __shared__ int scratch[kWarps];
    __shared__ uint16_t ids[kMovePages], to[kMovePages / 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    allow_dependent_launch();
    int4 r[kRounds];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) r[k] = load4(a.refs, k * kRound + 4 * tid, a.num_pages);
#pragma unroll
    for (int k = 0; k < kRounds; ++k) mine += __popc(used4(r[k]));
    const int used = block_sum(mine, scratch);
    mine = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += k * kRound + 4 * tid + i < used ? used4(r[k]) >> i & 1u : 0u;
    const int low = block_sum(mine, scratch);         // of them, those that stay
    int rank = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const unsigned bits = used4(r[k]);
        const int upto = warp_upto(__popc(bits));
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        const int sums = scratch[lane];
        int u = rank + upto - __popc(bits) + warp_sum(lane < warp ? sums : 0);     // used pages before this one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int page = k * kRound + 4 * tid + i;
            const bool on = bits >> i & 1u;
            if (page < a.num_pages) {
                ids[page] = static_cast<uint16_t>(on && page >= used ? kMoves | (u - low) : page);
                if (on && page >= used) a.list_src[u - low] = page;
                if (!on && page < used) to[page - u] = static_cast<uint16_t>(page), a.list_dst[page - u] = page;
            }
            u += on;
        }
        rank += warp_sum(sums);
        __syncthreads();
    }
    if (tid == 0) *a.n_list = used - low;
    const auto new_id = [&](int page) -> int {
        const unsigned x = ids[page];
        return x & kMoves ? to[x & (kMoves - 1)] : x;
    };
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int count[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {                 // a page's count is written by whom it belongs to now
            const int page = k * kRound + 4 * tid + i;
            if (page >= a.num_pages) continue;
            const int id = new_id(page);
            a.new_page[page] = id;
            if (count[i] > 0) a.refs_out[id] = count[i];
            if (page >= used) a.refs_out[page] = 0;
        }
    }
    each_piece(a.batch, a.max_pages, [&](int b, int j0) {
        const int n = __ldcg(a.seq_tokens + b);
        if (!in_table(n, a.max_pages)) {
            if (j0 == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            return;
        }
        const int end = pages_of(n);
        const int64_t row = static_cast<int64_t>(b) * a.max_pages;
        int x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = j0 + 32 * i < end ? __ldcg(a.page_table + row + j0 + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + 32 * i;
            if (j >= end) continue;
            if (x[i] >= 0 && x[i] < a.num_pages) x[i] = new_id(x[i]);
            else report_error(a.st, LOCKS_ERR_BAD_INDEX);
            a.page_table_out[row + j] = x[i];
        }
    });
}

// ------------------------------------------------------------------ copy

// A block takes a piece of up to kCopyBytes of a page of one array: eight 16-byte loads a
// thread in flight. HBM bounds it.
constexpr int kCopyThreads = 256, kCopyLoads = 8;
constexpr int kCopyBytes = kCopyThreads * kCopyLoads * 16;

template <typename T>
__device__ __forceinline__ void copy_piece(uint8_t* to, const uint8_t* from, int bytes) {
    constexpr int kSize = sizeof(T);
    for (int at = threadIdx.x * kSize; at < bytes; at += kCopyThreads * kCopyLoads * kSize) {
        T x[kCopyLoads];
#pragma unroll
        for (int i = 0; i < kCopyLoads; ++i)
            if (at + i * kCopyThreads * kSize < bytes) x[i] = __ldcs(reinterpret_cast<const T*>(from + at + i * kCopyThreads * kSize));
#pragma unroll
        for (int i = 0; i < kCopyLoads; ++i)
            if (at + i * kCopyThreads * kSize < bytes) __stcs(reinterpret_cast<T*>(to + at + i * kCopyThreads * kSize), x[i]);
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    int n = a.max_pairs;
    if (a.n_pairs) {
        n = __ldcg(a.n_pairs);
        if (n < 0 || n > a.max_pairs) {
            if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            n = 0;
        }
    }
    // arrays one after the other, of each all pairs, of a pair the pieces: a block's next piece
    // is gridDim.x further on
    int64_t x = blockIdx.x;
    for (int i = 0; i < a.num_planes; ++i) {
        const int64_t bytes = a.page_bytes[i];
        const int64_t pieces = (bytes + kCopyBytes - 1) / kCopyBytes;
        for (; x < n * pieces; x += gridDim.x) {
            const int pair = static_cast<int>(x / pieces);
            const int64_t at = (x % pieces) * kCopyBytes;
            const int from = __ldcg(a.src + pair), to = __ldcg(a.dst + pair);
            if (from < 0 || to < 0) continue;
            if (from >= a.num_pages || to >= a.num_pages) {
                if (threadIdx.x == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
                continue;
            }
            uint8_t* const d = a.base[i] + to * bytes + at;
            const uint8_t* const s = a.base[i] + from * bytes + at;
            const int here = static_cast<int>(min(bytes - at, static_cast<int64_t>(kCopyBytes)));
            if (((bytes | reinterpret_cast<uintptr_t>(a.base[i])) & 15) == 0) copy_piece<uint4>(d, s, here);
            else copy_piece<uint2>(d, s, here);
        }
        x -= n * pieces;
    }
}

int pieces_of(int max_pages, int piece) { return std::max(1, (max_pages + piece - 1) / piece); }

}  // namespace

PoolLayout pool_layout(int batch, int pages) {
    const size_t row = (static_cast<size_t>(batch) * 4 + 255) / 256 * 256;
    PoolLayout w;
    w.needed = 256;
    w.block_counts = w.needed + 256;
    w.scan = w.block_counts + kMaxPoolBlocks * sizeof(int32_t);
    w.shift = w.scan + row;
    w.keeper = w.shift + row;
    w.fresh = w.keeper + row;
    w.flags = w.fresh + row;
    w.bytes = w.flags + (static_cast<size_t>(pages) / 4 + 256) / 256 * 256;
    return w;
}

// Whether one block does the call: a row to a thread, pieces of rows for two turns of its warps.
static bool in_one(const PoolArgs& a, int pages, int64_t rows, int entries) {
    return a.num_pages <= pages && a.batch <= kOneBatch && rows * warp_pieces(entries) <= kOnePieces;
}

cudaError_t launch_take(const PoolArgs& a, cudaStream_t stream) {
    if (in_one(a, kTakePages, 0, 0)) return launch_dependent(take_one_kernel, 1, kThreads, 0, stream, 1, a);
    const int blocks = pool_blocks(a.num_pages);
    const cudaError_t e = launch_dependent(take_count_kernel, blocks + 1, kThreads, 0, stream, 1, a);
    return e != cudaSuccess ? e : launch_dependent(take_place_kernel, blocks + 1, kThreads, 0, stream, 1, a);
}

cudaError_t launch_fork(const PoolArgs& a, cudaStream_t stream) {
    if (in_one(a, kForkPages, a.batch, a.max_pages)) return launch_dependent(fork_one_kernel, 1, kThreads, 0, stream, 1, a);
    const int blocks = pool_blocks(a.num_pages), pieces = pieces_of(a.max_pages, kRound);
    const cudaError_t e = launch_dependent(fork_count_kernel, blocks + 1, kThreads, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.max_pages > 0 ? static_cast<int64_t>(a.batch) * pieces : 0;
    return launch_dependent(fork_place_kernel, blocks + 1 + rows, kThreads, 0, stream, 1, a, pieces);
}

cudaError_t launch_compact(const PoolArgs& a, cudaStream_t stream) {
    if (in_one(a, kMovePages, a.batch, a.max_pages)) return launch_dependent(compact_one_kernel, 1, kThreads, 0, stream, 1, a);
    const int blocks = std::max(1, pool_blocks(a.num_pages)), pieces = pieces_of(a.max_pages, kRound);
    cudaError_t e = blocks > 1 ? launch_dependent(compact_count_kernel, blocks, kThreads, 0, stream, 1, a) : cudaSuccess;
    if (e != cudaSuccess) return e;
    e = launch_dependent(compact_place_kernel, blocks, kThreads, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    const int64_t rows = std::max<int64_t>(1, a.max_pages > 0 ? static_cast<int64_t>(a.batch) * pieces : 0);
    return launch_dependent(renumber_kernel, rows, kThreads, 0, stream, 1, a, pieces);
}

cudaError_t launch_free(const PoolArgs& a, int num_sms, cudaStream_t stream) {
    if (a.refs_out != a.refs && a.num_pages > 0) {
        const int64_t ctas = (static_cast<int64_t>(a.num_pages) + 4 * kRowThreads - 1) / (4 * kRowThreads);
        const cudaError_t e = launch_dependent(copy_refs_kernel, ctas, kRowThreads, 0, stream, 1, a);
        if (e != cudaSuccess) return e;
    }
    if (a.rows == 0) return cudaSuccess;              // (rows without entries have their counts looked at)
    const int pieces = pieces_of(a.stride, kRowPiece);
    const int64_t ctas = std::min<int64_t>(static_cast<int64_t>(a.rows) * pieces, static_cast<int64_t>(num_sms) * 64);
    return launch_dependent(free_kernel, ctas, kRowThreads, 0, stream, 1, a, pieces);
}

// As many CTAs as are resident at once go through small copies and small pieces; large copies of large
// pieces are faster by many CTAs, which SMs get as they come free. Measured, 4 / 64 CTAs an SM (us): 2400
// pages of 4 KB 5.4 / 6.9, 20000 41.5 / 46.8; 2000 of 8 KB 8.2 / 8.8, 20000 60.5 / 62.5; of 16 KB 10.6 / 11.0,
// 107 / 101; of 32 KB 19.0 / 18.3, 214 / 194.
cudaError_t launch_copy_pages(const CopyArgs& a, int num_sms, cudaStream_t stream) {
    int64_t pieces = 0, bytes = 0;
    for (int i = 0; i < a.num_planes; ++i) {
        pieces += (a.page_bytes[i] + kCopyBytes - 1) / kCopyBytes;
        bytes += a.page_bytes[i];
    }
    const int64_t items = pieces * a.max_pairs;
    if (items == 0 && !a.n_pairs) return cudaSuccess; // (a count is looked at all the same)
    const bool large = items >= 2048 && bytes / pieces >= kCopyBytes / 2;
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(items, static_cast<int64_t>(num_sms) * (large ? 64 : 4)));
    return launch_dependent(copy_kernel, ctas, kCopyThreads, 0, stream, 1, a);
}

}  // namespace locks
