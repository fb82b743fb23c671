// pool.cu - the page pool's calls (locks_pool.h): copying, forking, taking, freeing and
// compacting pages.
//
// Which pages are free follows from the reference counts alone, so the calls that look for
// free pages (fork, take) or rank the used ones (compact) scan them: one cluster of CTAs, a
// contiguous segment of the pool to a warp, counts joined through distributed shared memory.
// 4 bytes a page are little (1M pages: 4 MB, which L2 holds), and what bounds these calls is
// latency: one round of loads to count, a barrier, one to place. Tables are rewritten by all
// SMs in a second launch, which starts while the first runs.
#include <algorithm>

#include "pool_internal.h"

namespace locks {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kScanRows = 4096;                       // rows whose prefix sums lie in shared memory

__device__ __forceinline__ bool in_table(int tokens, int max_pages) {
    return tokens >= 0 && tokens <= static_cast<int64_t>(max_pages) * kPage;
}
__device__ __forceinline__ int pages_of(int tokens) { return tokens / kPage + (tokens % kPage != 0); }
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// This warp's segment of the pool: pages first .. last, a multiple of 128 but for the pool's end.
struct Segment {
    int first, last;
};
__device__ __forceinline__ Segment segment_of(int pages) {
    const int64_t warps = static_cast<int64_t>(cluster_size()) * kWarps;
    const int64_t per = (pages + warps * 128 - 1) / (warps * 128) * 128;
    const int64_t first = (static_cast<int64_t>(cluster_ctarank()) * kWarps + (threadIdx.x >> 5)) * per;
    return {static_cast<int>(min(first, static_cast<int64_t>(pages))),
            static_cast<int>(min(first + per, static_cast<int64_t>(pages)))};
}
// Counts of pages at .. at + 3 (a lane's), those past `last` as if held by nobody and not free.
__device__ __forceinline__ int4 load4(const int32_t* refs, int at, int last) {
    if (at + 4 <= last) return __ldcg(reinterpret_cast<const int4*>(refs + at));
    int4 r;
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
// Bit k: page at + k is free / used (neither past the end, whose counts are INT32_MIN; a count
// that a caller let fall to that value is as good as any below 0 and reads as not free).
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

// Counts pages of a kind (free4 or used4) in this warp's segment, and copies the counts to
// refs_out on the way where that is another array.
template <typename Kind>
__device__ __forceinline__ int count_segment(const PoolArgs& a, const Segment& seg, Kind kind) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    const bool copy = a.refs_out != a.refs;
#pragma unroll 4
    for (int at = seg.first + 4 * lane; at < seg.last; at += 128) {
        const int4 r = load4(a.refs, at, seg.last);
        n += __popc(kind(r));
        if (copy) store4(a.refs_out, at, seg.last, r);
    }
    return warp_sum(n);
}

// Calls f(page, rank) for the pages of a kind in this warp's segment, ranks counted from `rank`;
// stops behind rank `most`.
template <typename Kind, typename F>
__device__ __forceinline__ void walk_segment(const PoolArgs& a, const Segment& seg, Kind kind, int rank, int most, F f) {
    const int lane = threadIdx.x & 31;
#pragma unroll 2
    for (int at0 = seg.first; at0 < seg.last; at0 += 128) {
        if (rank >= most) return;
        const int at = at0 + 4 * lane;
        const unsigned bits = at < seg.last ? kind(load4(a.refs, at, seg.last)) : 0u;
        const int upto = warp_upto(__popc(bits));
        int r = rank + upto - __popc(bits);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (bits >> k & 1u) {
                if (r < most) f(at + k, r);
                ++r;
            }
        rank += __shfl_sync(kAll, upto, 31);
    }
}

// What the cluster's CTAs share: the warps' counts and the CTA's.
struct Counts {
    int warp[kWarps];
    int cta;
    int extra;                                        // compact: used pages below the end of the used ones
};
// From the warps' counts: how many of the kind are before this warp's segment, and in all.
__device__ __forceinline__ void join_counts(Counts& c, int mine, int& before, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) c.warp[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const int n = warp_sum(c.warp[lane]);
        if (lane == 0) c.cta = n;
    }
    cluster_sync_all();
    const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const int x = lane < ctas ? static_cast<int>(ld_dsmem_u32(dsmem_addr(&c.cta, lane))) : 0;
    total = warp_sum(x);
    before = warp_sum(lane < rank ? x : 0) + warp_sum(lane < warp ? c.warp[lane] : 0);
}

// Sums over the batch, by one CTA: calls put(b, sum of count(0..b)) for every row in turn of
// its thread, and returns the sum of all.
template <typename Count, typename Put>
__device__ __forceinline__ int scan_rows(int batch, int* scratch, Count count, Put put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int mine = b < batch ? count(b) : 0;
        int upto = warp_upto(mine);
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        const int sums = scratch[lane];
        upto += base + warp_sum(lane < warp ? sums : 0);
        if (b < batch) put(b, upto, mine);
        base += warp_sum(sums);
        __syncthreads();
    }
    return base;
}

// ------------------------------------------------------------------ take

// Pages that row b needs; -1: its counts are wrong.
__device__ __forceinline__ int pages_needed(const PoolArgs& a, int b) {
    const int old = __ldcg(a.seq_tokens + b), now = __ldcg(a.new_tokens + b);
    if (!in_table(old, a.max_pages) || !in_table(now, a.max_pages) || now < old) return -1;
    return pages_of(now) - pages_of(old);
}

__global__ void __launch_bounds__(kThreads) take_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ Counts counts;
    __shared__ int scratch[kWarps], near_scan[kScanRows], served;
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_size());
    grid_dependency_wait();
    allow_dependent_launch();
    const Segment seg = segment_of(a.num_pages);
    const int free_here = count_segment(a, seg, free4);
    // pages needed by rows 0..b: in every CTA, or where the rows are many by one for all
    const bool near = a.batch <= kScanRows;
    int* const scan = near ? near_scan : a.scan;
    if (tid == 0) served = 0;
    if (near || rank == 0)
        scan_rows(a.batch, scratch, [&](int b) { return max(0, pages_needed(a, b)); },
                  [&](int b, int upto, int) { scan[b] = upto; });
    int before, free;
    join_counts(counts, free_here, before, free);
    // rows whose pages are all there: those before the first that lacks some
    int mine = 0;
    for (int b = tid; b < a.batch; b += kThreads)
        if (scan[b] <= free) mine = max(mine, scan[b]);
    if (mine > 0) atomicMax(&served, mine);
    __syncthreads();
    const int taken = served;
    walk_segment(a, seg, free4, before, taken, [&](int page, int r) {
        int lo = 0, hi = a.batch - 1;                 // the first row whose sum passes r
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (scan[mid] > r) hi = mid;
            else lo = mid + 1;
        }
        const int j = pages_of(__ldcg(a.seq_tokens + lo)) + r - (lo > 0 ? scan[lo - 1] : 0);
        a.page_table_out[static_cast<int64_t>(lo) * a.max_pages + j] = page;
        a.refs_out[page] = 1;
    });
    // seq_tokens is read above by every CTA (and may be seq_tokens_out)
    cluster_sync_all();
    for (int b = rank * kThreads + tid; b < a.batch; b += ctas * kThreads) {
        const int need = pages_needed(a, b);
        int tokens = __ldcg(a.seq_tokens + b);
        if (need < 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        else if (need > 0 && scan[b] > free) report_error(a.st, LOCKS_ERR_NO_PAGES);
        else tokens = __ldcg(a.new_tokens + b);
        a.seq_tokens_out[b] = tokens;
    }
    if (a.n_free && rank == 0 && tid == 0) *a.n_free = free - taken;
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

__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ Counts counts;
    __shared__ int scratch[kWarps], needed;
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_size());
    grid_dependency_wait();
    allow_dependent_launch();
    const Segment seg = segment_of(a.num_pages);
    const int free_here = count_segment(a, seg, free4);
    if (rank == 0) {
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
        const int n = scan_rows(a.batch, scratch, [&](int b) { return needs_page(a, b) ? 1 : 0; },
                                [&](int b, int upto, int mine) {
                                    if (mine) a.fresh[upto - 1] = b;
                                    a.scan[b] = upto;
                                });
        if (tid == 0) needed = n;
    }
    int before, free;
    join_counts(counts, free_here, before, free);
    const int want = static_cast<int>(ld_dsmem_u32(dsmem_addr(&needed, 0)));
    const int n = min(want, free);
    walk_segment(a, seg, free4, before, n, [&](int page, int r) {
        const int b = __ldcg(a.fresh + r), p = parent_of(a, b), at = tokens_of(a, p) / kPage;
        a.page_table_out[static_cast<int64_t>(b) * a.max_pages + at] = page;
        a.list_src[r] = __ldcg(a.page_table + static_cast<int64_t>(p) * a.max_pages + at);
        a.list_dst[r] = page;
        a.refs_out[page] = 1;
    });
    for (int b = rank * kThreads + tid; b < a.batch; b += ctas * kThreads) {
        const int p = parent_of(a, b);
        int tokens = p >= 0 ? tokens_of(a, p) : 0;
        if (needs_page(a, b) && __ldcg(a.scan + b) > free) {
            report_error(a.st, LOCKS_ERR_NO_PAGES);
            tokens = tokens / kPage * kPage;
        }
        a.seq_tokens_out[b] = tokens;
    }
    if (rank == 0 && tid == 0) *a.n_list = n;
    cluster_sync_all();                               // `needed` is read by all
}

// The tables' rows, and what their holds change by. A block takes a piece of a row.
constexpr int kRowThreads = 256, kRowPiece = 4 * kRowThreads;
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const __grid_constant__ PoolArgs a, int pieces) {
    const int b = blockIdx.x / pieces, j0 = (blockIdx.x % pieces) * kRowPiece + threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    const int p = parent_of(a, b);
    const int64_t row = static_cast<int64_t>(b) * a.max_pages;
    if (p >= 0) {                                     // row b of the new table
        const int n = tokens_of(a, p), full = n / kPage;
        const int end = full + (n % kPage != 0 && __ldcg(a.keeper + p) == b ? 1 : 0);
        const int32_t* from = a.page_table + static_cast<int64_t>(p) * a.max_pages;
        int x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kRowThreads;
            if (j < end) x[i] = __ldcg(from + j);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kRowThreads;
            if (j < end) a.page_table_out[row + j] = x[i];
        }
    }
    const int n = tokens_of(a, b), full = n / kPage, children = __ldcg(a.children + b);
    if (children == 1) return;                        // every page has as many holders as before
    const int end = children == 0 ? pages_of(n) : full;   // a last page is kept by one child
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kRowThreads;
        if (j >= end) continue;
        const int page = __ldcg(a.page_table + row + j);
        if (page >= 0 && page < a.num_pages) atomicAdd(a.refs_out + page, children - 1);
        else report_error(a.st, LOCKS_ERR_BAD_INDEX);
    }
}

// ------------------------------------------------------------------ free

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

__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ Counts counts;
    const int tid = threadIdx.x, lane = tid & 31, rank = static_cast<int>(cluster_ctarank());
    const int ctas = static_cast<int>(cluster_size());
    grid_dependency_wait();
    allow_dependent_launch();
    const Segment seg = segment_of(a.num_pages);
    if (tid == 0) counts.extra = 0;
    const int used_here = count_segment(a, seg, used4);
    int before, used;
    join_counts(counts, used_here, before, used);
    // used pages below id `used`: known where that lies
    if (seg.first <= used && used < seg.last) {
        int n = 0;
        for (int at = seg.first + 4 * lane; at < used; at += 128) {
            const unsigned bits = used4(load4(a.refs, at, seg.last));
            n += __popc(bits & (at + 4 <= used ? 15u : (1u << (used - at)) - 1u));
        }
        n = warp_sum(n);
        if (lane == 0) counts.extra = before + n;
    }
    cluster_sync_all();
    int low = lane < ctas ? static_cast<int>(ld_dsmem_u32(dsmem_addr(&counts.extra, lane))) : 0;
    low = used < a.num_pages ? warp_sum(low) : used;  // one CTA's, 0 in the others
    const int moves = used - low;
    // the k-th hole below `used` and the k-th used page from there on
    int rank_used = before;
    for (int at0 = seg.first; at0 < seg.last; at0 += 128) {
        const int at = at0 + 4 * lane;
        const unsigned bits = at < seg.last ? used4(load4(a.refs, at, seg.last)) : 0u;
        const int upto = warp_upto(__popc(bits));
        int u = rank_used + upto - __popc(bits);      // used pages before at + k
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = at + k;
            if (page >= seg.last) break;
            const bool on = bits >> k & 1u;
            if (on && page >= used) a.list_src[u - low] = page;
            if (!on && page < used) a.list_dst[page - u] = page;
            a.new_page[page] = page;
            u += on;
        }
        rank_used += __shfl_sync(kAll, upto, 31);
    }
    cluster_sync_all();
    for (int i = rank * kThreads + tid; i < moves; i += ctas * kThreads) {
        const int from = __ldcg(a.list_src + i), to = __ldcg(a.list_dst + i);
        a.new_page[from] = to;
        a.refs_out[to] = __ldcg(a.refs + from);
        a.refs_out[from] = 0;
    }
    if (rank == 0 && tid == 0) *a.n_list = moves;
}

__global__ void __launch_bounds__(kRowThreads) renumber_kernel(const __grid_constant__ PoolArgs a, int pieces) {
    const int b = blockIdx.x / pieces, j0 = (blockIdx.x % pieces) * kRowPiece + threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
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
        const int j = j0 + i * kRowThreads;
        x[i] = j < end ? __ldcg(a.page_table + row + j) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kRowThreads;
        if (j >= end) continue;
        if (x[i] >= 0 && x[i] < a.num_pages) x[i] = __ldcg(a.new_page + x[i]);
        else report_error(a.st, LOCKS_ERR_BAD_INDEX);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kRowThreads;
        if (j < end) a.page_table_out[row + j] = x[i];
    }
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

// CTAs of the cluster that scans the pool: each takes about 8192 pages, two loads a thread.
int cluster_of(int pages) {
    int n = 1;
    while (n < kMaxCluster && static_cast<int64_t>(n) * 8192 < pages) n *= 2;
    return n;
}
template <auto Kern>
cudaError_t launch_scan(const PoolArgs& a, cudaStream_t stream) {
    const int n = cluster_of(a.num_pages);
    const cudaError_t e = ensure_kernel_attrs<Kern>(0, true);
    return e != cudaSuccess ? e : launch_dependent(Kern, n, kThreads, 0, stream, n, a);
}
int pieces_of(int max_pages) { return (max_pages + kRowPiece - 1) / kRowPiece; }

}  // namespace

PoolLayout pool_layout(int batch) {
    const size_t row = (static_cast<size_t>(batch) * 4 + 255) / 256 * 256;
    PoolLayout w;
    w.scan = 256;
    w.children = w.scan + row;
    w.keeper = w.children + row;
    w.fresh = w.keeper + row;
    w.bytes = w.fresh + row;
    return w;
}

cudaError_t launch_take(const PoolArgs& a, cudaStream_t stream) { return launch_scan<take_kernel>(a, stream); }

cudaError_t launch_fork(const PoolArgs& a, int, cudaStream_t stream) {
    const cudaError_t e = launch_scan<fork_kernel>(a, stream);
    const int pieces = pieces_of(a.max_pages);
    if (e != cudaSuccess || pieces == 0 || a.batch == 0) return e;
    return launch_dependent(fork_rows_kernel, static_cast<int64_t>(a.batch) * pieces, kRowThreads, 0, stream, 1, a, pieces);
}

cudaError_t launch_compact(const PoolArgs& a, int, cudaStream_t stream) {
    const cudaError_t e = launch_scan<compact_kernel>(a, stream);
    const int pieces = pieces_of(a.max_pages);
    if (e != cudaSuccess || pieces == 0 || a.batch == 0) return e;
    return launch_dependent(renumber_kernel, static_cast<int64_t>(a.batch) * pieces, kRowThreads, 0, stream, 1, a, pieces);
}

cudaError_t launch_free(const PoolArgs& a, int num_sms, cudaStream_t stream) {
    if (a.refs_out != a.refs) {
        const int64_t ctas = (static_cast<int64_t>(a.num_pages) + 4 * kRowThreads - 1) / (4 * kRowThreads);
        const cudaError_t e = launch_dependent(copy_refs_kernel, ctas, kRowThreads, 0, stream, 1, a);
        if (e != cudaSuccess) return e;
    }
    if (a.rows == 0 || a.stride == 0) return cudaSuccess;
    const int pieces = pieces_of(a.stride);
    const int64_t ctas = std::min<int64_t>(static_cast<int64_t>(a.rows) * pieces, static_cast<int64_t>(num_sms) * 64);
    return launch_dependent(free_kernel, ctas, kRowThreads, 0, stream, 1, a, pieces);
}

cudaError_t launch_copy_pages(const CopyArgs& a, int num_sms, cudaStream_t stream) {
    int64_t pieces = 0;
    for (int i = 0; i < a.num_planes; ++i) pieces += (a.page_bytes[i] + kCopyBytes - 1) / kCopyBytes;
    const int64_t ctas = std::min<int64_t>(pieces * a.max_pairs, static_cast<int64_t>(num_sms) * 8);
    return launch_dependent(copy_kernel, ctas, kCopyThreads, 0, stream, 1, a);
}

}  // namespace locks
