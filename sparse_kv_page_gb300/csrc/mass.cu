// mass.cu - the attention mass kept per page, and eviction by it
// (locks_accumulate_mass, locks_evict_pages).
//
// Mass: share_h(j) = exp(s_hj - L_h), L_h = log sum_j exp(s_hj) over the sequence's
// pages, added to each page's mass as the mean over the query heads. L_h needs every
// score before the first share, so the scores are read twice: the first launch takes a
// (max, sum exp) pair per (query head, slice of pages), the second joins a head's pairs
// and reads the scores again, this time from L2 (the score tables of 4 x 1M tokens at
// 32 heads, 33.5 MB, fit in it several times). The scorer's own pairs, where given, are
// joined to one per head by a first launch that does not touch the scores: 4 x 65,536 pages
// at 32 heads 9.9 us for 13.0, one sequence of 8192 4.8 for 4.4 (a row of 304 pairs a head).
#include "cache_internal.h"

namespace locks {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlicePages = 8192;        // pages per pair
constexpr int kPerThread = kSlicePages / kThreads;
constexpr int kMassPages = 128;          // pages per CTA of the second launch, four a lane

__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
    const float M = fmaxf(m, m2);
    if (M == -INFINITY) return;
    l = l * fast_exp2((m - M) * kLog2e) + l2 * fast_exp2((m2 - M) * kLog2e);
    m = M;
}

// A sequence's pages, or -1 where the caller's count is out of range.
__device__ __forceinline__ int pages_of(const int32_t* seq_pages, int b, int max_pages) {
    const int n = seq_pages[b];
    return n < 0 || n > max_pages ? -1 : n;
}

// Only finite scores and -inf count; NaN and +inf read as -inf.
__device__ __forceinline__ float score_of(float s) { return s < INFINITY ? s : -INFINITY; }

__global__ void __launch_bounds__(kThreads) partials_kernel(const MassArgs a, float2* out, bool vec) {
    __shared__ float2 part[kThreads / 32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int slice = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int n = pages_of(a.seq_pages, b, a.max_pages);
    const int64_t row = static_cast<int64_t>(b) * a.hq + h;
    const float* s = a.scores + row * a.max_pages;
    const int first = slice * kSlicePages;
    float x[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; i += 4) {
        if (vec) {                                          // rows are whole 16-byte pieces
            const int j = first + (i * kThreads) + 4 * tid;
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (j < n) v = *reinterpret_cast<const float4*>(s + j);
            x[i] = score_of(v.x);
            x[i + 1] = j + 1 < n ? score_of(v.y) : -INFINITY;
            x[i + 2] = j + 2 < n ? score_of(v.z) : -INFINITY;
            x[i + 3] = j + 3 < n ? score_of(v.w) : -INFINITY;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = first + (i + e) * kThreads + tid;
                x[i + e] = j < n ? score_of(s[j]) : -INFINITY;
            }
        }
    }
    float m = x[0], l = 0.f;
#pragma unroll
    for (int i = 1; i < kPerThread; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m > -INFINITY) {                                    // uniform in the warp
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) l += fast_exp2((x[i] - m) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((tid & 31) == 0) part[tid >> 5] = make_float2(m, l);
    __syncthreads();
    if (tid == 0) {
        m = part[0].x, l = part[0].y;
        for (int w = 1; w < kThreads / 32; ++w) join(m, l, part[w].x, part[w].y);
        out[row * a.row + slice] = make_float2(m, l);
    }
}

// The scorer's pairs of each (sequence, query head), joined to one: a warp each. Only the slots
// of the scorer CTAs whose items reach into the sequence are the scorer's: the others hold
// whatever they held before. A pair whose sum is not above 0, or whose maximum is a NaN, holds
// no scores (the selection's normaliser reads the same slots by the same rule).
__global__ void __launch_bounds__(kThreads)
    reduce_kernel(const float2* in, ScorerSlots slots, int hq, int64_t heads, float2* out) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t h = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (h >= heads) return;
    const int64_t b = h / hq;
    const int first = static_cast<int>(b * slots.chunks / slots.per);
    const int last = min(slots.grid - 1, static_cast<int>(((b + 1) * slots.chunks - 1) / slots.per));
    const float2* row = in + (h * slots.grid + first) * slots.warps;
    const int n = (last - first + 1) * slots.warps;
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
        const float2 v = row[i];
        if (v.y > 0.f && v.x == v.x) join(m, l, v.x, v.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
    if (lane == 0) out[h] = make_float2(m, l);
}

// Grid: (blocks of kMassPages pages, batch). Warp w adds up heads w, w + 8, ... of the CTA's
// pages, and the warps' sums meet in shared memory. The scores were there before the first
// launch began (it starts this one only after waiting for its own predecessor), so the
// first of them are loaded before its pairs are waited for.
__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs a, bool vec) {
    __shared__ float sums[kWarps][kMassPages];
    constexpr int kBatch = 4;                               // heads in flight per warp
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = pages_of(a.seq_pages, b, a.max_pages);
    const int first = blockIdx.x * kMassPages;
    // a lane's four pages: side by side where the rows are whole 16-byte pieces
    const int j0 = vec ? first + 4 * lane : first + lane, step = vec ? 1 : 32;
    const float* s = a.scores + static_cast<int64_t>(b) * a.hq * a.max_pages;
    const int64_t base = static_cast<int64_t>(b) * a.max_pages;
    float4 x[kBatch];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * kWarps;
            x[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (h >= a.hq) continue;
            const float* r = s + static_cast<int64_t>(h) * a.max_pages;
            if (vec) {
                if (j0 < n) x[i] = *reinterpret_cast<const float4*>(r + j0);
            } else {
                if (j0 < n) x[i].x = r[j0];
                if (j0 + 32 < n) x[i].y = r[j0 + 32];
                if (j0 + 64 < n) x[i].z = r[j0 + 64];
                if (j0 + 96 < n) x[i].w = r[j0 + 96];
            }
        }
    };
    load(warp);
    const int mine = first + tid;                           // threads 0..127 finish a page each
    const bool writes = tid < kMassPages && mine < n;
    const float old = writes && a.decay != 0.f ? a.mass[base + mine] * a.decay : 0.f;
    grid_dependency_wait();
    allow_dependent_launch();
    if (n < 0 && tid == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
    if (first >= n) return;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int h0 = warp; h0 < a.hq; h0 += kBatch * kWarps) {
        if (h0 != warp) load(h0);
        // eight lanes join the pairs of one of the four heads
        float m = -INFINITY, l = 0.f;
        const int h = h0 + (lane >> 3) * kWarps;
        if (h < a.hq) {
            const float2* p = a.partials + (static_cast<int64_t>(b) * a.hq + h) * a.row;
            for (int i = lane & 7; i < a.row; i += 8) {
                const float2 v = p[i];
                join(m, l, v.x, v.y);
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
        // no score above -inf, or a normaliser that is no number: the head adds nothing
        const bool ok = m > -INFINITY && m < INFINITY && l > 0.f && l < INFINITY;
        const float inv = ok ? 1.f / (l * a.hq) : 0.f;
        m = ok ? m : 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float mi = __shfl_sync(0xffffffffu, m, 8 * i), w = __shfl_sync(0xffffffffu, inv, 8 * i);
            if (w == 0.f) continue;                         // also heads past the last; uniform
            acc[0] += fast_exp2((score_of(x[i].x) - mi) * kLog2e) * w;
            acc[1] += fast_exp2((score_of(x[i].y) - mi) * kLog2e) * w;
            acc[2] += fast_exp2((score_of(x[i].z) - mi) * kLog2e) * w;
            acc[3] += fast_exp2((score_of(x[i].w) - mi) * kLog2e) * w;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][j0 - first + e * step] = acc[e];
    __syncthreads();
    if (writes) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += sums[w][tid];
        a.mass_out[base + mine] = old + sum;
    }
}

bool rows_aligned(const MassArgs& a) {
    return a.max_pages % 4 == 0 && reinterpret_cast<uintptr_t>(a.scores) % 16 == 0;
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------ eviction

// One cluster of CL CTAs per sequence. A CTA keeps its share of the sequence's masses and
// table entries in shared memory: the inputs are read once, and all of them before the
// first write, so the outputs may be the inputs. The e-th smallest key (order-preserving
// image of the mass) is found by a radix select; the CTAs' histograms are joined through
// distributed shared memory. What it costs is those exchanges (about 2.4 us each over 16
// CTAs), so it stops as soon as it can: when all keys of the chosen bin are equal (pages
// that never drew any mass), or when they are few enough for every CTA to gather and rank
// them. One CTA alone takes 11 bits a pass; clusters take 8, as the bytes of 16 histograms
// of 2048 bins cost more than the passes they save (4 x 65,536 pages: 26.6 us).
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kMaxBins = 2048;               // two 16-bit counts to a word
template <int CL>
constexpr int kDigit = CL == 1 ? 11 : 8;     // bits a pass
constexpr int kGather = 256;
constexpr int kMaxShare = 24576;             // pages of a CTA
static_assert(16 * kMaxShare == kMaxEvictPages, "the longest table");

struct EvictShared {
    uint32_t hist[2][kMaxBins / 2];
    uint32_t kmin[2], kmax[2];           // of the keys counted
    uint32_t list[kGather], all[kGather];
    int listed;
    uint32_t wsum[kEvictWarps];
    int digit, below, inside;
    uint32_t key;
    int want;
    uint32_t cnt;                        // this CTA's pages below (high half) and at (low) the threshold
};

__device__ __forceinline__ uint32_t mass_key(float m) { return orderable_key(m + 0.f); }   // -0 counts as 0

template <int CL>
__device__ __forceinline__ void join_sync() {
    if (CL == 1) __syncthreads();
    else cluster_sync_all();
}
template <int CL>
__device__ __forceinline__ uint32_t of_cta(const uint32_t* p, int r) {
    return CL == 1 ? *p : ld_dsmem_u32(dsmem_addr(p, r));
}

// Exclusive scan over the CTA in thread order, and the total. Two barriers.
__device__ __forceinline__ uint32_t scan_cta(uint32_t v, uint32_t& total, EvictShared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sh.wsum[warp] = upto;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kEvictWarps; ++w) {
        const uint32_t c = sh.wsum[w];
        before += w < warp ? c : 0;
        sum += c;
    }
    __syncthreads();
    total = sum;
    return before + upto - v;
}

template <int CL>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a, int share) {
    constexpr int kBits = kDigit<CL>, kWords = (1 << kBits) / 2;
    constexpr int kPer = (kWords + kEvictThreads - 1) / kEvictThreads;   // words of the histogram a thread
    __shared__ EvictShared sh;
    extern __shared__ float mass_s[];
    int32_t* table_s = reinterpret_cast<int32_t*>(mass_s + share);
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x / CL, tid = threadIdx.x;
    const int rank = CL == 1 ? 0 : static_cast<int>(cluster_ctarank());
    const int n = pages_of(a.seq_pages, b, a.max_pages);
    if (n < 0) {                                            // uniform in the cluster
        if (rank == 0 && tid == 0) {
            report_error(a.st, LOCKS_ERR_BAD_INDEX);
            a.n_evicted[b] = 0;
        }
        return;
    }
    const int e = max(0, n - a.keep);
    const int end = n + min(a.extra, a.max_pages - n);      // entries that stay or leave
    const int64_t base = static_cast<int64_t>(b) * a.max_pages;
    const int first = rank * share, mine = max(0, min(share, end - first));
#pragma unroll 4
    for (int i = tid; i < mine; i += kEvictThreads) {
        mass_s[i] = a.mass[base + first + i];
        table_s[i] = a.page_table[base + first + i];
    }
    // candidates: logical pages [lo, hi) of this CTA's share
    const int lo = max(0, a.sink - first), hi = min(mine, n - a.recent - first);
    uint32_t key = 0;                                       // the threshold (its known high bits at first)
    int want = e;                                           // its rank among the candidates left
    if (e > 0) {
        if (tid == 0) sh.listed = 0;
#pragma unroll 1
        for (int pass = 0, shift = 32; shift > 0; ++pass) {
            const int upto = shift, bits = min(kBits, shift);
            shift -= bits;
            uint32_t* hist = sh.hist[pass & 1];
            for (int i = tid; i < kWords; i += kEvictThreads) hist[i] = 0;
            if (tid == 0) sh.kmin[pass & 1] = 0xffffffffu, sh.kmax[pass & 1] = 0;
            __syncthreads();
            uint32_t kmin = 0xffffffffu, kmax = 0;
            for (int i = lo + tid; i < hi; i += kEvictThreads) {
                const uint32_t k = mass_key(mass_s[i]);
                if (pass == 0 || k >> upto == key) {
                    const uint32_t d = (k >> shift) & ((1u << bits) - 1);
                    atomicAdd(&hist[d >> 1], 1u << (16 * (d & 1)));
                    kmin = min(kmin, k);
                    kmax = max(kmax, k);
                }
            }
            if (pass > 0) {
                kmin = __reduce_min_sync(0xffffffffu, kmin);
                kmax = __reduce_max_sync(0xffffffffu, kmax);
                if ((tid & 31) == 0) atomicMin(&sh.kmin[pass & 1], kmin), atomicMax(&sh.kmax[pass & 1], kmax);
            }
            join_sync<CL>();
            uint32_t c[2 * kPer] = {};                      // this thread's bins
            if (tid * kPer < kWords) {
#pragma unroll
                for (int r = 0; r < CL; ++r)
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const uint32_t u = of_cta<CL>(&hist[tid * kPer + i], r);
                        c[2 * i] += u & 0xffffu;
                        c[2 * i + 1] += u >> 16;
                    }
            }
            kmin = 0xffffffffu, kmax = 0;
            if (pass > 0) {                                 // every warp learns the range of the keys
                const int r = tid & 31;
                if (r < CL) kmin = of_cta<CL>(&sh.kmin[pass & 1], r), kmax = of_cta<CL>(&sh.kmax[pass & 1], r);
                kmin = __reduce_min_sync(0xffffffffu, kmin);
                kmax = __reduce_max_sync(0xffffffffu, kmax);
            }
            if (pass > 0 && kmin == kmax) {                 // uniform in the cluster
                key = kmin;
                break;
            }
            uint32_t sum = 0, total;
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i) sum += c[i];
            uint32_t before = scan_cta(sum, total, sh);
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i) {
                if (before < static_cast<uint32_t>(want) && static_cast<uint32_t>(want) <= before + c[i]) {
                    sh.digit = 2 * kPer * tid + i;
                    sh.below = static_cast<int>(before);
                    sh.inside = static_cast<int>(c[i]);
                }
                before += c[i];
            }
            __syncthreads();
            key = (key << bits) | static_cast<uint32_t>(sh.digit);
            want -= sh.below;
            const int inside = sh.inside;
            if (shift > 0 && inside <= kGather) {            // uniform in the cluster: rank them here
                for (int i = lo + tid; i < hi; i += kEvictThreads) {
                    const uint32_t k = mass_key(mass_s[i]);
                    if (k >> shift == key) sh.list[atomicAdd(&sh.listed, 1)] = k;
                }
                join_sync<CL>();
                if (tid < kGather) {                        // the tid-th key of all lists
                    int from = -1, at = tid;
                    for (int r = 0; r < CL; ++r) {
                        const int cr = static_cast<int>(of_cta<CL>(reinterpret_cast<const uint32_t*>(&sh.listed), r));
                        if (from < 0) {
                            if (at < cr) from = r;
                            else at -= cr;
                        }
                    }
                    sh.all[tid] = from < 0 ? 0xffffffffu : of_cta<CL>(&sh.list[at], from);
                }
                __syncthreads();
                if (tid < inside) {
                    const uint32_t k = sh.all[tid];
                    int less = 0, same = 0;
                    for (int i = 0; i < inside; ++i) {
                        less += sh.all[i] < k;
                        same += sh.all[i] == k;
                    }
                    if (less < want && want <= less + same) sh.key = k, sh.want = want - less;   // equal writers agree
                }
                __syncthreads();
                key = sh.key;
                want = sh.want;
                break;
            }
        }
    }
    // `want` of the pages at the threshold leave, lowest first. A thread takes pages side by
    // side (an odd number of them: no bank conflicts), so that one scan places them all.
    const int per = (share + kEvictThreads - 1) / kEvictThreads | 1;
    const int i0 = min(tid * per, mine), i1 = min(i0 + per, mine);
    uint32_t mark = 0;                                      // below (high half) and at (low half) the threshold
    if (e > 0) {
        for (int i = max(i0, lo); i < min(i1, hi); ++i) {
            const uint32_t k = mass_key(mass_s[i]);
            mark += k < key ? 0x10000u : k == key ? 1u : 0u;
        }
    }
    uint32_t total;
    mark = scan_cta(mark, total, sh);
    int less_before = mark >> 16, eq_before = mark & 0xffffu;
    if (CL > 1) {
        if (tid == 0) sh.cnt = total;
        cluster_sync_all();                                 // also: every CTA has read its inputs
        const int r = tid & 31;
        const uint32_t c = r < rank ? ld_dsmem_u32(dsmem_addr(&sh.cnt, r)) : 0u;
        less_before += __reduce_add_sync(0xffffffffu, c >> 16);
        eq_before += __reduce_add_sync(0xffffffffu, c & 0xffffu);
        // shared memory stays until every CTA has read it
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    for (int i = i0; i < i1; ++i) {
        const float m = mass_s[i];
        const int32_t t = table_s[i];
        const bool cand = e > 0 && i >= lo && i < hi;
        const uint32_t k = mass_key(m);
        const bool less = cand && k < key, eq = cand && k == key;
        const int before = less_before + min(eq_before, want);
        if (less || (eq && eq_before < want)) {
            if (before < a.evict_cap) a.evicted[static_cast<int64_t>(b) * a.evict_cap + before] = t;
        } else {
            a.page_table_out[base + first + i - before] = t;
            a.mass_out[base + first + i - before] = m;
        }
        less_before += less;
        eq_before += eq;
    }
    if (rank == 0 && tid == 0) {
        a.n_evicted[b] = e;
        a.seq_pages_out[b] = n - e;
    }
    if (CL > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int CL>
cudaError_t launch_evict_t(const EvictArgs& a, cudaStream_t stream) {
    const int share = (a.max_pages + CL - 1) / CL;
    const size_t smem = static_cast<size_t>(share) * 8;
    cudaError_t e = ensure_kernel_attrs<evict_kernel<CL>>(static_cast<int>(smem), CL > 8);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * CL, 1, 1);
    cfg.blockDim = dim3(kEvictThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, evict_kernel<CL>, a, share);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// No sum before the division: max_pages may be any int32.
int mass_partials_row(int max_pages) { return max_pages / kSlicePages + (max_pages % kSlicePages != 0); }

cudaError_t launch_mass_partials(const MassArgs& a, float2* partials, cudaStream_t stream) {
    return launch_pdl(partials_kernel, dim3(a.row, a.hq, a.batch), kThreads, 0, stream, a, partials, rows_aligned(a));
}

cudaError_t launch_mass(const MassArgs& a, cudaStream_t stream) {
    const int blocks = a.max_pages / kMassPages + (a.max_pages % kMassPages != 0);
    return launch_pdl(mass_kernel, dim3(blocks, a.batch, 1), kThreads, 0, stream, a, rows_aligned(a));
}

cudaError_t launch_mass_reduce(const float2* in, const ScorerSlots& slots, const MassArgs& a, float2* out,
                               cudaStream_t stream) {
    const int64_t heads = static_cast<int64_t>(a.batch) * a.hq;
    return launch_pdl(reduce_kernel, dim3(static_cast<unsigned>((heads + kWarps - 1) / kWarps)), kThreads, 0, stream, in,
                      slots, a.hq, heads, out);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    // More CTAs a sequence shorten the passes over its pages and lengthen every exchange, and
    // clusters that together pass a CTA per SM run one another's launches down. us a call with
    // 1 / 2 / 4 / 8 CTAs a sequence: one sequence of 1100 pages 4.3 / 5.1 / 4.6 / 5.0, of 2000
    // 5.9 / 5.3 / 4.7 / 5.0, of 4000 9.6 / 7.2 / 5.6 / 5.3; 19 of 4000 9.7 / 7.3 / 5.7 / 7.5;
    // 64 of 2000 6.2 / 5.5 / 6.9 / 11.5, of 8000 16.8 / 11.8 / 10.8 / 13.5; 256 of 4000 15.3 /
    // 16.1 / 19.4 / 37.5. With 8 / 16: one of 16,384 pages 7.9 / 8.3, of 65,536 18.3 / 14.0;
    // eight of 65,536 18.9 / 21.2. Sixteen also hold the longest tables (24,576 pages a CTA at
    // most).
    if (a.max_pages <= 1536) return launch_evict_t<1>(a, stream);
    if (a.max_pages <= 16384) {
        if (a.batch <= 8 && a.max_pages > 2048) return launch_evict_t<8>(a, stream);
        if (a.batch <= 24 || (a.batch <= 96 && a.max_pages > 4096)) return launch_evict_t<4>(a, stream);
        return a.batch <= 96 ? launch_evict_t<2>(a, stream) : launch_evict_t<1>(a, stream);
    }
    if (a.batch > 4 && a.max_pages <= 8 * kMaxShare) return launch_evict_t<8>(a, stream);
    return launch_evict_t<16>(a, stream);
}

}  // namespace locks
