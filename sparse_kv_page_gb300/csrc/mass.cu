// mass.cu - the attention mass kept per page, and eviction by it
// (locks_accumulate_mass, locks_evict_pages).
//
// Mass: share_h(j) = exp(s_hj - L_h), L_h = log sum_j exp(s_hj) over the sequence's
// pages, added to each page's mass as the mean over the query heads. L_h needs every
// score before the first share, so the scores are read twice: one launch takes a
// (max, sum exp) pair per (query head, slice of pages), the next joins a head's pairs
// and streams the scores again, this time from L2 (the score tables of 4 x 1M tokens at
// 32 heads, 33.5 MB, fit in it several times). With the scorer's own pairs the first
// launch falls away.
#include "cache_internal.h"

namespace locks {
namespace {

constexpr int kThreads = 256;
constexpr int kSlicePages = 2048;        // pages per pair
constexpr int kPerThread = kSlicePages / kThreads;
constexpr int kMassThreads = 128;
constexpr int kMassPages = 4 * kMassThreads;   // pages per CTA of the second pass

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

// Grid: (blocks of kMassPages pages, batch). Dynamic shared memory: a float2 per head,
// its maximum and (1 / Hq) / sum.
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const MassArgs a, bool vec) {
    extern __shared__ float2 norm[];
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int n = pages_of(a.seq_pages, b, a.max_pages);
    if (n < 0) {
        if (tid == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        return;
    }
    const int first = blockIdx.x * kMassPages;
    if (first >= n) return;
    for (int h = tid >> 5; h < a.hq; h += kMassThreads / 32) {
        const float2* p = a.partials + (static_cast<int64_t>(b) * a.hq + h) * a.row;
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < a.row; i += 32) {
            const float2 v = p[i];
            join(m, l, v.x, v.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
        // no score above -inf, or a normaliser that is no number: the head adds nothing
        const bool ok = m > -INFINITY && m < INFINITY && l > 0.f && l < INFINITY;
        if (lane == 0) norm[h] = ok ? make_float2(m, 1.f / (l * a.hq)) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    const float* s = a.scores + static_cast<int64_t>(b) * a.hq * a.max_pages;
    const int64_t base = static_cast<int64_t>(b) * a.max_pages;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
        const int j = first + 4 * tid;
        if (j >= n) return;
#pragma unroll 8
        for (int h = 0; h < a.hq; ++h) {
            const float4 v = *reinterpret_cast<const float4*>(s + static_cast<int64_t>(h) * a.max_pages + j);
            const float2 c = norm[h];
            acc[0] += fast_exp2((score_of(v.x) - c.x) * kLog2e) * c.y;
            acc[1] += fast_exp2((score_of(v.y) - c.x) * kLog2e) * c.y;
            acc[2] += fast_exp2((score_of(v.z) - c.x) * kLog2e) * c.y;
            acc[3] += fast_exp2((score_of(v.w) - c.x) * kLog2e) * c.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < n)
                a.mass_out[base + j + e] = a.decay != 0.f ? a.mass[base + j + e] * a.decay + acc[e] : acc[e];
    } else {
#pragma unroll 4
        for (int h = 0; h < a.hq; ++h) {
            const float* r = s + static_cast<int64_t>(h) * a.max_pages;
            const float2 c = norm[h];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = first + e * kMassThreads + tid;
                if (j < n) acc[e] += fast_exp2((score_of(r[j]) - c.x) * kLog2e) * c.y;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = first + e * kMassThreads + tid;
            if (j < n) a.mass_out[base + j] = a.decay != 0.f ? a.mass[base + j] * a.decay + acc[e] : acc[e];
        }
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
// first write, so the outputs may be the inputs. The e-th smallest key is found by a radix
// select, most significant 8 bits first, on the order-preserving image of the mass; the
// CTAs' histograms are joined through distributed shared memory.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

struct EvictShared {
    uint32_t hist[2][256];
    uint32_t sum[256];
    int wsum[2][kEvictWarps];
    int digit, below;
    int cnt[2];                          // this CTA's pages below / at the threshold
};

__device__ __forceinline__ uint32_t mass_key(float m) { return orderable_key(m + 0.f); }   // -0 counts as 0

template <int CL>
__device__ __forceinline__ void join_sync() {
    if (CL == 1) __syncthreads();
    else cluster_sync_all();
}

// Exclusive scan of two flags over the CTA (in thread order) and their totals.
__device__ __forceinline__ void scan_flags(bool f0, bool f1, int (&pos)[2], int (&tot)[2], EvictShared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned b0 = __ballot_sync(0xffffffffu, f0), b1 = __ballot_sync(0xffffffffu, f1);
    if (lane == 0) sh.wsum[0][warp] = __popc(b0), sh.wsum[1][warp] = __popc(b1);
    __syncthreads();
    int p0 = 0, p1 = 0, t0 = 0, t1 = 0;
#pragma unroll
    for (int w = 0; w < kEvictWarps; ++w) {
        const int c0 = sh.wsum[0][w], c1 = sh.wsum[1][w];
        p0 += w < warp ? c0 : 0;
        p1 += w < warp ? c1 : 0;
        t0 += c0;
        t1 += c1;
    }
    __syncthreads();
    pos[0] = p0 + __popc(b0 & lanemask_lt());
    pos[1] = p1 + __popc(b1 & lanemask_lt());
    tot[0] = t0;
    tot[1] = t1;
}

template <int CL>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a, int share) {
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
    for (int i = tid; i < mine; i += kEvictThreads) {
        mass_s[i] = a.mass[base + first + i];
        table_s[i] = a.page_table[base + first + i];
    }
    // candidates: logical pages [lo, hi) of this CTA's share
    const int lo = max(0, a.sink - first), hi = min(mine, n - a.recent - first);
    uint32_t prefix = 0;
    int want = e;                                           // rank of the threshold among the candidates left
    if (e > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            uint32_t* hist = sh.hist[pass & 1];
            for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kEvictThreads) {
                const uint32_t key = mass_key(mass_s[i]);
                if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            join_sync<CL>();
            if (tid < 256) {
                uint32_t c = 0;
                if (CL == 1) {
                    c = hist[tid];
                } else {
#pragma unroll
                    for (int r = 0; r < CL; ++r) c += ld_dsmem_u32(dsmem_addr(&hist[tid], r));
                }
                sh.sum[tid] = c;
            }
            __syncthreads();
            if (tid < 32) {                                 // the bin that holds rank `want` (1-based)
                uint32_t c[8], t = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) t += c[i] = sh.sum[tid * 8 + i];
                uint32_t upto = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (tid >= o) upto += y;
                }
                uint32_t before = upto - t;
                if (before < static_cast<uint32_t>(want) && static_cast<uint32_t>(want) <= upto) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (before < static_cast<uint32_t>(want) && static_cast<uint32_t>(want) <= before + c[i]) {
                            sh.digit = tid * 8 + i;
                            sh.below = static_cast<int>(before);
                        }
                        before += c[i];
                    }
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | static_cast<uint32_t>(sh.digit);
            want -= sh.below;
        }
        // prefix is now the threshold key; `want` of the pages at it leave, lowest first
        int c0 = 0, c1 = 0;
        for (int i = lo + tid; i < hi; i += kEvictThreads) {
            const uint32_t key = mass_key(mass_s[i]);
            c0 += key < prefix;
            c1 += key == prefix;
        }
        c0 = __reduce_add_sync(0xffffffffu, c0);
        c1 = __reduce_add_sync(0xffffffffu, c1);
        if ((tid & 31) == 0) sh.wsum[0][tid >> 5] = c0, sh.wsum[1][tid >> 5] = c1;
        __syncthreads();
        if (tid == 0) {
            c0 = c1 = 0;
            for (int w = 0; w < kEvictWarps; ++w) c0 += sh.wsum[0][w], c1 += sh.wsum[1][w];
            sh.cnt[0] = c0;
            sh.cnt[1] = c1;
        }
    }
    join_sync<CL>();                                        // counts, and every CTA's inputs are read
    int out_before = 0, eq_before = 0;                      // evicted / at the threshold in lower CTAs
    if (e > 0 && CL > 1) {
        int less = 0;
        for (int r = 0; r < rank; ++r) {
            less += static_cast<int>(ld_dsmem_u32(dsmem_addr(&sh.cnt[0], r)));
            eq_before += static_cast<int>(ld_dsmem_u32(dsmem_addr(&sh.cnt[1], r)));
        }
        out_before = less + min(eq_before, want);
    }
#pragma unroll 1
    for (int i0 = 0; i0 < mine; i0 += kEvictThreads) {
        const int i = i0 + tid;
        const bool cand = e > 0 && i >= lo && i < hi;
        const uint32_t key = cand ? mass_key(mass_s[i]) : 0u;
        const bool less = cand && key < prefix, eq = cand && key == prefix;
        int pos[2], tot[2];
        scan_flags(less, eq, pos, tot, sh);
        // of the pages at the threshold, those before this one that leave
        const int eq_out = min(max(want - eq_before, 0), pos[1]);
        const bool gone = less || (eq && eq_before + pos[1] < want);
        const int before = out_before + pos[0] + eq_out;
        if (i < mine) {
            const int at = first + i;
            if (gone) {
                if (before < a.evict_cap) a.evicted[static_cast<int64_t>(b) * a.evict_cap + before] = table_s[i];
            } else {
                a.page_table_out[base + at - before] = table_s[i];
                a.mass_out[base + at - before] = mass_s[i];
            }
        }
        out_before += tot[0] + min(max(want - eq_before, 0), tot[1]);
        eq_before += tot[1];
    }
    if (rank == 0 && tid == 0) {
        a.n_evicted[b] = e;
        a.seq_pages_out[b] = n - e;
    }
    join_sync<CL>();                                        // shared memory stays until every reader is done
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

int mass_partials_row(int max_pages) { return (max_pages + kSlicePages - 1) / kSlicePages; }

cudaError_t launch_mass_partials(const MassArgs& a, float2* partials, cudaStream_t stream) {
    return launch_pdl(partials_kernel, dim3(a.row, a.hq, a.batch), kThreads, 0, stream, a, partials, rows_aligned(a));
}

cudaError_t launch_mass(const MassArgs& a, cudaStream_t stream) {
    const int blocks = (a.max_pages + kMassPages - 1) / kMassPages;
    return launch_pdl(mass_kernel, dim3(blocks, a.batch, 1), kMassThreads, a.hq * sizeof(float2), stream, a,
                      rows_aligned(a));
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    // A cluster barrier costs about as much as a pass over a few thousand pages: one CTA
    // takes short tables, sixteen the long ones (24,576 pages each at most).
    if (a.max_pages <= 4096) return launch_evict_t<1>(a, stream);
    return launch_evict_t<16>(a, stream);
}

}  // namespace locks
