// prefix_pages.cu - the parts of the shared-prefix attention (locks_prefix_attention) that go
// by pages on mma.sync, where a tile of 128 rows and 128 tokens would be mostly empty:
//
// 1. Few sequences, lists of up to 512 pages, in one launch. One cluster of eight CTAs per
//    (sequence, kv head): its 32 or 64 warps take the pages of the sequence's list (its group's
//    prefix, then its own) in turn with an online softmax, and their partials meet in shared
//    memory and then, a query head per CTA, through distributed shared memory. A prefix is read
//    once per sequence, which L2 serves; what the tiled kernel's evenly cut line, its pipeline
//    and its second launch cost (10 us at the least) is what this one saves: 12.1 -> 4.8 us for
//    two sequences behind 333 tokens. Latency bounds it.
//
// 2. Many sequences, in one launch where lists are short, else as the second launch behind the
//    tiled kernel, which has the prefixes: a CTA per (sequence, kv head) attends to the pages and
//    joins the prefix's partials, if any, to them. As items of the tiled kernel every (sequence,
//    kv head) takes a tile's pipeline of its own, about 2.8 us of an SM: 96 sequences of up to
//    100 tokens behind 16, 8 kv heads: 27.1 -> 8.9 us; behind 4000 tokens 38.2 -> 28.3.
//
// fp32 queries and the weights enter the products as a bf16 high and low part (what is left out
// of a weight is at most 2^-16 of it), as in the tiled kernel. What bounds a warp's page is its
// 32 products (fp32) and their chain, 0.3 us; copies of its next pages run beside them.
#include <type_traits>

#include "prefix_units.cuh"

namespace locks {
namespace {

constexpr int kRowBytes = kD * 2;
constexpr int kPageBytes = kPage * kRowBytes;
constexpr int kSlotBytes = 2 * kPageBytes;            // K and V of a page

// CTAs that an SM holds: 227 KB are 27 slots and the partials.
template <int kWarps, int kDepth>
constexpr int kCtasPerSm = 27 / (kWarps * kDepth);

// The one-launch form: a cluster of CTAs per (sequence, kv head).
constexpr int kCluster = 8;
constexpr int kSmallPages = 512;                      // longest list taken, see prefix_is_small
static_assert(kSmallPages <= 32 * kCluster * 4, "a warp's page ids lie in its lanes");
template <int kWarps>
struct Small {
    float m[kWarps][16], l[kWarps][16];               // warps' partials
    float cta_m[16], cta_l[16];                       // the CTA's
    float cta_o[16][kD];
};

// Byte offset of 16-byte chunk c of a token's row: swizzled, for ldmatrix.
__device__ __forceinline__ int chunk_offset(int token, int c) { return token * kRowBytes + ((c ^ (token & 7)) << 4); }

// 16 bytes, or zeros that read nothing.
__device__ __forceinline__ void copy_or_zero(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A sequence's tokens: its group's prefix, if any, and then its own.
struct List {
    int group, pre_tokens, own_tokens;
    int pre_pages, pages;
};
// Whole warps; `report` on one that reports bad counts and bounds.
__device__ __forceinline__ List find_list(const PrefixArgs& a, int b, bool report) {
    const int lane = threadIdx.x & 31;
    List r = {-1, 0, 0, 0, 0};
    if (a.num_groups > 0) {                              // up to 32: a group a lane
        Unit pre = {0, 0, 0, 0, false};
        const bool on = lane < a.num_groups;
        const int start = on ? __ldcg(a.group_start + lane) : 0, end = on ? __ldcg(a.group_start + lane + 1) : 0;
        const int tokens = on ? __ldcg(a.prefix_tokens + lane) : 0;
        int bound = 0;
        const int before = bound_before(start, bound);
        if (on) pre = group_unit(a, start, end, tokens, before);
        if (pre.bad && report) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        r.group = __ffs(__ballot_sync(0xffffffffu, on && b >= pre.seq0 && b < pre.seq0 + pre.num_seqs)) - 1;
        if (r.group >= 0) r.pre_tokens = __shfl_sync(0xffffffffu, pre.tokens, r.group);
    }
    return r;
}
// ... with the sequence's own tokens.
__device__ __forceinline__ void add_own(const PrefixArgs& a, int b, bool report, List& r) {
    const Unit own = own_unit(a, b, __ldcg(a.seq_tokens + b));
    if (own.bad && report) report_error(a.st, LOCKS_ERR_BAD_INDEX);
    r.own_tokens = own.tokens;
    r.pre_pages = (r.pre_tokens + kPage - 1) / kPage;
    r.pages = r.pre_pages + (own.tokens + kPage - 1) / kPage;
}
__device__ __forceinline__ int page_id(const PrefixArgs& a, const List& list, int b, int page) {
    const int x = __ldcg(page < list.pre_pages
                             ? a.prefix_table + static_cast<int64_t>(list.group) * a.max_prefix_pages + page
                             : a.page_table + static_cast<int64_t>(b) * a.max_pages + page - list.pre_pages);
    if (x >= 0 && x < a.num_phys) return x;
    report_error(a.st, LOCKS_ERR_BAD_INDEX);
    return 0;
}

// A warp's pages of sequence b's list: page first + i * step for i < count (up to 32, the id of
// page i in lane i). Products are formed with the
// queries as columns, S^T = K Q^T and O^T = V^T P^T, eight to a block: a group's few queries
// would leave most of sixteen rows empty (4 queries: 32 products a page, 64 as rows). Leaves, per
// column 2 * (lane % 4) + c of block n, the maximum m[n][c], this lane's part of the sum and the
// accumulator o[n][16 dims][.].
template <bool kSplitQ, int kBlocks, int kDepth>
__device__ __forceinline__ void attend_pages(const PrefixArgs& a, int b, int kvh, uint8_t* mine, int ids, int first,
                                             int step, int count, const List& list, float (&o)[kBlocks][8][4],
                                             float (&m)[kBlocks][2], float (&l)[kBlocks][2]) {
    const int lane = threadIdx.x & 31;
    const auto valid_of = [&](int page) {
        return min(kPage, page < list.pre_pages ? list.pre_tokens - page * kPage
                                                : list.own_tokens - (page - list.pre_pages) * kPage);
    };
    const auto load = [&](int i, int slot) {             // page i of this warp, its tokens alone
        const int id = __shfl_sync(0xffffffffu, ids, i), valid = valid_of(first + i * step);
        const int64_t at = (static_cast<int64_t>(id) * a.hkv + kvh) * (kPage * kD) + lane * 8;
        uint8_t* to = mine + slot * kSlotBytes;
#pragma unroll
        for (int j = 0; j < kPage / 2; ++j) {            // two tokens
            const int token = 2 * j + (lane >> 4), offset = chunk_offset(token, lane & 15);
            copy_or_zero(to + offset, a.k_cache + at + j * 2 * kD, token < valid);
            copy_or_zero(to + kPageBytes + offset, a.v_cache + at + j * 2 * kD, token < valid);
        }
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        if (i < count) load(i, i);
        copies_commit();
    }

    // query fragments (columns past the group are zero)
    const int gid = lane >> 2, tig = lane & 3, g = a.group;
    uint32_t qh[kBlocks][8][2], ql[kBlocks][kSplitQ ? 8 : 1][2];
    {
        const int64_t row = static_cast<int64_t>(b) * a.hq + kvh * g;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + gid;
                    const int64_t at = (row + r) * kD + k * 16 + e * 8 + tig * 2;
                    qh[n][k][e] = 0;
                    if (kSplitQ) ql[n][kSplitQ ? k : 0][e] = 0;
                    if (r < g) {
                        if (kSplitQ) {
                            const float2 v = __ldcg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at));
                            qh[n][k][e] = pack_bf16x2(v.x, v.y);
                            ql[n][kSplitQ ? k : 0][e] = pack_bf16x2(v.x - __uint_as_float(qh[n][k][e] << 16),
                                                                    v.y - __uint_as_float(qh[n][k][e] & 0xffff0000u));
                        } else {
                            qh[n][k][e] =
                                __ldcg(reinterpret_cast<const unsigned*>(static_cast<const uint16_t*>(a.q) + at));
                        }
                    }
                }
    }

#pragma unroll
    for (int n = 0; n < kBlocks; ++n) {
#pragma unroll
        for (int d = 0; d < 8; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    int at = 0;                                          // the slot of page i
    for (int i = 0; i < count; ++i) {
        const uint8_t* slot = mine + at * kSlotBytes;
        copies_wait<kDepth - 1>();
        __syncwarp();
        const int valid = valid_of(first + i * step);
        // scores of 16 tokens; two sums each (of fp32 queries' high and low parts, else of every
        // other k), as a product waits for the one before
        float s[kBlocks][4], t[kBlocks][4];
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = t[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t r[4];
            ldmatrix_x4(r, slot + chunk_offset((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) {
                if (kSplitQ || k % 2 == 0) mma_bf16_16816(s[n], r, qh[n][k][0], qh[n][k][1]);
                if (kSplitQ) mma_bf16_16816(t[n], r, ql[n][kSplitQ ? k : 0][0], ql[n][kSplitQ ? k : 0][1]);
                else if (k % 2 == 1) mma_bf16_16816(t[n], r, qh[n][k][0], qh[n][k][1]);
            }
        }
        uint32_t p[kBlocks][2], pl[kBlocks][2];          // high and low parts
        float f[kBlocks][2];
        bool same = true;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
            // tokens past the end have no weight (and zeros for values); e: token gid + 8 * (e / 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = gid + 8 * (e >> 1) < valid ? s[n][e] + t[n][e] : -INFINITY;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float top = fmaxf(s[n][c], s[n][c + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float to = fmaxf(m[n][c], top), base = to == -INFINITY ? 0.f : to * kScaleLog2;
                f[n][c] = m[n][c] == to ? 1.f : fast_exp2(fmaf(m[n][c], kScaleLog2, -base));
                same = same && f[n][c] == 1.f;
                m[n][c] = to;
                s[n][c] = fast_exp2(fmaf(s[n][c], kScaleLog2, -base));
                s[n][c + 2] = fast_exp2(fmaf(s[n][c + 2], kScaleLog2, -base));
                l[n][c] = l[n][c] * f[n][c] + (s[n][c] + s[n][c + 2]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {                // tokens down, queries along: turned
                const uint32_t hi = pack_bf16x2(s[n][2 * h], s[n][2 * h + 1]);
                p[n][h] = movmatrix_trans(hi);
                pl[n][h] = movmatrix_trans(pack_bf16x2(s[n][2 * h] - __uint_as_float(hi << 16),
                                                       s[n][2 * h + 1] - __uint_as_float(hi & 0xffff0000u)));
            }
        }
        if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
            for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                for (int d = 0; d < 8; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][d][e] *= f[n][e & 1];
        }
        constexpr int kDims = kBlocks == 1 ? 4 : 2;      // sixteen dims at a time, between a sum's two products
#pragma unroll
        for (int d0 = 0; d0 < 8; d0 += kDims) {
            uint32_t r[kDims][4];
#pragma unroll
            for (int d = 0; d < kDims; ++d)
                ldmatrix_x4_trans(r[d], slot + kPageBytes + chunk_offset((lane & 7) + (lane >> 4) * 8,
                                                                         2 * (d0 + d) + ((lane >> 3) & 1)));
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) {
#pragma unroll
                for (int d = 0; d < kDims; ++d) mma_bf16_16816(o[n][d0 + d], r[d], p[n][0], p[n][1]);
#pragma unroll
                for (int d = 0; d < kDims; ++d) mma_bf16_16816(o[n][d0 + d], r[d], pl[n][0], pl[n][1]);
            }
        }
        __syncwarp();
        if (i + kDepth < count) load(i + kDepth, at);
        copies_commit();
        if (++at == kDepth) at = 0;
    }
}

// A warp's partial into shared memory: the accumulator, a query a row, over its slots, which
// nothing is copied into any more.
constexpr int kPartStride = kD + 4;                      // floats: eight queries' stores in different banks
template <int kBlocks>
__device__ __forceinline__ void put_partial(uint8_t* mine, float* m_s, float* l_s, const float (&o)[kBlocks][8][4],
                                            const float (&m)[kBlocks][2], float (&l)[kBlocks][2]) {
    const int gid = (threadIdx.x & 31) >> 2, tig = threadIdx.x & 3;
    float* o_s = reinterpret_cast<float*>(mine);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int x = 4; x < 32; x *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
            if (gid == 0) m_s[n * 8 + tig * 2 + c] = m[n][c], l_s[n * 8 + tig * 2 + c] = l[n][c];
        }
#pragma unroll
        for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o_s[(n * 8 + tig * 2 + (e & 1)) * kPartStride + d * 16 + gid + 8 * (e >> 1)] = o[n][d][e];
    }
}

// Row r of the warps' partials, four dims a lane.
template <int kWarps, int kDepth>
__device__ __forceinline__ float4 row_of_warps(const uint8_t* slots, const float (*m_s)[16], const float (*l_s)[16], int r,
                                               float& top, float& sum) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = fast_exp2((m_s[w][r] - base) * kScaleLog2);
        const float4 v = *reinterpret_cast<const float4*>(slots + w * kDepth * kSlotBytes +
                                                          (r * kPartStride + (threadIdx.x & 31) * 4) * 4);
        sum += f * l_s[w][r];
        x.x += f * v.x, x.y += f * v.y, x.z += f * v.z, x.w += f * v.w;
    }
    return x;
}

template <bool kSplitQ, int kBlocks, int kWarps, int kDepth>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<kWarps, kDepth>)
    small_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(1024) uint8_t slots[];
    constexpr int kAllWarps = kCluster * kWarps;
    auto* sh = reinterpret_cast<Small<kWarps>*>(slots + kWarps * kDepth * kSlotBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int seg = blockIdx.x / kCluster, b = seg / a.hkv, kvh = seg % a.hkv, g = a.group;
    uint8_t* mine = slots + warp * kDepth * kSlotBytes;
    grid_dependency_wait();
    allow_dependent_launch();

    List list = find_list(a, b, rank == 0 && warp == 0);
    add_own(a, b, rank == 0 && threadIdx.x == 0, list);
    const int first = rank * kWarps + warp;              // this warp's pages: first, first + kAllWarps, ...
    const int count = list.pages > first ? (list.pages - first + kAllWarps - 1) / kAllWarps : 0;
    const int ids = lane < count ? page_id(a, list, b, first + lane * kAllWarps) : 0;
    float o[kBlocks][8][4], m[kBlocks][2], l[kBlocks][2];
    attend_pages<kSplitQ, kBlocks, kDepth>(a, b, kvh, mine, ids, first, kAllWarps, count, list, o, m, l);
    put_partial<kBlocks>(mine, sh->m[warp], sh->l[warp], o, m, l);
    // the CTA's partial from the warps'
    __syncthreads();
    for (int r = warp; r < g; r += kWarps) {
        float top, sum;
        const float4 x = row_of_warps<kWarps, kDepth>(slots, sh->m, sh->l, r, top, sum);
        *reinterpret_cast<float4*>(&sh->cta_o[r][lane * 4]) = x;
        if (lane == 0) sh->cta_m[r] = top, sh->cta_l[r] = sum;
    }
    cluster_sync_all();
    const int dim = threadIdx.x % kD;
    for (int r = rank + kCluster * (threadIdx.x / kD); r < g; r += kCluster * (kWarps * 32 / kD)) {   // a query head per CTA
        float cm[kCluster], cl[kCluster], co[kCluster], top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            cm[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_m[r], c));
            cl[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_l[r], c));
            co[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_o[r][dim], c));
        }
#pragma unroll
        for (int c = 0; c < kCluster; ++c) top = fmaxf(top, cm[c]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const float f = fast_exp2((cm[c] - base) * kScaleLog2);
            sum += f * cl[c];
            x += f * co[c];
        }
        const int64_t row = static_cast<int64_t>(b) * a.hq + kvh * g + r;
        const float v = list.pages > 0 ? x / sum : 0.f;
        reinterpret_cast<__nv_bfloat16*>(a.out)[row * kD + dim] = __float2bfloat16_rn(v);
        if (a.lse && dim == 0) a.lse[row] = list.pages > 0 ? fmaf(top, kInvSqrtD, logf(sum)) : -INFINITY;
    }
    cluster_sync_all();                                  // shared memory stays until every CTA has read it
}

template <bool kSplitQ, int kBlocks, int kWarps, int kDepth>
cudaError_t launch_small_t(const PrefixArgs& a, cudaStream_t stream) {
    constexpr int kBytes = kWarps * kDepth * kSlotBytes + static_cast<int>(sizeof(Small<kWarps>));
    cudaError_t e = ensure_kernel_attrs<small_kernel<kSplitQ, kBlocks, kWarps, kDepth>>(kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * a.hkv * kCluster, 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, small_kernel<kSplitQ, kBlocks, kWarps, kDepth>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The second launch where own tokens are attended to by pages: a CTA per (sequence, kv head),
// its warps taking the list's pages in turn, and then a warp per query head joining their
// partials and the prefix's. Own tokens need nothing from the first launch, every CTA of which
// waited for what lies before it before it let this one start: so they are read ahead of the
// wait, past L1, by the CTAs that find room while the first launch ends. `alone`: there is no
// first launch, and the list holds the prefix too.
template <int kWarps>
struct Own {
    float m[kWarps][16], l[kWarps][16];
};
constexpr int kOwnPages = 32 * 4;                     // longest list taken: a warp's page ids lie in its lanes

template <bool kSplitQ, int kBlocks, int kWarps, int kDepth>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<kWarps, kDepth>)
    own_kernel(const __grid_constant__ PrefixArgs a, int grid, bool alone) {
    extern __shared__ __align__(1024) uint8_t slots[];
    auto* sh = reinterpret_cast<Own<kWarps>*>(slots + kWarps * kDepth * kSlotBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / a.hkv, kvh = blockIdx.x % a.hkv, g = a.group;
    uint8_t* mine = slots + warp * kDepth * kSlotBytes;
    List list = {-1, 0, 0, 0, 0};
    if (alone) {
        grid_dependency_wait();
        list = find_list(a, b, warp == 0);
    }
    add_own(a, b, threadIdx.x == 0, list);
    const int count = list.pages > warp ? (list.pages - warp + kWarps - 1) / kWarps : 0;
    const int ids = lane < count ? page_id(a, list, b, warp + lane * kWarps) : 0;
    float o[kBlocks][8][4], m[kBlocks][2], l[kBlocks][2];
    attend_pages<kSplitQ, kBlocks, kDepth>(a, b, kvh, mine, ids, warp, kWarps, count, list, o, m, l);
    put_partial<kBlocks>(mine, sh->m[warp], sh->l[warp], o, m, l);
    __syncthreads();
    if (!alone) grid_dependency_wait();
    allow_dependent_launch();
    int64_t total = 0;
    PrefixSeq s;
    s.pre_tiles = 0;
    if (!alone) {
        total = *a.total;
        s = a.seqs[b];
    }
    for (int r = warp; r < g; r += kWarps) {
        float top, sum;
        float4 x = row_of_warps<kWarps, kDepth>(slots, sh->m, sh->l, r, top, sum);
        const PrefixRows p = prefix_rows(a, s, b, kvh, r, total, ctas_of(total, grid));
        const auto part_row = [&](int i) { return p.row + static_cast<int64_t>(i) * kTile; };
        for (int i = 0; i < p.count; i += 8) join_partials<8>(a, part_row, i, p.count, top, sum, x);
        const int64_t row = static_cast<int64_t>(b) * a.hq + kvh * g + r;
        const bool some = list.pages > 0 || p.count > 0;
        const float inv = some ? 1.f / sum : 0.f;
        *reinterpret_cast<uint2*>(a.out + row * kD + lane * 4) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
        if (a.lse && lane == 0) a.lse[row] = some ? fmaf(top, kInvSqrtD, logf(sum)) : -INFINITY;
    }
}

template <bool kSplitQ, int kBlocks, int kWarps, int kDepth>
cudaError_t launch_own_t(const PrefixArgs& a, int grid, cudaStream_t stream) {
    constexpr int kBytes = kWarps * kDepth * kSlotBytes + static_cast<int>(sizeof(Own<kWarps>));
    cudaError_t e = ensure_kernel_attrs<own_kernel<kSplitQ, kBlocks, kWarps, kDepth>>(kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * a.hkv, 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, own_kernel<kSplitQ, kBlocks, kWarps, kDepth>, a, grid, a.own_alone);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// By the tables' widths, which is what the host knows, and up to two CTAs an SM. Measured (this
// one / the tiled kernel and its second launch, us; kv heads x queries each): 1 sequence 8 x 4,
// 515 pages 9.4 / 16.9; 4 sequences 8 x 4 (256 CTAs), 259 pages 10.3 / 13.5, 515 pages 15.3 /
// 16.9; 1 sequence 2 x 16, 515 pages 12.6 / 12.8; 14 sequences 2 x 16 (224 CTAs), 378 pages
// 17.2 / 17.0; 7 sequences 8 x 4 (448 CTAs), 67 pages 11.9 / 10.6. Groups are looked for by one
// warp.
static int64_t list_pages(const PrefixArgs& a) {
    return static_cast<int64_t>(a.num_groups > 0 ? a.max_prefix_pages : 0) + a.max_pages;
}
static int64_t small_ctas(const PrefixArgs& a) { return static_cast<int64_t>(a.batch) * a.hkv * kCluster; }
// Eight warps a CTA, one CTA an SM, for longer lists where the clusters fit side by side: 14
// do, 16 run in two rounds (1024 tokens: 7.2 us, 9.3). Eight warps / four: 515 pages 9.4 / 11.1
// us, 131 pages 6.2 / 6.1, 19 pages 5.0 / 4.4.
static bool small_is_wide(const PrefixArgs& a, int num_sms) {
    return 4 * small_ctas(a) <= 3 * static_cast<int64_t>(num_sms) && list_pages(a) > 192;
}
bool prefix_is_small(const PrefixArgs& a, int num_sms) {
    if (list_pages(a) <= 16 && a.group <= 8) return false;    // list_by_pages: 3.3 - 4.2 us for 4.4
    if (a.num_groups > 32 || small_ctas(a) > 2 * static_cast<int64_t>(num_sms)) return false;
    return list_pages(a) <= (a.group <= 8 || small_is_wide(a, num_sms) ? kSmallPages : 384);
}

cudaError_t launch_prefix_small(const PrefixArgs& a, int num_sms, cudaStream_t stream) {
    const bool wide = small_is_wide(a, num_sms);
    const auto launch = [&](auto split, auto blocks) {
        constexpr bool kSplitQ = decltype(split)::value;
        constexpr int kBlocks = decltype(blocks)::value;
        return wide ? launch_small_t<kSplitQ, kBlocks, 8, 2>(a, stream) : launch_small_t<kSplitQ, kBlocks, 4, 3>(a, stream);
    };
    const auto by_group = [&](auto split) {
        return a.group <= 8 ? launch(split, std::integral_constant<int, 1>()) : launch(split, std::integral_constant<int, 2>());
    };
    return a.q_type == LOCKS_FP32 ? by_group(std::true_type()) : by_group(std::false_type());
}

// Measured (this / the other forms, us; 8 kv heads of 4 queries; tables of 1 + 7 pages): 7
// sequences 3.9 / 9.9, 96 sequences 8.9 / 17.7, 256 sequences 22.6 / 34.0. Every sequence reads
// the prefix for itself: 21 prefix pages and one of its own, 96 sequences 15.1 / 18.0, 256
// sequences 34.4 / 29.5; 63 and one, 15 sequences 10.1 / 11.4 with four warps a CTA, 40
// sequences 15.5 / 14.4. 1 + 119 pages: 96 sequences 64.1 / 71.8, 256 143.5 / 166.5. Sixteen
// queries to a kv head, 2 kv heads, 96 sequences: 21 + 21 pages 17.5 / 19.3, 1 + 63 23.3 / 22.8.
bool list_by_pages(const PrefixArgs& a, int num_sms) {
    if (a.num_groups > 32 || list_pages(a) > (a.group > 8 ? 48 : kOwnPages)) return false;
    const int64_t ctas = static_cast<int64_t>(a.batch) * a.hkv, room = 3 * static_cast<int64_t>(num_sms);
    const int64_t prefix = a.num_groups > 0 ? a.max_prefix_pages : 0;
    const int64_t most = a.group > 8 ? 24 : ctas <= num_sms ? 96 : 48;    // pages of a prefix, one wave of CTAs
    return prefix * (ctas > room ? ctas : room) <= most * room;
}

bool own_by_pages(const PrefixArgs& a, int num_sms) {
    // Measured (this / as items of the tiled kernel, us; 8 kv heads of 4 queries, a prefix of
    // 4000 tokens): 96 sequences of up to 1 page 24.9 / 37.0, 32 pages 40.0 / 45.8, 125 pages
    // 82.8 / 79.1; 19 sequences 15.2 / 17.9, 19.3 / 21.5, 33.8 / 28.1. Sixteen queries to a kv
    // head (96 sequences, 2 kv heads) 26.1 / 27.1, 32.1 / 29.3.
    if (a.group > 8 || a.max_pages > 64) return false;
    // A warp joins its rows one after the other, eight partials at a time, 0.7 us each; the
    // tiled kernel's own second launch has more warps for them. A prefix's block of rows has
    // about num_sms / (all blocks) partials.
    const int64_t rows = static_cast<int64_t>(a.batch) * a.group;
    const int64_t pieces = num_sms / (a.hkv * ((rows + kTile - 1) / kTile)) + 1;
    return (a.group + 3) / 4 * ((pieces + 7) / 8) <= 6;
}

cudaError_t launch_own(const PrefixArgs& a, int grid, cudaStream_t stream) {
    // Three CTAs an SM, or two with a page more in flight where that is room enough (19
    // sequences of up to 125 pages, 8 kv heads: 27.6 / 23.7 us; 96 sequences of one page 16.6 /
    // 19.2), or one of eight warps for long lists of few sequences (16 sequences of 64 pages
    // behind 128K tokens: 97.1, 94.4, 91.9).
    const int64_t ctas = static_cast<int64_t>(a.batch) * a.hkv, pages = a.own_alone ? list_pages(a) : a.max_pages;
    const auto launch = [&](auto split) {
        constexpr bool kSplitQ = decltype(split)::value;
        if (a.group > 8) return launch_own_t<kSplitQ, 2, 4, 2>(a, grid, stream);
        return ctas > 2 * grid                    ? launch_own_t<kSplitQ, 1, 4, 2>(a, grid, stream)
               : ctas > grid || pages <= 32       ? launch_own_t<kSplitQ, 1, 4, 3>(a, grid, stream)
                                                  : launch_own_t<kSplitQ, 1, 8, 2>(a, grid, stream);
    };
    return a.q_type == LOCKS_FP32 ? launch(std::true_type()) : launch(std::false_type());
}

}  // namespace locks
