// prefix_small.cu - the shared-prefix attention (locks_prefix_attention) for short lists and
// few sequences, in one launch.
//
// One cluster of eight CTAs per (sequence, kv head): its 32 warps take the pages of the
// sequence's list (its group's prefix, then its own) in turn, sixteen queries x sixteen
// tokens at a time on mma.sync with an online softmax, and their partials meet in shared
// memory and then, a query head per CTA, through distributed shared memory. A prefix is read
// once per sequence, which L2 serves; what the tiled kernel's evenly cut line, its pipeline
// and its second launch cost (11 us at the least) is what this one saves: 12.1 -> 6.1 us for
// two sequences behind 333 tokens. Latency bounds it: a list of 16 pages or fewer takes 5 us.
//
// A warp keeps two pages in flight, each as four 2 KB TMA boxes; fp32 queries enter the
// products as a bf16 high and low part, weights are rounded to bf16 once (at most 2^-8 of
// the sum of |weight * v|), as there.
#include "prefix_units.cuh"

namespace locks {
namespace {

constexpr int kCluster = 8;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kAllWarps = kCluster * kWarps;
constexpr int kBoxBytes = kPage * 128;
constexpr int kSlotBytes = 4 * kBoxBytes;             // K and V of a page, two 64-dim halves each
constexpr int kSmallPages = 256;                      // longest list taken, see prefix_is_small
static_assert(kSmallPages <= 32 * kAllWarps, "a warp's page ids lie in its lanes");
constexpr uint64_t kDrainNs = 500000000ull;           // a load that was issued lands by itself

struct Small {
    uint64_t full[kWarps][2];
    float m[kWarps][16], l[kWarps][16];               // warps' partials
    float cta_m[16], cta_l[16];                       // the CTA's
    float cta_o[16][kD];
};
constexpr int kSmemBytes = kWarps * 2 * kSlotBytes + static_cast<int>(sizeof(Small));

// Byte offset of (token, dim) in a slot's K or V: 16-byte chunks swizzled with the token.
__device__ __forceinline__ int slot_offset(int token, int dim) {
    return (dim >> 6) * kBoxBytes + token * 128 + ((((dim & 63) >> 3) ^ (token & 7)) << 4);
}

template <bool kSplitQ>
__global__ void __launch_bounds__(kThreads, 2) small_kernel(const __grid_constant__ PrefixArgs a) {
    extern __shared__ __align__(1024) uint8_t slots[];   // boxes: 1024-byte aligned
    Small* sh = reinterpret_cast<Small*>(slots + kWarps * 2 * kSlotBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int seg = blockIdx.x / kCluster, b = seg / a.hkv, kvh = seg % a.hkv, g = a.group;
    uint8_t* mine = slots + warp * 2 * kSlotBytes;
    if (lane == 0) {
        mbar_init(&sh->full[warp][0], 1);
        mbar_init(&sh->full[warp][1], 1);
        fence_barrier_init();
    }
    __syncwarp();
    grid_dependency_wait();
    allow_dependent_launch();

    // the sequence's group, a group a lane
    Unit pre = {0, 0, 0, 0, false};
    int group = -1;
    if (a.num_groups > 0) {
        const bool on = lane < a.num_groups;
        const int start = on ? a.group_start[lane] : 0, end = on ? a.group_start[lane + 1] : 0;
        const int tokens = on ? a.prefix_tokens[lane] : 0;
        int bound = 0;
        const int before = bound_before(start, bound);
        if (on) pre = group_unit(a, start, end, tokens, before);
        if (pre.bad && rank == 0 && warp == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        const unsigned in = __ballot_sync(0xffffffffu, on && b >= pre.seq0 && b < pre.seq0 + pre.num_seqs);
        group = __ffs(in) - 1;
    }
    const int pre_tokens = group >= 0 ? __shfl_sync(0xffffffffu, pre.tokens, group) : 0;
    const Unit own = own_unit(a, b, a.seq_tokens[b]);
    if (own.bad && rank == 0 && threadIdx.x == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
    const int pre_pages = (pre_tokens + kPage - 1) / kPage, pages = pre_pages + (own.tokens + kPage - 1) / kPage;
    const int first = rank * kWarps + warp;              // this warp's pages: first, first + 32, ...
    const int count = pages > first ? (pages - first + kAllWarps - 1) / kAllWarps : 0;
    int ids = 0;                                         // of page first + 32 * lane
    if (lane < count) {
        const int page = first + lane * kAllWarps;
        ids = page < pre_pages ? a.prefix_table[static_cast<int64_t>(group) * a.max_prefix_pages + page]
                               : a.page_table[static_cast<int64_t>(b) * a.max_pages + page - pre_pages];
        if (ids < 0 || ids >= a.num_phys) {
            report_error(a.st, LOCKS_ERR_BAD_INDEX);
            ids = 0;
        }
    }
    auto load = [&](int i) {                             // page i of this warp into slot i % 2
        const int id = __shfl_sync(0xffffffffu, ids, i);
        uint64_t* bar = &sh->full[warp][i & 1];
        if (lane == 0) mbar_arrive_expect_tx(bar, kSlotBytes);
        __syncwarp();
        if (lane < 4)                                    // K halves, V halves
            tma_load_2d(mine + (i & 1) * kSlotBytes + lane * kBoxBytes, lane < 2 ? &a.tm_k : &a.tm_v, (lane & 1) * 64,
                        (id * a.hkv + kvh) * kPage, bar);
    };
    if (count > 0) load(0);
    if (count > 1) load(1);

    // query fragments (rows gid and gid + 8 of the group; rows past it are zero)
    const int gid = lane >> 2, tig = lane & 3;
    uint32_t qh[8][4], ql[kSplitQ ? 8 : 1][4];
    {
        const int64_t row = static_cast<int64_t>(b) * a.hq + kvh * g;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = gid + (e & 1) * 8, c = k * 16 + (e >> 1) * 8 + tig * 2;
                qh[k][e] = 0;
                if (kSplitQ) ql[kSplitQ ? k : 0][e] = 0;
                if (r < g) {
                    if (kSplitQ) {
                        const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + (row + r) * kD + c);
                        qh[k][e] = pack_bf16x2(v.x, v.y);
                        ql[kSplitQ ? k : 0][e] = pack_bf16x2(v.x - __uint_as_float(qh[k][e] << 16),
                                                             v.y - __uint_as_float(qh[k][e] & 0xffff0000u));
                    } else {
                        qh[k][e] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + (row + r) * kD + c);
                    }
                }
            }
    }

    float o[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    for (int i = 0; i < count; ++i) {
        uint8_t* slot = mine + (i & 1) * kSlotBytes;
        ok = mbar_wait_bounded(&sh->full[warp][i & 1], (i >> 1) & 1, a.st.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) report_error(a.st, LOCKS_ERR_TIMEOUT);
            for (int k = i; k < min(i + 2, count); ++k)
                mbar_wait_bounded(&sh->full[warp][k & 1], (k >> 1) & 1, kDrainNs);
            break;
        }
        const int page = first + i * kAllWarps;
        const int valid = min(kPage, page < pre_pages ? pre_tokens - page * kPage : own.tokens - (page - pre_pages) * kPage);
        // scores of 16 queries x 16 tokens
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t r[4];
            ldmatrix_x4(r, slot + slot_offset((lane & 7) + ((lane >> 4) << 3), k * 16 + ((lane >> 3) & 1) * 8));
            mma_bf16_16816(s[0], qh[k], r[0], r[1]);
            mma_bf16_16816(s[1], qh[k], r[2], r[3]);
            if (kSplitQ) {
                mma_bf16_16816(s[0], ql[kSplitQ ? k : 0], r[0], r[1]);
                mma_bf16_16816(s[1], ql[kSplitQ ? k : 0], r[2], r[3]);
            }
        }
        if (valid < kPage) {
            // tokens past the end: no weight, and rows of V that cannot reach a sum as 0 * NaN
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n * 8 + tig * 2 + (e & 1) >= valid) s[n][e] = -INFINITY;
            for (int j = lane; j < (kPage - valid) * 16; j += 32)
                *reinterpret_cast<uint4*>(slot + 2 * kBoxBytes + ((j >> 3) & 1) * kBoxBytes + (valid + (j >> 4)) * 128 +
                                          (j & 7) * 16) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {                    // row gid, then row gid + 8
            float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float to = fmaxf(m[h], top), base = to == -INFINITY ? 0.f : to * kScaleLog2;
            const float f = m[h] == to ? 1.f : fast_exp2(fmaf(m[h], kScaleLog2, -base));
            m[h] = to;
            l[h] *= f;
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float u = fast_exp2(fmaf(s[n][2 * h], kScaleLog2, -base));
                const float v = fast_exp2(fmaf(s[n][2 * h + 1], kScaleLog2, -base));
                l[h] += u + v;
                p[2 * n + h] = pack_bf16x2(u, v);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {                    // sixteen dims at a time
            uint32_t r[4];
            ldmatrix_x4_trans(r, slot + 2 * kBoxBytes +
                                     slot_offset((lane & 7) + ((lane >> 3) & 1) * 8, n * 16 + (lane >> 4) * 8));
            mma_bf16_16816(o[2 * n], p, r[0], r[1]);
            mma_bf16_16816(o[2 * n + 1], p, r[2], r[3]);
        }
        if (i + 2 < count) {
            fence_proxy_async_smem();
            __syncwarp();
            load(i + 2);
        }
    }

    // the warp's partial over its own slots, the CTA's from the warps'
    float* o_s = reinterpret_cast<float*>(mine);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (tig == 0) sh->m[warp][gid + 8 * h] = m[h], sh->l[warp][gid + 8 * h] = l[h];
#pragma unroll
        for (int n = 0; n < 16; ++n)
            *reinterpret_cast<float2*>(o_s + (gid + 8 * h) * kD + n * 8 + tig * 2) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
    }
    __syncthreads();
    for (int r = 0; r < g; ++r) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh->m[w][r]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2((sh->m[w][r] - base) * kScaleLog2);
            sum += f * sh->l[w][r];
            x += f * reinterpret_cast<const float*>(slots + w * 2 * kSlotBytes)[r * kD + threadIdx.x];
        }
        sh->cta_o[r][threadIdx.x] = x;
        if (threadIdx.x == 0) sh->cta_m[r] = top, sh->cta_l[r] = sum;
    }
    cluster_sync_all();
    for (int r = rank; r < g; r += kCluster) {           // a query head per CTA
        float cm[kCluster], cl[kCluster], co[kCluster], top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            cm[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_m[r], c));
            cl[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_l[r], c));
            co[c] = ld_dsmem_f32(dsmem_addr(&sh->cta_o[r][threadIdx.x], c));
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
        const float v = pages > 0 ? x / sum : 0.f;
        reinterpret_cast<__nv_bfloat16*>(a.out)[row * kD + threadIdx.x] = __float2bfloat16_rn(v);
        if (a.lse && threadIdx.x == 0) a.lse[row] = pages > 0 ? fmaf(top, kInvSqrtD, logf(sum)) : -INFINITY;
    }
    cluster_sync_all();                                  // shared memory stays until every CTA has read it
}

template <bool kSplitQ>
cudaError_t launch_small_t(const PrefixArgs& a, cudaStream_t stream) {
    cudaError_t e = ensure_kernel_attrs<small_kernel<kSplitQ>>(kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * a.hkv * kCluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
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
    e = cudaLaunchKernelEx(&cfg, small_kernel<kSplitQ>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool prefix_is_small(const PrefixArgs& a, int num_sms) {
    // By the tables' widths, which is what the host knows. Measured on both kernels (this one /
    // the tiled one, us), 8 kv heads of 4 queries: 1 sequence 64 pages 6.6 / 12.3, 256 pages
    // 10.9 / 13.6, 512 pages 16.9 / 17.6; 2 sequences 256 pages 12.4 / 14.0, 512 pages
    // 19.4 / 17.7; 4 sequences 128 pages 11.7 / 13.5, 256 pages 16.2 / 15.2; 7 sequences 64
    // pages 15.3 / 13.3. So: up to 256 pages where every CTA has an SM, up to 160 where two
    // CTAs share one. Groups are looked for by one warp.
    const int64_t pages = static_cast<int64_t>(a.num_groups > 0 ? a.max_prefix_pages : 0) + a.max_pages;
    const int64_t ctas = static_cast<int64_t>(a.batch) * a.hkv * kCluster;
    if (a.num_groups > 32) return false;
    return ctas <= num_sms ? pages <= kSmallPages : ctas <= 2 * static_cast<int64_t>(num_sms) && pages <= 160;
}

cudaError_t launch_prefix_small(const PrefixArgs& a, cudaStream_t stream) {
    return a.q_type == LOCKS_FP32 ? launch_small_t<true>(a, stream) : launch_small_t<false>(a, stream);
}

}  // namespace locks
