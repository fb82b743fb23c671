// packed_attend.cu - decode attention over packed pages (locks_packed_attention).
//
// All steps of the call, a page of a kv head each (a recent bf16 page counts kRecentSteps),
// lie on one line, row after row (a row is a sequence and a kv head). The line is cut evenly
// into CTAs and a CTA's part into warps, whatever the lengths of the rows, and a warp goes
// through its pages with an online softmax. A row that ends up in several warps is joined in
// shared memory at the CTA's end, one that goes past the CTA by a second kernel.
//
// The products are formed on mma.sync with the queries as columns, S^T = K Q^T and
// O^T = V^T P^T: few queries read a page, so HBM bounds the call as long as a page costs a warp
// few instructions. The codes lie in the pages in the order of the A fragments, so that a lane
// loads its fragments with four 16-byte loads, and a pair of codes becomes a pair of bf16
// values by one AND: a 4-bit field in the low byte of a bf16 is the subnormal (or first
// normal) number field * 2^-133, exactly. Fields 4 bits further up count 16 times as much; the
// queries' side is divided by 16 there, for values the output. What is left of 2^-133 after
// the scaling of queries and weights by powers of two goes into the final factors. A token's
// scales multiply the group's sums (keys) or the weights (values); zeros enter through a
// product of their own with the queries' sums (keys) and through a sum per group (values).
#include <algorithm>

#include "pool_internal.h"

namespace locks {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRecentSteps = 3;                       // 8 KB against 2.4
constexpr float kScaleLog2 = kInvSqrtD * kLog2e;
// Queries are scaled by 2^(100 - e), e the exponent of the row's largest (within -20..60, so that
// the factor is a number); scores are then in units of 2^(e - 33). Recent keys are scaled by 2^-60,
// so that neither they nor their products leave fp32's range.
constexpr float kQueryShift = 0x1p100f, kRecentScore = 0x1p-73f;
// Weights carry 2^40, so that their products with codes stay normal numbers.
constexpr float kWeightBits = 40.f;
constexpr float kSumUnit = 0x1p-40f, kOutUnit = 0x1p93f, kRecentWeight = 0x1p-133f;
constexpr float kSlack = 8.f;                         // log2 that a score may pass the maximum by

// Variants: queries of a group in one block of 8 columns together with their low parts (kPair,
// groups up to 4), in one block, or in two.
template <int kKind>
struct Shape;
template <>
struct Shape<0> {
    static constexpr bool kPair = true;
    static constexpr int kBlocks = 1, kWarps = 8, kCtas = 2, kDepth = 4, kRows = 4;
};
template <>
struct Shape<1> {
    static constexpr bool kPair = false;
    static constexpr int kBlocks = 1, kWarps = 12, kCtas = 1, kDepth = 5, kRows = 8;
};
template <>
struct Shape<2> {
    static constexpr bool kPair = false;
    static constexpr int kBlocks = 2, kWarps = 8, kCtas = 1, kDepth = 7, kRows = 16;
};

constexpr int kPartStride = kD + 4;                   // floats: columns' stores in different banks
template <int kRows>
constexpr int kPartBytes = kRows * kPartStride * 4;

// Shared memory of a CTA besides the slots and the partials.
template <int kWarps, int kRows>
struct Control {
    int64_t upto[kWarps * 32];                        // steps of the sequences up to each thread's last
    int64_t warp_sum[kWarps];
    struct Entry {
        int64_t step0;                                // the row's first step on the line
        int32_t row, len;                             // -1: unused; steps of the row
        int32_t begins, ends;                         // the part holds the row's first / last step
    } entry[kWarps * 2];                              // a warp's first row, and its last
    float m[kWarps * 2][kRows], l[kWarps * 2][kRows];
};

// 16 bytes, or zeros that read nothing.
__device__ __forceinline__ void copy_or_zero(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ float low_of(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_of(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

struct Len {
    int pages, recent;                                // packed pages; recent tokens
    __device__ int recent_pages() const { return (recent + kPage - 1) / kPage; }
    __device__ int steps() const { return pages + kRecentSteps * recent_pages(); }
};
__device__ __forceinline__ int checked(const PackedArgs& a, int n, int64_t most, bool report) {
    if (n >= 0 && n <= most) return n;
    if (report) report_error(a.st, LOCKS_ERR_BAD_INDEX);
    return 0;
}
__device__ __forceinline__ Len row_len(const PackedArgs& a, int b, int h, bool report) {
    Len r;
    r.pages = a.selected ? checked(a, __ldcg(a.n_selected + static_cast<int64_t>(b) * a.hkv + h), a.k_cap, report)
                         : checked(a, __ldcg(a.seq_pages + b), a.max_pages, report);
    r.recent = a.max_recent > 0 ? checked(a, __ldcg(a.recent_tokens + b), static_cast<int64_t>(a.max_recent) * kPage, report) : 0;
    return r;
}
// Steps of all rows of sequence b.
__device__ __forceinline__ int64_t seq_steps(const PackedArgs& a, int b, bool report) {
    if (!a.selected) return static_cast<int64_t>(row_len(a, b, 0, report).steps()) * a.hkv;
    int64_t n = 0;
    for (int h = 0; h < a.hkv; ++h) n += row_len(a, b, h, report).steps();
    return n;
}
// Physical page of a row's packed page i.
__device__ __forceinline__ int packed_id(const PackedArgs& a, int b, int h, int i) {
    int j = i;
    if (a.selected) j = __ldcg(a.selected + (static_cast<int64_t>(b) * a.hkv + h) * a.k_cap + i);
    if (j >= 0 && j < a.max_pages) {
        const int x = __ldcg(a.page_table + static_cast<int64_t>(b) * a.max_pages + j);
        if (x >= 0 && x < a.num_packed) return x;
    }
    report_error(a.st, LOCKS_ERR_BAD_INDEX);
    return 0;
}

// CTA c of n holds steps first(c) .. first(c + 1) of the line.
__device__ __forceinline__ int64_t first_step(int64_t total, int c, int n) {
    const int64_t x = total * c;
    return x < (1ll << 32) ? static_cast<uint32_t>(x) / static_cast<uint32_t>(n) : x / n;
}
__device__ __forceinline__ int cta_of(int64_t total, int64_t step, int n) {
    return static_cast<int>(((step + 1) * n - 1) / total);
}

// The queries of a row as B fragments, in bf16 parts, and what they need beside them.
template <int kKind, bool kSplit>
struct Queries {
    using S = Shape<kKind>;
    static constexpr bool kLow = kSplit && !S::kPair;    // low parts as fragments of their own
    uint32_t hi[S::kBlocks][8][2];
    uint32_t lo[kLow ? S::kBlocks : 1][8][2];
    uint32_t sums[S::kBlocks][2];                     // B fragment of the groups' sums, in three parts
    float unit[S::kBlocks][2];                        // a score's unit, of the accumulators' columns

    __device__ __forceinline__ void load(const PackedArgs& a, int b, int h) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n) {
            const int query = S::kPair ? gid & 3 : n * 8 + gid;
            const bool on = query < a.group;
            const int64_t at = (static_cast<int64_t>(b) * a.hq + h * a.group + (on ? query : 0)) * kD + 2 * tig;
            float2 x[8][2];
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int64_t e = at + 16 * k + 8 * c;
                    if (a.q_type == LOCKS_FP32) {
                        x[k][c] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + e));
                    } else {
                        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + e));
                        x[k][c] = make_float2(low_of(w), high_of(w));
                    }
                    if (!on) x[k][c] = make_float2(0.f, 0.f);
                    big = fmaxf(big, fmaxf(fabsf(x[k][c].x), fabsf(x[k][c].y)));
                }
            big = fmaxf(big, __shfl_xor_sync(kAll, big, 1));
            big = fmaxf(big, __shfl_xor_sync(kAll, big, 2));
            const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -20), 60);
            const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * kQueryShift;
            float sum[4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k % 2 == 0) sum[k / 2] = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float div = c == 0 ? up : up * 0.0625f;        // fields 4 bits up count 16 times
                    const float y0 = x[k][c].x * div, y1 = x[k][c].y * div;
                    uint32_t w = pack_bf16x2(y0, y1);
                    if (kSplit) {
                        const uint32_t v = pack_bf16x2(y0 - low_of(w), y1 - high_of(w));
                        if (S::kPair) w = gid < 4 ? w : v;
                        if (kLow) lo[n][k][c] = v;
                    }
                    hi[n][k][c] = w;
                    float part = low_of(w) + high_of(w);
                    if (kLow) part += low_of(lo[n][k][c]) + high_of(lo[n][k][c]);
                    sum[k / 2] += c == 0 ? part : part * 16.f;
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                sum[g] += __shfl_xor_sync(kAll, sum[g], 1);
                sum[g] += __shfl_xor_sync(kAll, sum[g], 2);
                sum[g] *= 0x1p-66f;                       // by 2^-133, as the codes are
                sum[g] *= 0x1p-67f;
            }
            // rows k = 0..3 of the fragment: the groups' sums to 8 bits; 4..7: the next 8; 8..11
            float s0 = tig & 1 ? sum[2] : sum[0], s1 = tig & 1 ? sum[3] : sum[1];
            const uint32_t w0 = pack_bf16x2(s0, s1);
            s0 -= low_of(w0), s1 -= high_of(w0);
            const uint32_t w1 = pack_bf16x2(s0, s1);
            s0 -= low_of(w1), s1 -= high_of(w1);
            const uint32_t w2 = pack_bf16x2(s0, s1);
            sums[n][0] = tig < 2 ? w0 : w1;
            sums[n][1] = tig < 2 ? w2 : 0u;
            const float back = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (0x1p33f * kScaleLog2);
            unit[n][0] = __shfl_sync(kAll, back, 8 * tig);
            unit[n][1] = __shfl_sync(kAll, back, 8 * tig + 4);
        }
    }
};

// A warp's running softmax over a row: columns 2 * tig + c of each block.
template <int kKind, bool kSplit>
struct Running {
    using S = Shape<kKind>;
    using Q = Queries<kKind, kSplit>;
    float o[S::kBlocks][8][4];                        // O^T of 16 dims each, in units of 2^-93 (dims + 8: 2^-89)
    float m[S::kBlocks][2];                           // maximum, log2
    float l[S::kBlocks][2];                           // this lane's part of the sum, times 2^40
    float z[S::kBlocks][2][2];                        // [group]: of weights times zeros

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n) {
#pragma unroll
            for (int d = 0; d < 8; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) m[n][c] = -INFINITY, l[n][c] = 0.f, z[n][0][c] = z[n][1][c] = 0.f;
        }
    }

    // Scores (tokens gid, gid + 8) to weights times 2^40. The maximum moves only when a score
    // passes it by more than kSlack: weights and sums are floating-point numbers, so the slack
    // costs no bits, and most pages pass with one vote.
    __device__ __forceinline__ void weigh(float (&s)[S::kBlocks][4], const Q& q) {
        bool over = false;
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] *= q.unit[n][i & 1];
                over |= s[n][i] > m[n][i & 1] + kSlack;
            }
        if (__any_sync(kAll, over)) {
#pragma unroll
            for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
                    top = fmaxf(top, m[n][c]);
                    const float f = m[n][c] == -INFINITY ? 0.f : fast_exp2(m[n][c] - top);
                    m[n][c] = top;
                    l[n][c] *= f;
                    z[n][0][c] *= f;
                    z[n][1][c] *= f;
#pragma unroll
                    for (int d = 0; d < 8; ++d) o[n][d][c] *= f, o[n][d][c + 2] *= f;
                }
        }
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float base = m[n][c] == -INFINITY ? kWeightBits : kWeightBits - m[n][c];
                s[n][c] = fast_exp2(s[n][c] + base);
                s[n][c + 2] = fast_exp2(s[n][c + 2] + base);
                l[n][c] += s[n][c] + s[n][c + 2];
            }
    }

    // Weights as B fragments, tokens as rows: a high and a low part, in columns of their own
    // (kPair) or apart. The high part is cut off rather than rounded, the low part of kPair
    // too: what is left out is less than 2^-14 of a weight (2^-15 where the low part is rounded).
    __device__ __forceinline__ static void parts(const float (&p)[4], uint32_t (&hi)[2], uint32_t (&lo)[2]) {
        const uint32_t low_columns = S::kPair && (threadIdx.x & 2) ? 0xffff0000u : 0u;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t a = __float_as_uint(p[2 * t]), b = __float_as_uint(p[2 * t + 1]);
            if (S::kPair) {
                const float x = p[2 * t] - __uint_as_float(a & low_columns);
                const float y = p[2 * t + 1] - __uint_as_float(b & low_columns);
                hi[t] = movmatrix_trans(prmt(__float_as_uint(x), __float_as_uint(y), 0x7632u));
            } else {
                const uint32_t w = prmt(a, b, 0x7632u);
                hi[t] = movmatrix_trans(w);
                lo[t] = movmatrix_trans(pack_bf16x2(p[2 * t] - low_of(w), p[2 * t + 1] - high_of(w)));
            }
        }
    }

    __device__ __forceinline__ void packed_page(const uint8_t* unit, const Q& q) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
        float s[S::kBlocks][4];
        {
            const uint4 k0 = *reinterpret_cast<const uint4*>(unit + 16 * lane);
            const uint4 k1 = *reinterpret_cast<const uint4*>(unit + 512 + 16 * lane);
            const uint4 t0 = *reinterpret_cast<const uint4*>(unit + kUnitKScales + 16 * gid);
            const uint4 t1 = *reinterpret_cast<const uint4*>(unit + kUnitKScales + 16 * (gid + 8));
            const uint32_t z0 = tig & 1 ? t0.w : t0.z, z1 = tig & 1 ? t1.w : t1.z;
            const uint32_t zeros[4] = {z0, z1, z0, z1};
#pragma unroll
            for (int n = 0; n < S::kBlocks; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                mma_bf16_16816(s[n], zeros, q.sums[n][0], q.sums[n][1]);
            }
            const uint32_t w[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
            const uint32_t scale0[2] = {t0.x, t0.y}, scale1[2] = {t1.x, t1.y};
#pragma unroll
            for (int g = 0; g < 4; ++g) {             // 32 dims
                float acc[S::kBlocks][4];
#pragma unroll
                for (int n = 0; n < S::kBlocks; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 2 * g + i;
                    const uint32_t up = w[k] >> 8;
                    const uint32_t f[4] = {w[k] & 0x000f000fu, up & 0x000f000fu, w[k] & 0x00f000f0u, up & 0x00f000f0u};
#pragma unroll
                    for (int n = 0; n < S::kBlocks; ++n) {
                        mma_bf16_16816(acc[n], f, q.hi[n][k][0], q.hi[n][k][1]);
                        if (Q::kLow) mma_bf16_16816(acc[n], f, q.lo[n][k][0], q.lo[n][k][1]);
                    }
                }
                const float a0 = g & 1 ? high_of(scale0[g >> 1]) : low_of(scale0[g >> 1]);
                const float a1 = g & 1 ? high_of(scale1[g >> 1]) : low_of(scale1[g >> 1]);
#pragma unroll
                for (int n = 0; n < S::kBlocks; ++n) {
                    s[n][0] = fmaf(a0, acc[n][0], s[n][0]);
                    s[n][1] = fmaf(a0, acc[n][1], s[n][1]);
                    s[n][2] = fmaf(a1, acc[n][2], s[n][2]);
                    s[n][3] = fmaf(a1, acc[n][3], s[n][3]);
                }
            }
        }
        add_low(s);
        weigh(s, q);
        const uint4 v0 = *reinterpret_cast<const uint4*>(unit + kUnitVCodes + 16 * lane);
        const uint4 v1 = *reinterpret_cast<const uint4*>(unit + kUnitVCodes + 512 + 16 * lane);
        const uint2 t0 = *reinterpret_cast<const uint2*>(unit + kUnitVScales + 8 * gid);
        const uint2 t1 = *reinterpret_cast<const uint2*>(unit + kUnitVScales + 8 * (gid + 8));
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int g = 0; g < 2; ++g) {                 // 64 dims
            const float a0 = g ? high_of(t0.x) : low_of(t0.x), a1 = g ? high_of(t1.x) : low_of(t1.x);
            const float z0 = g ? high_of(t0.y) : low_of(t0.y), z1 = g ? high_of(t1.y) : low_of(t1.y);
            uint32_t hi[S::kBlocks][2], lo[S::kBlocks][2];
#pragma unroll
            for (int n = 0; n < S::kBlocks; ++n) {
                const float p[4] = {s[n][0] * a0, s[n][1] * a0, s[n][2] * a1, s[n][3] * a1};
                z[n][g][0] = fmaf(s[n][0], z0, fmaf(s[n][2], z1, z[n][g][0]));
                z[n][g][1] = fmaf(s[n][1], z0, fmaf(s[n][3], z1, z[n][g][1]));
                parts(p, hi[n], lo[n]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 4 * g + i;
                const uint32_t up = w[d] >> 8;
                const uint32_t f[4] = {w[d] & 0x000f000fu, w[d] & 0x00f000f0u, up & 0x000f000fu, up & 0x00f000f0u};
#pragma unroll
                for (int n = 0; n < S::kBlocks; ++n) {
                    mma_bf16_16816(o[n][d], f, hi[n][0], hi[n][1]);
                    if (!S::kPair) mma_bf16_16816(o[n][d], f, lo[n][0], lo[n][1]);
                }
            }
        }
    }

    // A bf16 page in shared memory, K and then V, rows of 256 bytes swizzled by 16-byte chunks
    // (chunk_offset), zero from row `valid` on.
    __device__ __forceinline__ void recent_page(const uint8_t* page, int valid, const Q& q) {
        const int lane = threadIdx.x & 31, gid = lane >> 2;
        const uint32_t down = 0x21802180u, down16 = 0x23802380u;         // 2^-60, 2^-56: exponents 67, 71
        float s[S::kBlocks][4];
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t f[4];
            ldmatrix_x4(f, page + chunk_offset(lane & 15, 2 * k + (lane >> 4)));
            f[0] = bf16x2_mul(f[0], down), f[1] = bf16x2_mul(f[1], down);
            f[2] = bf16x2_mul(f[2], down16), f[3] = bf16x2_mul(f[3], down16);
#pragma unroll
            for (int n = 0; n < S::kBlocks; ++n) {
                mma_bf16_16816(s[n], f, q.hi[n][k][0], q.hi[n][k][1]);
                if (Q::kLow) mma_bf16_16816(s[n], f, q.lo[n][k][0], q.lo[n][k][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] *= kRecentScore;
        add_low(s);
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (gid + 8 * (i >> 1) >= valid) s[n][i] = -INFINITY;
        weigh(s, q);
        uint32_t hi[S::kBlocks][2], lo[S::kBlocks][2];
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] *= kRecentWeight;
            parts(s[n], hi[n], lo[n]);
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            // rows of the fragment are dims: a0 (dims, tokens), a1 (dims + 8, tokens), a2 (dims, tokens + 8), a3
            uint32_t f[4];
            ldmatrix_x4_trans(f, page + kPage * kD * 2 +
                                     chunk_offset((lane & 7) + 8 * (lane >> 4), 2 * d + (lane >> 3 & 1)));
            f[1] = bf16x2_mul(f[1], 0x41804180u), f[3] = bf16x2_mul(f[3], 0x41804180u);      // 16
#pragma unroll
            for (int n = 0; n < S::kBlocks; ++n) {
                mma_bf16_16816(o[n][d], f, hi[n][0], hi[n][1]);
                if (!S::kPair) mma_bf16_16816(o[n][d], f, lo[n][0], lo[n][1]);
            }
        }
    }

    // Low parts of the queries in columns of their own (bf16 queries fill those with copies).
    __device__ __forceinline__ static void add_low(float (&s)[S::kBlocks][4]) {
        if (S::kPair && kSplit) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][i] += __shfl_xor_sync(kAll, s[0][i], 2);
        }
    }
    __device__ __forceinline__ static int chunk_offset(int token, int c) { return token * kD * 2 + ((c ^ (token & 7)) << 4); }

    // The row's sums and unnormalised output, from all lanes: f(query, dim, value) for every
    // query of the group, with m (log2) and l of each query by g(query, m, l).
    template <typename F, typename G>
    __device__ __forceinline__ void finish(int group, F f, G g) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int n = 0; n < S::kBlocks; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x *= 2) {
                    l[n][c] += __shfl_xor_sync(kAll, l[n][c], x);
                    z[n][0][c] += __shfl_xor_sync(kAll, z[n][0][c], x);
                    z[n][1][c] += __shfl_xor_sync(kAll, z[n][1][c], x);
                }
                const int query = S::kPair ? 2 * (tig & 1) + c : n * 8 + 2 * tig + c;
                const bool on = query < group && !(S::kPair && tig >= 2);
                const float sum = l[n][c] * kSumUnit;
                if (on && gid == 0) g(query, m[n][c], sum);
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    float x0 = o[n][d][c], x1 = o[n][d][c + 2];
                    if (S::kPair) x0 += __shfl_xor_sync(kAll, x0, 2), x1 += __shfl_xor_sync(kAll, x1, 2);
                    const float zero = z[n][d / 4][c] * kSumUnit;
                    if (on) {
                        f(query, d * 16 + gid, fmaf(x0, kOutUnit, zero), sum);
                        f(query, d * 16 + gid + 8, fmaf(x1, kOutUnit * 0.0625f, zero), sum);
                    }
                }
            }
    }
};

__device__ __forceinline__ void store_row(const PackedArgs& a, int64_t row, float value, float sum, int dim) {
    a.out[row * kD + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : value / sum));
}
__device__ __forceinline__ void store_lse(const PackedArgs& a, int64_t row, float m, float sum) {
    if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
}

template <int kKind, bool kSplit>
__global__ void __launch_bounds__(Shape<kKind>::kWarps * 32, Shape<kKind>::kCtas)
    attend_kernel(const __grid_constant__ PackedArgs a) {
    using S = Shape<kKind>;
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32, kDepth = S::kDepth;
    static_assert(kDepth * kUnitBytes >= 4 * kPage * kD, "a recent page lies in the slots");
    static_assert(kDepth * kUnitBytes >= kPartBytes<S::kRows>, "a partial lies in the slots");
    extern __shared__ __align__(128) uint8_t slots[];
    __shared__ Control<kWarps, S::kRows> ctl;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* const mine = slots + warp * kDepth * kUnitBytes;
    // partials: a warp's first row beside the slots, its last row in its slots
    const auto part = [&](int e) {
        return reinterpret_cast<float*>(e & 1 ? slots + (e >> 1) * kDepth * kUnitBytes
                                              : slots + kWarps * kDepth * kUnitBytes + (e >> 1) * kPartBytes<S::kRows>);
    };
    grid_dependency_wait();
    allow_dependent_launch();

    // the line of steps
    const int per = (a.batch + kThreads - 1) / kThreads;
    {
        int64_t sum = 0;
        for (int i = 0; i < per; ++i) {
            const int b = threadIdx.x * per + i;
            if (b < a.batch) sum += seq_steps(a, b, blockIdx.x == 0);
        }
        int64_t upto = sum;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
            const int64_t y = __shfl_up_sync(kAll, upto, x);
            if (lane >= x) upto += y;
        }
        if (lane == 31) ctl.warp_sum[warp] = upto;
        if (threadIdx.x < kWarps * 2) ctl.entry[threadIdx.x].row = -1;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += ctl.warp_sum[w];
        ctl.upto[threadIdx.x] = upto;
    }
    // rows without tokens are nobody's
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < static_cast<int64_t>(a.batch) * a.hkv;
         r += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int b = static_cast<int>(r / a.hkv), h = static_cast<int>(r % a.hkv);
        if (row_len(a, b, h, false).steps() != 0) continue;
        for (int q = 0; q < a.group; ++q) {
            const int64_t row = static_cast<int64_t>(b) * a.hq + h * a.group + q;
            for (int d = 0; d < kD; d += 8) *reinterpret_cast<uint4*>(a.out + row * kD + d) = make_uint4(0, 0, 0, 0);
            store_lse(a, row, 0.f, 0.f);
        }
    }
    __syncthreads();
    const int64_t total = ctl.upto[kThreads - 1];
    const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kWarps - 1) / kWarps));
    const int64_t cta0 = ctas > 0 ? first_step(total, blockIdx.x, ctas) : 0;
    const int64_t cta1 = static_cast<int>(blockIdx.x) < ctas ? first_step(total, blockIdx.x + 1, ctas) : cta0;
    int64_t pos = cta0 + (cta1 - cta0) * warp / kWarps;
    const int64_t end = cta0 + (cta1 - cta0) * (warp + 1) / kWarps;

    if (pos < end) {
        // the row at pos
        int b = 0, h = 0, off = 0;
        Len len;
        {
            int before = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) before += __popc(__ballot_sync(kAll, ctl.upto[i * 32 + lane] <= pos));
            int64_t at = pos - (before > 0 ? ctl.upto[before - 1] : 0);
            b = before * per;
            for (int64_t n; b < a.batch - 1 && at >= (n = seq_steps(a, b, false)); ++b) at -= n;
            for (len = row_len(a, b, 0, false); h < a.hkv - 1 && at >= len.steps(); len = row_len(a, b, ++h, false))
                at -= len.steps();
            off = static_cast<int>(at);
        }
        Queries<kKind, kSplit> q;
        Running<kKind, kSplit> run;
        for (bool first = true; pos < end; first = false) {
            const int steps = len.steps();
            const int n = static_cast<int>(min(end - pos, static_cast<int64_t>(steps - off)));
            // packed pages off .. off + count
            const int count = max(0, min(off + n, len.pages) - off);
            const int64_t unit0 = static_cast<int64_t>(h) * kUnitBytes, page_bytes = static_cast<int64_t>(a.hkv) * kUnitBytes;
            int ids = lane < count ? packed_id(a, b, h, off + lane) : 0, next = 0;
            const auto load = [&](int i, int slot) {
                if ((i & 31) == 0) {                  // ids of 32 pages, fetched 32 pages ahead
                    if (i > 0) ids = next;
                    if (i + 32 + lane < count) next = packed_id(a, b, h, off + i + 32 + lane);
                }
                const uint8_t* from = a.packed + __shfl_sync(kAll, ids, i & 31) * page_bytes + unit0 + lane * 16;
                uint8_t* to = mine + slot * kUnitBytes + lane * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) cp_async_16(to + j * 512, from + j * 512);
                if (lane < kUnitBytes / 16 - 128) cp_async_16(to + 2048, from + 2048);
            };
#pragma unroll
            for (int i = 0; i < kDepth - 1; ++i) {
                if (i < count) load(i, i);
                copies_commit();
            }
            q.load(a, b, h);
            run.clear();
            int slot = 0;
#pragma unroll 1
            for (int i = 0; i < count; ++i) {
                copies_wait<kDepth - 2>();
                __syncwarp();                         // everyone's copies are there, and the slot ahead is read
                if (i + kDepth - 1 < count) load(i + kDepth - 1, slot == 0 ? kDepth - 1 : slot - 1);
                copies_commit();
                run.packed_page(mine + slot * kUnitBytes, q);
                if (++slot == kDepth) slot = 0;
            }
            copies_wait<0>();
            __syncwarp();
            // recent pages whose first step is among this part's
            const int r0 = max(0, (off - len.pages + kRecentSteps - 1) / kRecentSteps);
            const int r1 = min(len.recent_pages(), (off + n - len.pages + kRecentSteps - 1) / kRecentSteps);
#pragma unroll 1
            for (int r = r0; r < r1; ++r) {
                const int valid = min(kPage, len.recent - r * kPage);
                int id = __ldcg(a.recent_table + static_cast<int64_t>(b) * a.max_recent + r);
                if (id < 0 || id >= a.num_cache) {
                    report_error(a.st, LOCKS_ERR_BAD_INDEX);
                    id = 0;
                }
                const int64_t from = (static_cast<int64_t>(id) * a.hkv + h) * (kPage * kD) + lane * 8;
#pragma unroll
                for (int j = 0; j < kPage / 2; ++j) {  // two tokens
                    const int token = 2 * j + (lane >> 4), to = run.chunk_offset(token, lane & 15);
                    copy_or_zero(mine + to, a.k_cache + from + j * 2 * kD, token < valid);
                    copy_or_zero(mine + kPage * kD * 2 + to, a.v_cache + from + j * 2 * kD, token < valid);
                }
                copies_commit();
                copies_wait<0>();
                __syncwarp();
                run.recent_page(mine, valid, q);
                __syncwarp();
            }
            const bool begins = off == 0, ends = off + n == steps;
            if (begins && ends) {
                const int64_t row = static_cast<int64_t>(b) * a.hq + h * a.group;
                run.finish(
                    a.group, [&](int query, int dim, float x, float sum) { store_row(a, row + query, x, sum, dim); },
                    [&](int query, float m, float sum) { store_lse(a, row + query, m, sum); });
            } else {
                const int e = warp * 2 + (first ? 0 : 1);
                float* o = part(e);
                run.finish(
                    a.group, [&](int query, int dim, float x, float) { o[query * kPartStride + dim] = x; },
                    [&](int query, float m, float sum) { ctl.m[e][query] = m, ctl.l[e][query] = sum; });
                if (lane == 0) {
                    auto& entry = ctl.entry[e];
                    entry.step0 = pos - off;
                    entry.row = b * a.hkv + h;
                    entry.len = steps;
                    entry.begins = begins;
                    entry.ends = ends;
                }
            }
            pos += n;
            off = 0;
            if (pos < end) {
                do {
                    if (++h == a.hkv) ++b, h = 0;
                    len = row_len(a, b, h, false);
                } while (len.steps() == 0 && b < a.batch - 1);
            }
        }
    }

    // rows that lie in several warps
    __syncthreads();
    int owned = -1, last = 0;                         // the row that goes on behind this CTA
    for (int e = 0; e < kWarps * 2;) {
        if (ctl.entry[e].row < 0) {
            ++e;
            continue;
        }
        const auto head = ctl.entry[e];
        int stop = e;
        bool ends = false;
        for (int f = e; f < kWarps * 2; ++f) {
            if (ctl.entry[f].row < 0) continue;
            if (ctl.entry[f].row != head.row) break;
            stop = f;
            ends = ctl.entry[f].ends;
        }
        const bool whole = head.begins && ends;
        if (head.begins && !ends) owned = head.row, last = cta_of(total, head.step0 + head.len - 1, ctas);
        const int64_t row = static_cast<int64_t>(head.row / a.hkv) * a.hq + (head.row % a.hkv) * a.group;
        const int slot = 2 * blockIdx.x + (head.begins ? 1 : 0);
        for (int i = threadIdx.x; i < a.group * kD; i += kThreads) {
            const int query = i / kD, dim = i % kD;
            float top = -INFINITY;
            for (int f = e; f <= stop; ++f)
                if (ctl.entry[f].row >= 0) top = fmaxf(top, ctl.m[f][query]);
            const float base = top == -INFINITY ? 0.f : top;
            float x = 0.f, sum = 0.f;
            for (int f = e; f <= stop; ++f)
                if (ctl.entry[f].row >= 0) {
                    const float w = fast_exp2(ctl.m[f][query] - base);
                    x = fmaf(w, part(f)[query * kPartStride + dim], x);
                    sum = fmaf(w, ctl.l[f][query], sum);
                }
            if (whole) {
                store_row(a, row + query, x, sum, dim);
                if (dim == 0) store_lse(a, row + query, top, sum);
            } else {
                a.part_o[(static_cast<int64_t>(slot) * a.group + query) * kD + dim] = x;
                if (dim == 0) a.part_ml[slot * a.group + query] = make_float2(top, sum);
            }
        }
        e = stop + 1;
    }
    if (threadIdx.x == 0) {
        a.cuts[blockIdx.x].row = owned;
        a.cuts[blockIdx.x].last = last;
    }
}

// Joins the rows that lie in several CTAs: a block per (CTA that a row begins in, query).
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ PackedArgs a) {
    __shared__ float weight[kMaxPackedCtas], sums[kJoinThreads / 32], tops[kJoinThreads / 32], acc[kJoinThreads];
    const int c = blockIdx.x / a.group, query = blockIdx.x % a.group, tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    const PackedCut cut = a.cuts[c];
    if (cut.row < 0) return;
    const int n = cut.last - c + 1;                   // up to kMaxPackedCtas <= kJoinThreads
    const auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < n) ml = a.part_ml[slot(tid) * a.group + query];
    float top = ml.x;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
    if (tid % 32 == 0) tops[tid / 32] = top;
    __syncthreads();
    for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, tops[i]);
    const float w = tid < n ? fast_exp2(ml.x - (top == -INFINITY ? 0.f : top)) : 0.f;
    weight[tid] = w;
    float sum = tid < n ? w * ml.y : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(kAll, sum, x);
    if (tid % 32 == 0) sums[tid / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < kJoinThreads / 32; ++i) sum += sums[i];
    const int dim = tid % kD;
    float x = 0.f;
#pragma unroll 8
    for (int i = tid / kD; i < n; i += kJoinThreads / kD)
        x = fmaf(weight[i], a.part_o[(static_cast<int64_t>(slot(i)) * a.group + query) * kD + dim], x);
    acc[tid] = x;
    __syncthreads();
    if (tid < kD) {
        for (int i = 1; i < kJoinThreads / kD; ++i) x += acc[i * kD + tid];
        const int64_t row = static_cast<int64_t>(cut.row / a.hkv) * a.hq + (cut.row % a.hkv) * a.group + query;
        store_row(a, row, x, sum, dim);
        if (tid == 0) store_lse(a, row, top, sum);
    }
}
static_assert(kMaxPackedCtas <= kJoinThreads, "a thread per partial");

template <int kKind, bool kSplit>
cudaError_t launch_t(const PackedArgs& a, int num_sms, cudaStream_t stream) {
    using S = Shape<kKind>;
    constexpr int kSmem = S::kWarps * (S::kDepth * kUnitBytes + kPartBytes<S::kRows>);
    cudaError_t e = ensure_kernel_attrs<attend_kernel<kKind, kSplit>>(kSmem);
    if (e != cudaSuccess) return e;
    // no more CTAs than the longest lists have steps for
    const int64_t steps = static_cast<int64_t>(a.batch) * a.hkv *
                          ((a.selected ? a.k_cap : a.max_pages) + static_cast<int64_t>(kRecentSteps) * a.max_recent);
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(std::min(num_sms * S::kCtas, kMaxPackedCtas),
                                                                (steps + S::kWarps - 1) / S::kWarps));
    e = launch_dependent(attend_kernel<kKind, kSplit>, ctas, S::kWarps * 32, kSmem, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel, ctas * a.group, kJoinThreads, 0, stream, 1, a);
}

}  // namespace

PackedLayout packed_layout(int group) {
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = 2 * static_cast<size_t>(kMaxPackedCtas) * group;
    PackedLayout w;
    w.ml = 256 + up(kMaxPackedCtas * sizeof(PackedCut));
    w.o = w.ml + up(rows * sizeof(float2));
    w.bytes = w.o + up(rows * kD * sizeof(float));
    return w;
}

cudaError_t launch_packed_attention(const PackedArgs& a, int num_sms, cudaStream_t stream) {
    const auto by_type = [&](auto kind) {
        constexpr int kKind = decltype(kind)::value;
        return a.q_type == LOCKS_FP32 ? launch_t<kKind, true>(a, num_sms, stream) : launch_t<kKind, false>(a, num_sms, stream);
    };
    if (a.group <= 4) return by_type(std::integral_constant<int, 0>());
    if (a.group <= 8) return by_type(std::integral_constant<int, 1>());
    return by_type(std::integral_constant<int, 2>());
}

}  // namespace locks
