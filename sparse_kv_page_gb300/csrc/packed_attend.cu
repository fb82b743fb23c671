// packed_attend.cu - decode attention over packed pages (locks_packed_attention).
//
// A CTA takes a part of a row (a sequence and a kv head), or of two neighbouring rows, its warps an
// equal share each, two pages at a time with an online softmax; the warps' partials meet in shared
// memory. Two forms cut the rows into parts (8 kv heads of 4 queries unless said):
//
// 1. Short rows: a cluster of 1 to 8 CTAs a row, joined through distributed shared memory, in one
//    launch. Latency bounds it: 8.0 us for two sequences of 347 tokens, 12.8 for 2048 selected
//    tokens of eight sequences.
// 2. Long rows: all steps of the call, a page of a kv head each (a recent bf16 page counts
//    kRecentSteps), lie on one line, row after row, that is cut evenly into as many CTAs as there
//    are SMs, whatever the lengths of the rows. A CTA goes through its piece two rows at a time, so
//    that where rows are long its warps meet once, at the end. A row that goes past a CTA is joined
//    by a second kernel from partials in the workspace. Sixteen sequences of up to 128K tokens take
//    360 us, 95% of the copy rate; two of 1M with 2 kv heads of 16 queries 196 us, 45%: there a
//    page takes a warp 50 products and 454 instructions (299 for 4 queries), at three warps a
//    scheduler.
//
// The products are formed on mma.sync with the queries as columns, S^T = K Q^T and
// O^T = V^T P^T: few queries read a page, so HBM bounds the call as long as a page costs a warp
// few instructions. The codes lie in the pages in the order of the A fragments, so that a lane
// loads its fragments with four 16-byte loads, and a pair of codes becomes a pair of fp16
// values by one AND: a 4-bit field in the low bits of an fp16 is the subnormal number field *
// 2^-24, exactly. Fields 4 bits further up count 16 times as much; the queries' side is divided
// by 16 there, for values the output. Queries and weights are scaled by powers of two into fp16's
// range. A token's scales multiply the group's sums (keys) or the weights (values); zeros enter
// through a product of their own with the queries' sums (keys) and through a sum per group
// (values). Where values' scales are so far apart that one power of two does not bring them all
// into fp16's range, the weights enter in two bf16 parts (the same fields are subnormals of 2^-133
// there).
#include <algorithm>
#include <atomic>

#include "packed_units.cuh"

namespace locks {
namespace {

constexpr int kCentre = 8;                            // pairs of pages, a power of two
constexpr float kAhead = 0.625f;

// Variants: queries of a group in one block of 8 columns together with their low parts (kPair,
// groups up to 4; bf16 queries have none and fill those columns with copies), in one block, or in
// two. 16 warps of 128 registers, or 12 of 168 for the accumulators of two blocks; kDepth pages of
// each warp are in shared memory or on their way.
template <int kKind>
struct Shape {
    static constexpr bool kPair = kKind == 0;
    static constexpr int kBlocks = kKind == 2 ? 2 : 1, kRows = kPair ? 4 : 8 * kBlocks;
    static constexpr int kWarps = kKind == 2 ? 12 : 16, kDepth = kKind == 2 ? 6 : 5;
    static constexpr int kThreads = kWarps * 32;
};
constexpr int kMaxCluster = 8;
constexpr int kPartStride = kD + 4;                   // floats: columns' stores in different banks

// Shared memory of a CTA besides the slots.
template <int kKind>
struct Control {
    using S = Shape<kKind>;
    uint4 frag[2][S::kBlocks][8][32];                 // of both rows: B fragments of the queries: high parts, low parts
    uint2 sums[2][S::kBlocks][32];                    // ... of the groups' sums
    float unit[2][S::kBlocks * 8];                    // a score's unit, by column
    // the warps' partials: which rows a warp had some of (bits), m and l; its output lies in its
    // slots, or for the warp that had both rows that of the first in `both`
    int32_t had[S::kWarps];
    float m[2][S::kWarps][S::kRows], l[2][S::kWarps][S::kRows];
    float factor[2][S::kWarps][S::kRows];             // of the warps' partials when they are joined
    float top[2][S::kRows], sum[2][S::kRows];         // the CTA's m and l
    float both[S::kRows * kPartStride];
    union {
        struct {                                      // short rows: the CTA's partial
            float o[S::kRows][kD];
        } cta;
        LineShared<S::kThreads> line;                 // long rows
    };
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
// D = A B + D and D = A B on mma.sync m16n8k16. Not volatile, as nothing but the operands counts:
// the compiler may move products past one another, which saves it register copies.
#define LOCKS_MMA(name, type)                                                                                        \
    __device__ __forceinline__ void name(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {          \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "    \
            "{%0,%1,%2,%3};"                                                                                         \
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                         \
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));                                         \
    }                                                                                                                \
    __device__ __forceinline__ void name##_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "    \
            "{%10,%10,%10,%10};"                                                                                     \
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                         \
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));                               \
    }
LOCKS_MMA(mma_f16, "f16")
LOCKS_MMA(mma_bf16, "bf16")
#undef LOCKS_MMA
__device__ __forceinline__ uint32_t transposed(uint32_t x) {          // of 8 x 8 16-bit elements
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Dims 32 g .. 32 g + 31 of one block of a row's queries as B fragments, in fp16 parts (fp32 queries
// keep 22 bits), by one warp.
template <int kKind, bool kSplit>
__device__ __forceinline__ void put_queries(const PackedArgs& a, int b, int h, int which, int block, int g, Control<kKind>& ctl) {
    using S = Shape<kKind>;
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int query = S::kPair ? gid & 3 : block * 8 + gid;
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
    const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * kQueryTop;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k / 2 != g) continue;
        uint32_t hi[2], lo[2] = {0u, 0u};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float by = c == 0 ? up : up * 0.0625f;          // fields 4 bits up count 16 times
            const float y0 = x[k][c].x * by, y1 = x[k][c].y * by;
            hi[c] = pack_f16x2(y0, y1);
            const float2 x0 = f16x2_of(hi[c]);
            if (kSplit) {
                lo[c] = pack_f16x2(y0 - x0.x, y1 - x0.y);
                if (S::kPair) {                                   // columns 4..7 are the low parts
                    if (gid >= 4) hi[c] = lo[c];
                    lo[c] = 0u;
                }
            }
            const float2 x1 = f16x2_of(hi[c]), x2 = f16x2_of(lo[c]);
            const float part = x1.x + x1.y + (x2.x + x2.y);
            sum += c == 0 ? part : part * 16.f;
        }
        ctl.frag[which][block][k][lane] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
    }
    sum += __shfl_xor_sync(kAll, sum, 1);
    sum += __shfl_xor_sync(kAll, sum, 2);
    sum *= kCode;
    // the sum's fragment: rows k = g, 4 + g and 8 + g are its first 8 bits, the next 8, and the next
    if (tig < 3) {
        const float s0 = __bfloat162float(__float2bfloat16_rn(sum)), s1 = __bfloat162float(__float2bfloat16_rn(sum - s0));
        const float mine = tig == 0 ? s0 : tig == 1 ? s1 : sum - s0 - s1;
        const int k = 4 * tig + g;                    // of lane 4 gid + k % 8 / 2, half k % 2, register k / 8
        reinterpret_cast<uint16_t*>(&ctl.sums[which][block][4 * gid + k % 8 / 2])[2 * (k / 8) + k % 2] =
            __bfloat16_as_ushort(__float2bfloat16_rn(mine));
    } else {                                          // rows 12 .. 15 are zero
        const int k = 12 + g;
        reinterpret_cast<uint16_t*>(&ctl.sums[which][block][4 * gid + k % 8 / 2])[2 * (k / 8) + k % 2] = 0;
    }
    if (tig == 0 && g == 0)
        ctl.unit[which][block * 8 + gid] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * kScoreUnit;
}
// ... of all blocks and dims of the CTA's rows, by its first warps.
template <int kKind, bool kSplit>
__device__ __forceinline__ void put_all_queries(const PackedArgs& a, int b0, int h0, int b1, int h1, int rows, Control<kKind>& ctl) {
    using S = Shape<kKind>;
    for (int i = threadIdx.x >> 5; i < rows * S::kBlocks * 4; i += S::kWarps) {
        const int which = i / (S::kBlocks * 4);
        put_queries<kKind, kSplit>(a, which ? b1 : b0, which ? h1 : h0, which, i / 4 % S::kBlocks, i % 4, ctl);
    }
}

// A warp's running softmax over a part of a row: columns 2 * tig + c of each block.
template <int kKind, bool kSplit>
struct Running {
    using S = Shape<kKind>;
    static constexpr int kBlocks = S::kBlocks;
    static constexpr bool kLow = kSplit && !S::kPair; // low parts as fragments of their own
    float o[kBlocks][8][4];                           // O^T of 16 dims each, in units of 2^-24 (dims + 8: 2^-20)
    float m[kBlocks][2];                              // maximum, log2
    Two unit[kBlocks];
    Two l[kBlocks];                                   // this lane's part of the sum
    Two z[kBlocks][2];                                // [column], of both groups: of weights times zeros
    Two pw[kBlocks][2];                               // [group], of both columns: of weights times scales, as the
                                                      // products take them, since the last centre()
    float lift;                                       // log2 of the weights' factor
    uint32_t limit;                                   // the largest scale that it is good for, as two bf16s

    __device__ __forceinline__ void clear(const Control<kKind>& ctl, int which) {
        const int tig = threadIdx.x & 3;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
#pragma unroll
            for (int d = 0; d < 8; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) m[n][c] = -INFINITY, z[n][c] = pw[n][c] = two(0.f, 0.f);
            unit[n] = two(ctl.unit[which][n * 8 + 2 * tig], ctl.unit[which][n * 8 + 2 * tig + 1]);
            l[n] = two(0.f, 0.f);
        }
        lift = 0.f;                                   // until a scale is not 0: limit 2^-116, low 0
        limit = kLimits;
    }

    // Scores (tokens gid, gid + 8 of kPages pages) to weights. The maximum moves only when a score
    // passes it by more than kSlack, the factor when a scale passes its limit: weights and sums are
    // floating-point numbers, so the slack costs no bits, and most pages pass with one vote. `most` and
    // `least` are this lane's extreme scales, two bf16s each; `rest` is called, ahead of the weights, where
    // one is too small for the factor, or below 0.
    template <int kPages, typename Rest>
    __device__ __forceinline__ void weigh(float (&s)[kPages][kBlocks][4], uint32_t most, uint32_t least, Rest rest) {
        bool over = any_greater(most, limit) || any_less(least, low());
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
            const float limit0 = m[n][0] + kSlack, limit1 = m[n][1] + kSlack;
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int p = 0; p < kPages; ++p) {
                parts_of(mul2(two(s[p][n][0], s[p][n][1]), unit[n]), s[p][n][0], s[p][n][1]);
                parts_of(mul2(two(s[p][n][2], s[p][n][3]), unit[n]), s[p][n][2], s[p][n][3]);
                top0 = fmaxf(top0, fmaxf(s[p][n][0], s[p][n][2]));
                top1 = fmaxf(top1, fmaxf(s[p][n][1], s[p][n][3]));
            }
            over |= top0 > limit0 || top1 > limit1;
        }
        if (__any_sync(kAll, over)) {
            float change = 0.f;                       // log2
            float scale = fmaxf(fmaxf(low_of(most), high_of(most)), -fminf(low_of(least), high_of(least)));
#pragma unroll
            for (int x = 1; x < 32; x *= 2) scale = fmaxf(scale, __shfl_xor_sync(kAll, scale, x));
            if (scale > low_of(limit)) {              // kScaleTop - exponent, within -100..54 (see kScaleLeast)
                const int e = kScaleTop - min(max(static_cast<int>(__float_as_uint(scale) >> 23) - 127, kScaleLeast), 105);
                change = static_cast<float>(e) - lift;
                lift += change;
                limit = static_cast<uint32_t>(127 + kScaleLimit - e) * 0x00800080u;
            }
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = m[n][c];
#pragma unroll
                    for (int p = 0; p < kPages; ++p) top = fmaxf(top, fmaxf(s[p][n][c], s[p][n][c + 2]));
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
                    f[c] = m[n][c] == -INFINITY ? 0.f : fast_exp2(m[n][c] - top + change);
                    m[n][c] = top;
                    z[n][c] = mul2(z[n][c], two(f[c], f[c]));
                }
                const Two both = two(f[0], f[1]);
                l[n] = mul2(l[n], both);
                pw[n][0] = mul2(pw[n][0], both);
                pw[n][1] = mul2(pw[n][1], both);
#pragma unroll
                for (int d = 0; d < 8; ++d) o[n][d][0] *= f[0], o[n][d][1] *= f[1], o[n][d][2] *= f[0], o[n][d][3] *= f[1];
            }
            if (__any_sync(kAll, any_less(least, low()))) rest();
        }
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
            const Two by = base(n);
#pragma unroll
            for (int p = 0; p < kPages; ++p) {
#pragma unroll
                for (int t = 0; t < 4; t += 2) {
                    float x, y;
                    parts_of(add2(two(s[p][n][t], s[p][n][t + 1]), by), x, y);
                    s[p][n][t] = fast_exp2(x);
                    s[p][n][t + 1] = fast_exp2(y);
                    l[n] = add2(l[n], two(s[p][n][t], s[p][n][t + 1]));
                }
            }
        }
    }
    // The least scale that the factor is good for.
    static constexpr uint32_t kLimits = static_cast<uint32_t>(kScaleLimit - kScaleLow) * 0x00800080u;
    __device__ __forceinline__ uint32_t low() const { return limit - kLimits; }
    // What turns the scores of block n into log2 of weights.
    __device__ __forceinline__ Two base(int n) const {
        return two(m[n][0] == -INFINITY ? lift : lift - m[n][0], m[n][1] == -INFINITY ? lift : lift - m[n][1]);
    }

    // Two packed pages; the second one's tokens count only if `both` (it is read all the same).
    __device__ __forceinline__ void packed_pages(const uint8_t* unit0, const uint8_t* unit1, bool both,
                                                 const Control<kKind>& ctl, int which) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
        const uint8_t* const units[2] = {unit0, unit1};
        float s[2][kBlocks][4];
        {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int at = kUnitKScales + 16 * gid + 8 + 4 * (tig & 1);
                const uint32_t z0 = *reinterpret_cast<const uint32_t*>(units[p] + at);
                const uint32_t z1 = *reinterpret_cast<const uint32_t*>(units[p] + at + 128);
                const uint32_t zeros[4] = {z0, z1, z0, z1};
#pragma unroll
                for (int n = 0; n < kBlocks; ++n) {
                    const uint2 q = ctl.sums[which][n][lane];
                    mma_bf16_first(s[p][n], zeros, q.x, q.y);
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {    // 64 dims
                uint32_t w[2][4], scale[2][2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint4 x = *reinterpret_cast<const uint4*>(units[p] + 512 * half + 16 * lane);
                    w[p][0] = x.x, w[p][1] = x.y, w[p][2] = x.z, w[p][3] = x.w;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        scale[p][t] = *reinterpret_cast<const uint32_t*>(units[p] + kUnitKScales + 16 * (gid + 8 * t) + 4 * half);
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {         // 32 dims
                    float acc[2][kBlocks][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = 4 * half + 2 * g + i;
                        uint32_t f[2][4];
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const uint32_t x = w[p][2 * g + i], up = x >> 8;
                            f[p][0] = x & 0x000f000fu, f[p][1] = up & 0x000f000fu;
                            f[p][2] = x & 0x00f000f0u, f[p][3] = up & 0x00f000f0u;
                        }
#pragma unroll
                        for (int n = 0; n < kBlocks; ++n) {
                            uint4 q;
                            if (kLow) {
                                q = ctl.frag[which][n][k][lane];
                            } else {
                                const uint2 x = *reinterpret_cast<const uint2*>(&ctl.frag[which][n][k][lane]);
                                q = make_uint4(x.x, x.y, 0u, 0u);
                            }
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
                                if (i == 0) mma_f16_first(acc[p][n], f[p], q.x, q.y);
                                else mma_f16(acc[p][n], f[p], q.x, q.y);
                            }
#pragma unroll
                            for (int p = 0; p < 2; ++p)
                                if (kLow) mma_f16(acc[p][n], f[p], q.z, q.w);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float a = g ? high_of(scale[p][t]) : low_of(scale[p][t]);
#pragma unroll
                            for (int n = 0; n < kBlocks; ++n) {
                                s[p][n][2 * t] = fmaf(a, acc[p][n][2 * t], s[p][n][2 * t]);
                                s[p][n][2 * t + 1] = fmaf(a, acc[p][n][2 * t + 1], s[p][n][2 * t + 1]);
                            }
                        }
                }
            }
        }
        add_low<2>(s);
        if (!both) {
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) s[1][n][0] = s[1][n][1] = s[1][n][2] = s[1][n][3] = -INFINITY;
        }
        uint2 t[2][2];                                // scales and zeros of the values of tokens gid, gid + 8
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) t[p][i] = *reinterpret_cast<const uint2*>(units[p] + kUnitVScales + 8 * (gid + 8 * i));
        const uint32_t most = bf16x2_max(bf16x2_max(t[0][0].x, t[0][1].x), bf16x2_max(t[1][0].x, t[1][1].x));
        const uint32_t least = bf16x2_min(bf16x2_min(t[0][0].x, t[0][1].x), bf16x2_min(t[1][0].x, t[1][1].x));
        weigh<2>(s, most, least, [&] {
            add_wide(units, s, t);
#pragma unroll
            for (int p = 0; p < 2; ++p) t[p][0].x = t[p][1].x = 0u;      // nothing is left for the products below
        });
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float x[kBlocks][4][2];                   // weights times scales: [token, column][group]
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Two scales = two(low_of(t[p][i].x), high_of(t[p][i].x)), zeros = two(low_of(t[p][i].y), high_of(t[p][i].y));
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float y = s[p][n][2 * i + c];
                        const Two weight = two(y, y), scaled = mul2(weight, scales);
                        z[n][c] = fma2(weight, zeros, z[n][c]);
                        parts_of(scaled, x[n][2 * i + c][0], x[n][2 * i + c][1]);
                    }
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {             // 64 dims
                const uint4 v = *reinterpret_cast<const uint4*>(units[p] + kUnitVCodes + 512 * g + 16 * lane);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t f[kBlocks][2];
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t both = pack_f16x2(x[n][2 * i][g], x[n][2 * i + 1][g]);
                        const float2 y = f16x2_of(both);
                        pw[n][g] = add2(pw[n][g], two(y.x, y.y));
                        f[n][i] = transposed(both);                      // tokens as rows
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t c[4];
                    codes_of(w[i], c);
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n) mma_f16(o[n][4 * g + i], c, f[n][0], f[n][1]);
                }
            }
        }
    }
    // 16 dims' codes of the values, as fp16 or bf16 numbers.
    __device__ __forceinline__ static void codes_of(uint32_t w, uint32_t (&c)[4]) {
        const uint32_t up = w >> 8;
        c[0] = w & 0x000f000fu, c[1] = w & 0x00f000f0u, c[2] = up & 0x000f000fu, c[3] = up & 0x00f000f0u;
    }
    // The products of two pages' values, with weights times scales in two bf16 parts: all of the weights, not
    // what fp16 loses of them, as a product with an fp16 subnormal cuts off the sum that it is added to at a
    // fixed place, which left small groups' sums 5 to 8 bits. (Measured, all pages by two parts: 16 x 128K
    // tokens 375 us instead of 363, 2 x 1M with 16 queries 225 instead of 193; a branch of the whole turn 371
    // and 200.)
    __device__ __forceinline__ void add_wide(const uint8_t* const (&units)[2], const float (&s)[2][kBlocks][4],
                                             const uint2 (&t)[2][2]) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint4 v = *reinterpret_cast<const uint4*>(units[p] + kUnitVCodes + 512 * g + 16 * lane);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[kBlocks][2], lo[kBlocks][2];
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x, y;
                        parts_of(add2(two(s[p][n][2 * i], s[p][n][2 * i + 1]), base(n)), x, y);
                        const float scale = g ? high_of(t[p][i].x) : low_of(t[p][i].x);
                        x = fast_exp2(x) * scale, y = fast_exp2(y) * scale;
                        pw[n][g] = add2(pw[n][g], two(x, y));
                        split(x * kWide, y * kWide, hi[n][i], lo[n][i]);
                        hi[n][i] = transposed(hi[n][i]);
                        lo[n][i] = transposed(lo[n][i]);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t c[4];
                    codes_of(w[i], c);
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n) {
                        mma_bf16(o[n][4 * g + i], c, hi[n][0], hi[n][1]);
                        mma_bf16(o[n][4 * g + i], c, lo[n][0], lo[n][1]);
                    }
                }
            }
    }

    // Codes are counted from 0, so the accumulators of the output and the sums with the zeros grow in
    // opposite directions and cancel in the end, where a long row's output is far smaller than either
    // and nothing would be left of it but their rounding. Every kCentre pairs of pages the codes'
    // middle times the weights is moved from the one to the other, and `ahead` times as much again for
    // those to come (0 at the end): the products cut their sums towards 0, and errors of sums that grow
    // from below 0 to above cancel. With kAhead sums that grow evenly go from -0.38 to 0.62 of a turn's;
    // the output of two rows of a million tokens is off by 0.0018 - 0.0019 of itself, 0.0017 of them its
    // rounding to bf16. (The weights' roundings count with the codes' distances from 0 here; zeros with the
    // middle in them from the start would leave 0.0017, and take 4% longer.)
    __device__ __forceinline__ void centre(float ahead) {
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float x[2], y[2];
                parts_of(pw[n][g], x[0], x[1]);
                pw[n][g] = two(-ahead * x[0], -ahead * x[1]);
                x[0] = fmaf(x[0], ahead, x[0]), x[1] = fmaf(x[1], ahead, x[1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    parts_of(z[n][c], y[0], y[1]);
                    y[g] = fmaf(x[c], kMiddle, y[g]);
                    z[n][c] = two(y[0], y[1]);
#pragma unroll
                    for (int i = 4; i < 32; i *= 2) x[c] += __shfl_xor_sync(kAll, x[c], i);
                    x[c] *= -kMiddle * kCode;
#pragma unroll
                    for (int d = 4 * g; d < 4 * g + 4; ++d) {
                        o[n][d][c] += x[c];
                        o[n][d][c + 2] = fmaf(x[c], 16.f, o[n][d][c + 2]);
                    }
                }
            }
    }

    // A bf16 page in shared memory, K and then V, rows of 256 bytes swizzled by 16-byte chunks
    // (chunk_offset), zero from row `valid` on. Queries and weights meet it as two bf16 parts each.
    __device__ __forceinline__ void recent_page(const uint8_t* page, int valid, const Control<kKind>& ctl, int which) {
        const int lane = threadIdx.x & 31, gid = lane >> 2;
        float s[1][kBlocks][4];
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) s[0][n][0] = s[0][n][1] = s[0][n][2] = s[0][n][3] = 0.f;
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {
            uint32_t f[4];
            ldmatrix_x4(f, page + chunk_offset(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) {
                const uint4 q = ctl.frag[which][n][k][lane];
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 x = f16x2_of(c ? q.y : q.x), y = f16x2_of(c ? q.w : q.z);
                    split(x.x + y.x, x.y + y.y, hi[c], lo[c]);
                    if (c) hi[c] = bf16x2_mul(hi[c], 0x41804180u), lo[c] = bf16x2_mul(lo[c], 0x41804180u);      // 16
                }
                mma_bf16(s[0][n], f, hi[0], hi[1]);
                mma_bf16(s[0][n], f, lo[0], lo[1]);
            }
        }
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][n][i] *= kCode;
        add_low<1>(s);
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (gid + 8 * (i >> 1) >= valid) s[0][n][i] = -INFINITY;
        weigh<1>(s, 0u, 0x7f807f80u, [] {});
        uint32_t hi[kBlocks][2], lo[kBlocks][2];
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                split(s[0][n][2 * t] * kCode, s[0][n][2 * t + 1] * kCode, hi[n][t], lo[n][t]);
                hi[n][t] = transposed(hi[n][t]);
                lo[n][t] = transposed(lo[n][t]);
            }
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            // rows of the fragment are dims: a0 (dims, tokens), a1 (dims + 8, tokens), a2 (dims, tokens + 8), a3
            uint32_t f[4];
            ldmatrix_x4_trans(f, page + kPage * kD * 2 +
                                     chunk_offset((lane & 7) + 8 * (lane >> 4), 2 * d + (lane >> 3 & 1)));
            f[1] = bf16x2_mul(f[1], 0x41804180u), f[3] = bf16x2_mul(f[3], 0x41804180u);      // 16
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) {
                mma_bf16(o[n][d], f, hi[n][0], hi[n][1]);
                mma_bf16(o[n][d], f, lo[n][0], lo[n][1]);
            }
        }
    }
    // x and y as a pair of bf16 high parts and one of low parts.
    __device__ __forceinline__ static void split(float x, float y, uint32_t& hi, uint32_t& lo) {
        hi = pack_bf16x2(x, y);
        lo = pack_bf16x2(x - low_of(hi), y - high_of(hi));
    }

    // Low parts of the queries in columns of their own (bf16 queries fill those with copies).
    template <int kPages>
    __device__ __forceinline__ static void add_low(float (&s)[kPages][kBlocks][4]) {
        if (S::kPair && kSplit) {
#pragma unroll
            for (int p = 0; p < kPages; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[p][0][i] += __shfl_xor_sync(kAll, s[p][0][i], 2);
        }
    }
    __device__ __forceinline__ static int chunk_offset(int token, int c) { return token * kD * 2 + ((c ^ (token & 7)) << 4); }

    // The warp's partial: m (log2), l and the unnormalised output, a query a row of `part`.
    __device__ __forceinline__ void put(int group, float* part, float* ms, float* ls) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
            float sum[2], zero[2][2];
            parts_of(l[n], sum[0], sum[1]);
            parts_of(z[n][0], zero[0][0], zero[0][1]);
            parts_of(z[n][1], zero[1][0], zero[1][1]);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(lift)) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x *= 2) {
                    sum[c] += __shfl_xor_sync(kAll, sum[c], x);
                    zero[c][0] += __shfl_xor_sync(kAll, zero[c][0], x);
                    zero[c][1] += __shfl_xor_sync(kAll, zero[c][1], x);
                }
                const int query = n * 8 + 2 * tig + c;
                if (query >= group) continue;         // kPair: the second four columns too
                if (gid == 0) ms[query] = m[n][c], ls[query] = sum[c] * down;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    part[query * kPartStride + d * 16 + gid] = down * fmaf(o[n][d][c], 1.f / kCode, zero[c][d / 4]);
                    part[query * kPartStride + d * 16 + gid + 8] = down * fmaf(o[n][d][c + 2], 0.0625f / kCode, zero[c][d / 4]);
                }
            }
        }
    }
};

// What a warp has of a row: packed pages first, first + step, ... (`count` of them, the ids of the first
// 32 by lane in `ids`) and recent pages recent0, recent0 + step, ... before recent1.
struct Share {
    int b, h, first, step, count;
    uint32_t ids;
    int recent0, recent1, recent;                     // `recent` tokens in all
};

// Leaves the share's sums at `out`, ms and ls. `ahead` is called once the first copies are on their way.
template <int kKind, bool kSplit, typename Ahead>
__device__ __forceinline__ void attend_share(const PackedArgs& a, const Share share, int which, uint8_t* own,
                                             Control<kKind>& ctl, float* out, float* ms, float* ls, Ahead ahead) {
    using S = Shape<kKind>;
    constexpr int kDepth = S::kDepth;
    static_assert(kDepth * kUnitBytes >= 4 * kPage * kD, "a recent page lies in the slots");
    static_assert(kDepth * kUnitBytes >= S::kRows * kPartStride * 4, "a partial lies in the slots");
    const int lane = threadIdx.x & 31, b = share.b, h = share.h, count = share.count;
    const uint8_t* const base = a.packed + static_cast<int64_t>(h) * kUnitBytes + lane * 16;
    const uint32_t stride = static_cast<uint32_t>(a.hkv) * kUnitBytes;
    uint32_t ids = share.ids, next = 0;
    int put = 0;                                      // slot of the next page to fetch
    const auto load = [&](int i) {
        if (i < count) {
            if ((i & 31) == 0) {                      // ids of 32 pages, fetched 32 pages ahead
                if (i > 0) ids = next;
                if (i + 32 + lane < count) next = packed_id(a, b, h, share.first + (i + 32 + lane) * share.step);
            }
            const uint8_t* from = base + static_cast<uint64_t>(__shfl_sync(kAll, ids, i & 31)) * stride;
            uint8_t* to = own + put * kUnitBytes + lane * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async_16(to + j * 512, from + j * 512);
            if (lane < kUnitBytes / 16 - 128) cp_async_16(to + 2048, from + 2048);
        }
        copies_commit();
        if (++put == kDepth) put = 0;
    };
    const auto load_recent = [&](int r) {
        const int valid = min(kPage, share.recent - r * kPage);
        int id = __ldcg(a.recent_table + static_cast<int64_t>(b) * a.max_recent + r);
        if (id < 0 || id >= a.num_cache) {
            report_error(a.st, LOCKS_ERR_BAD_INDEX);
            id = 0;
        }
        const int64_t from = (static_cast<int64_t>(id) * a.hkv + h) * (kPage * kD) + lane * 8;
#pragma unroll
        for (int j = 0; j < kPage / 2; ++j) {         // two tokens
            const int token = 2 * j + (lane >> 4), to = Running<kKind, kSplit>::chunk_offset(token, lane & 15);
            copy_or_zero(own + to, a.k_cache + from + j * 2 * kD, token < valid);
            copy_or_zero(own + kPage * kD * 2 + to, a.v_cache + from + j * 2 * kD, token < valid);
        }
        copies_commit();
    };
    int recent = share.recent0;                       // the next recent page, and the one that is loaded
    bool loaded = false;
    if (count > 0) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) load(i);
    } else if (recent < share.recent1) {
        load_recent(recent);
        loaded = true;
    }
    ahead();
    Running<kKind, kSplit> run;
    run.clear(ctl, which);
    int at = 0;                                       // slot of the next page to use
#pragma unroll 1
    for (int i = 0; i < count; i += 2) {
        copies_wait<kDepth - 2>();
        __syncwarp();
        const uint8_t* const unit0 = own + at * kUnitBytes;
        if (++at == kDepth) at = 0;
        const uint8_t* const unit1 = i + 1 < count ? own + at * kUnitBytes : unit0;
        if (++at == kDepth) at = 0;
        run.packed_pages(unit0, unit1, i + 1 < count, ctl, which);
        if (((i / 2) & (kCentre - 1)) == kCentre - 1) run.centre(kAhead);
        __syncwarp();                                 // both are read
        load(i + kDepth);
        load(i + kDepth + 1);
    }
    if (count > 0) run.centre(0.f);
#pragma unroll 1
    for (; recent < share.recent1; recent += share.step) {
        if (!loaded) {
            copies_wait<0>();
            __syncwarp();                             // the slots are free
            load_recent(recent);
        }
        loaded = false;
        copies_wait<0>();
        __syncwarp();
        run.recent_page(own, min(kPage, share.recent - recent * kPage), ctl, which);
        __syncwarp();
    }
    copies_wait<0>();
    __syncwarp();
    run.put(a.group, out, ms, ls);
    __syncwarp();
}

// The CTA's m and l of each query of `rows` rows, and the factors that the warps' partials are joined
// with. All of the CTA calls it, once the partials are there.
template <int kKind>
__device__ __forceinline__ void join_sums(const PackedArgs& a, int rows, Control<kKind>& ctl) {
    using S = Shape<kKind>;
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < rows * a.group; i += S::kWarps) {        // a warp a query, a lane a partial
        const int which = i / a.group, query = i % a.group;
        const bool on = lane < S::kWarps && (ctl.had[lane] >> which & 1);
        const float m = on ? ctl.m[which][lane][query] : -INFINITY;
        float top = m;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
        const float f = on ? fast_exp2(m - (top == -INFINITY ? 0.f : top)) : 0.f;
        float sum = on ? f * ctl.l[which][lane][query] : 0.f;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(kAll, sum, x);
        if (lane < S::kWarps) ctl.factor[which][lane][query] = f;
        if (lane == 0) ctl.top[which][query] = top, ctl.sum[which][query] = sum;
    }
    __syncthreads();
}
// Query `query`, dim `dim` of row `which` from the warps' partials.
template <int kKind, bool kTwo>
__device__ __forceinline__ float join_warps(const uint8_t* slots, const Control<kKind>& ctl, int which, int query, int dim) {
    using S = Shape<kKind>;
    const float* const o = reinterpret_cast<const float*>(slots) + query * kPartStride + dim;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
        const int had = ctl.had[w];
        float y = o[w * (S::kDepth * kUnitBytes / 4)];
        if (kTwo && which == 0 && had == 3) y = ctl.both[query * kPartStride + dim];
        x = fmaf(ctl.factor[which][w][query], had >> which & 1 ? y : 0.f, x);
    }
    return x;
}

// Short rows: cluster r is row r, and its warps take its pages in turn, so that their ids are on the way
// before the row's length is known; recent pages go to the last warps.
template <int kKind, bool kSplit>
__global__ void __launch_bounds__(Shape<kKind>::kThreads, 1) row_kernel(const __grid_constant__ PackedArgs a, int ctas) {
    using S = Shape<kKind>;
    extern __shared__ __align__(128) uint8_t slots[];
    __shared__ Control<kKind> ctl;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int r = blockIdx.x / ctas;
    grid_dependency_wait();
    allow_dependent_launch();
    Share share;
    share.b = r / a.hkv;
    share.h = r % a.hkv;
    share.first = rank * S::kWarps + warp;
    share.step = ctas * S::kWarps;
    const int mine = share.first + lane * share.step;
    const bool some = mine < (a.selected ? a.k_cap : a.max_pages);
    int id = -1;
    if (some) {
        int j = mine;
        if (a.selected) j = __ldcg(a.selected + (static_cast<int64_t>(share.b) * a.hkv + share.h) * a.k_cap + mine);
        if (j >= 0 && j < a.max_pages) id = __ldcg(a.page_table + static_cast<int64_t>(share.b) * a.max_pages + j);
    }
    const Len len = row_len(a, share.b, share.h, rank == 0 && threadIdx.x == 0);
    share.count = len.pages > share.first ? (len.pages - share.first + share.step - 1) / share.step : 0;
    if (lane < share.count && (id < 0 || id >= a.num_packed)) {
        report_error(a.st, LOCKS_ERR_BAD_INDEX);
        id = 0;
    }
    share.ids = id;
    share.recent0 = share.step - 1 - share.first;
    share.recent1 = len.recent_pages();
    share.recent = len.recent;
    uint8_t* const own = slots + warp * S::kDepth * kUnitBytes;
    const bool has = share.count > 0 || share.recent0 < share.recent1;
    if (lane == 0) ctl.had[warp] = has ? 1 : 0;
    const auto queries = [&] {
        put_all_queries<kKind, kSplit>(a, share.b, share.h, 0, 0, 1, ctl);
        __syncthreads();
    };
    if (has) attend_share<kKind, kSplit>(a, share, 0, own, ctl, reinterpret_cast<float*>(own), ctl.m[0][warp], ctl.l[0][warp], queries);
    else queries();
    __syncthreads();
    join_sums<kKind>(a, 1, ctl);
    const int64_t row = static_cast<int64_t>(share.b) * a.hq + share.h * a.group;
    for (int i = threadIdx.x; i < a.group * kD; i += S::kThreads) {
        const int query = i / kD, dim = i % kD;
        const float x = join_warps<kKind, false>(slots, ctl, 0, query, dim);
        if (ctas == 1) {
            store_row(a, row + query, x, ctl.sum[0][query], dim);
            if (dim == 0) store_lse(a, row + query, ctl.top[0][query], ctl.sum[0][query]);
        } else {
            ctl.cta.o[query][dim] = x;
        }
    }
    if (ctas == 1) return;
    cluster_sync_all();
    for (int i = rank * S::kThreads + threadIdx.x; i < a.group * kD; i += ctas * S::kThreads) {
        const int query = i / kD, dim = i % kD;
        float m[kMaxCluster], l[kMaxCluster], x[kMaxCluster], top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            m[c] = -INFINITY;
            l[c] = x[c] = 0.f;
            if (c < ctas) {
                m[c] = ld_dsmem_f32(dsmem_addr(&ctl.top[0][query], c));
                l[c] = ld_dsmem_f32(dsmem_addr(&ctl.sum[0][query], c));
                x[c] = ld_dsmem_f32(dsmem_addr(&ctl.cta.o[query][dim], c));
            }
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) top = fmaxf(top, m[c]);
        const float base = top == -INFINITY ? 0.f : top;
        float value = 0.f, sum = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            const float f = fast_exp2(m[c] - base);
            value = fmaf(f, x[c], value);
            sum = fmaf(f, l[c], sum);
        }
        store_row(a, row + query, value, sum, dim);
        if (dim == 0) store_lse(a, row + query, top, sum);
    }
    cluster_sync_all();                               // nobody leaves while its sums are read
}

// Steps x0 .. x1 of a part as a warp's share.
__device__ __forceinline__ Share share_of(const PackedArgs& a, const Part part, int x0, int x1) {
    const int lane = threadIdx.x & 31;
    Share s;
    s.b = part.b;
    s.h = part.h;
    s.step = 1;
    s.first = min(part.off + x0, part.len.pages);
    s.count = min(part.off + x1, part.len.pages) - s.first;
    s.ids = lane < s.count ? packed_id(a, s.b, s.h, s.first + lane) : 0;
    // recent pages whose first step is among these
    const int behind = part.off - part.len.pages + kRecentSteps - 1;
    s.recent0 = max(0, (behind + x0) / kRecentSteps);
    s.recent1 = min(part.len.recent_pages(), max(0, (behind + x1) / kRecentSteps));
    s.recent = part.len.recent;
    return s;
}

// One or two parts (neighbouring rows) by all of the CTA, an equal share of the steps to a warp.
// Leaves the warps' partials in shared memory, for join_warps.
template <int kKind, bool kSplit>
__device__ __forceinline__ void attend_parts(const PackedArgs& a, const Part (&part)[2], int parts, uint8_t* slots,
                                             Control<kKind>& ctl) {
    using S = Shape<kKind>;
    const int warp = threadIdx.x >> 5;
    uint8_t* const own = slots + warp * S::kDepth * kUnitBytes;
    const int64_t all = static_cast<int64_t>(part[0].steps) + (parts > 1 ? part[1].steps : 0);
    const int64_t x0 = divide(all * warp, S::kWarps), x1 = divide(all * (warp + 1), S::kWarps);
    const bool has0 = x0 < x1 && x0 < part[0].steps, has1 = x0 < x1 && x1 > part[0].steps;
    if ((threadIdx.x & 31) == 0) ctl.had[warp] = (has0 ? 1 : 0) | (has1 ? 2 : 0);
    bool ready = false;
    const auto queries = [&] {
        if (ready) return;
        put_all_queries<kKind, kSplit>(a, part[0].b, part[0].h, part[1].b, part[1].h, parts, ctl);
        __syncthreads();
        ready = true;
    };
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (!(which ? has1 : has0)) continue;
        const int64_t base = which ? part[0].steps : 0;
        const int s0 = static_cast<int>(max(x0 - base, static_cast<int64_t>(0)));
        const int s1 = static_cast<int>(min(x1 - base, static_cast<int64_t>(which ? part[1].steps : part[0].steps)));
        float* out = which == 0 && has1 ? ctl.both : reinterpret_cast<float*>(own);
        attend_share<kKind, kSplit>(a, share_of(a, which ? part[1] : part[0], s0, s1), which, own, ctl, out, ctl.m[which][warp],
                                    ctl.l[which][warp], queries);
    }
    queries();
    __syncthreads();
    join_sums<kKind>(a, parts, ctl);
}

// Long rows: the line of steps.
template <int kKind, bool kSplit>
__global__ void __launch_bounds__(Shape<kKind>::kThreads, 1) line_kernel(const __grid_constant__ PackedArgs a) {
    using S = Shape<kKind>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
    extern __shared__ __align__(128) uint8_t slots[];
    __shared__ Control<kKind> ctl;
    const bool by_row = cuts_by_row(a, gridDim.x);
    grid_dependency_wait();
    allow_dependent_launch();

    Line<kThreads> line{a, ctl.line};
    line.scan(by_row);
    const int64_t total = line.total();
    const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kWarps - 1) / kWarps));
    int64_t pos = 0, end = 0;
    if (static_cast<int>(blockIdx.x) < ctas) {
        pos = first_step(total, blockIdx.x, ctas);
        end = first_step(total, blockIdx.x + 1, ctas);
    }
    if (!by_row && threadIdx.x == 0) a.cuts[blockIdx.x] = {-1, 0, 0};
    if (pos >= end) return;
    Part part[2];
    part[0] = line.at(pos);
#pragma unroll 1
    while (true) {
        part[0].steps = static_cast<int>(min(end - pos, static_cast<int64_t>(part[0].len.steps() - part[0].off)));
        int parts = 1;
        if (pos + part[0].steps < end) {
            part[1] = line.next(part[0], pos + part[0].steps);
            part[1].steps = static_cast<int>(min(end - pos - part[0].steps, static_cast<int64_t>(part[1].len.steps())));
            parts = 2;
        }
        attend_parts<kKind, kSplit>(a, part, parts, slots, ctl);
#pragma unroll 1
        for (int which = 0; which < parts; ++which) {
            const Part& p = which ? part[1] : part[0];
            const bool begins = p.off == 0, whole = begins && p.steps == p.len.steps();
            const int64_t row = static_cast<int64_t>(p.b) * a.hq + p.h * a.group;
            const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
            for (int i = threadIdx.x; i < a.group * kD; i += kThreads) {
                const int query = i / kD, dim = i % kD;
                const float x = join_warps<kKind, true>(slots, ctl, which, query, dim);
                const float top = ctl.top[which][query], sum = ctl.sum[which][query];
                if (whole) {
                    store_row(a, row + query, x, sum, dim);
                    if (dim == 0) store_lse(a, row + query, top, sum);
                } else {
                    a.part_o[(static_cast<int64_t>(slot) * a.group + query) * kD + dim] = x;
                    if (dim == 0) a.part_ml[slot * a.group + query] = make_float2(top, sum);
                }
            }
            if (begins && threadIdx.x == 0 && (by_row || !whole)) {
                const int r = p.b * a.hkv + p.h;
                const int last = cta_of(total, pos + p.len.steps() - 1, ctas);
                a.cuts[by_row ? r : static_cast<int>(blockIdx.x)] = {whole ? -1 : r, static_cast<int>(blockIdx.x), last};
            }
            pos += p.steps;
        }
        if (pos >= end) break;
        part[0] = line.next(part[parts - 1], pos);
        __syncthreads();                              // the slots and sums are read
    }
}

// Joins the rows that lie in several CTAs: a block per (cut, query).
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ PackedArgs a) {
    __shared__ float weight[kMaxPackedCtas], sums[kJoinThreads / 32], tops[kJoinThreads / 32], acc[kJoinThreads];
    const int query = blockIdx.x % a.group, tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    const PackedCut cut = a.cuts[blockIdx.x / a.group];
    if (cut.row < 0) return;
    const int n = cut.last - cut.first + 1;           // up to kMaxPackedCtas <= kJoinThreads
    const auto slot = [&](int i) { return i == 0 ? 2 * cut.first + 1 : 2 * (cut.first + i); };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < n) ml = a.part_ml[slot(tid) * a.group + query];
    float top = ml.x;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
    if (tid % 32 == 0) tops[tid / 32] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, tops[i]);
    const float w = tid < n ? fast_exp2(ml.x - (top == -INFINITY ? 0.f : top)) : 0.f;
    weight[tid] = w;
    float sum = tid < n ? w * ml.y : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(kAll, sum, x);
    if (tid % 32 == 0) sums[tid / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
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

// Clusters of n CTAs of the short form that fit on the device at once (0: none), from the occupancy
// API, kept per device.
template <int kKind, bool kSplit>
int resident_rows(int n, int num_sms, size_t smem) {
    using S = Shape<kKind>;
    if (n == 1) return num_sms;
    static std::atomic<int> kept[RaiseOnce::kDevices][4];        // one more than the number; 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= RaiseOnce::kDevices) return 0;
    std::atomic<int>& known = kept[dev][n == 2 ? 1 : n == 4 ? 2 : 3];
    if (const int k = known.load()) return k - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n, 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = n;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, row_kernel<kKind, kSplit>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        clusters = 0;
    }
    known.store(clusters + 1);
    return clusters;
}

// CTAs a row of the short form, or 0 for the line: what takes least by a fit to both (us). The short form
// goes in waves of as many clusters as fit at once, `wave` each and 2 for a cluster's join, and `page` for
// each page of a warp; the line takes `line`, `row` for each row of a CTA, and `page` with all pages spread
// over all SMs' warps. Measured (line / 1 / 2 / 4 / 8 CTAs, us, fp32 queries, no recent tokens), 8 kv heads of
// 4 queries: 1 sequence of 128 pages 13.6 / 12.3 / 10.3 / 8.6 / 8.6, of 1024 17.0 / 59.0 / 34.4 / 21.1 / 14.1; 8 of
// 128 17.6 / 12.5 / 10.7 / 17.0 / 40.0, 96 of 128 83.1 / 80.8. Of 8 queries, the same: 14.6 / 13.3 / 11.1 / 9.2 / 9.4,
// 18.1 / 65.7 / 37.7 / 22.8 / 15.3; 19.1 / 13.5 / 11.5 / 18.2 / 43.2, 93.0 / 88.0. 2 kv heads of 16: 1 of 128 17.7 /
// 21.5 / 16.8 / 13.8 / 11.3, 8 of 1024 33.5 / 112 / 62.7 / 36.4 / 44.4, 96 of 128 54.9 / 41.9 / 50.7 / 81.6.
struct FormCost {
    double wave, page, line, row;
};
constexpr FormCost kFormCost[3] = {{5.5, 0.85, 13, 4.5}, {5.8, 0.91, 14, 6.5}, {8.8, 1.17, 16, 15}};
template <int kKind, bool kSplit>
int row_ctas(const PackedArgs& a, int num_sms, size_t smem) {
    constexpr FormCost kCost = kFormCost[kKind];
    constexpr int kWarps = Shape<kKind>::kWarps;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.hkv;
    const int64_t pages = (a.selected ? a.k_cap : a.max_pages) + static_cast<int64_t>(a.max_recent);
    double best = kCost.line + kCost.row * static_cast<double>(rows) / num_sms +
                  kCost.page * static_cast<double>(rows) * static_cast<double>(pages) / (num_sms * kWarps);
    int ctas = 0;
    for (int n = 1; n <= kMaxCluster; n *= 2) {
        const int64_t at_once = resident_rows<kKind, kSplit>(n, num_sms, smem);
        if (at_once == 0) continue;
        const double wave = kCost.wave + (n > 1 ? 2 : 0) + kCost.page * static_cast<double>((pages + n * kWarps - 1) / (n * kWarps));
        const double all = wave * static_cast<double>((rows + at_once - 1) / at_once);
        if (all < best) best = all, ctas = n;
    }
    return ctas;
}

template <int kKind, bool kSplit>
cudaError_t launch_t(const PackedArgs& a, int num_sms, cudaStream_t stream) {
    using S = Shape<kKind>;
    constexpr int kSmem = S::kWarps * S::kDepth * kUnitBytes;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.hkv;
    cudaError_t e = ensure_kernel_attrs<row_kernel<kKind, kSplit>>(kSmem);
    if (e != cudaSuccess) return e;
    if (const int n = row_ctas<kKind, kSplit>(a, num_sms, kSmem))
        return launch_dependent(row_kernel<kKind, kSplit>, rows * n, S::kThreads, kSmem, stream, n, a, n);
    e = ensure_kernel_attrs<line_kernel<kKind, kSplit>>(kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(num_sms, kMaxPackedCtas);
    e = launch_dependent(line_kernel<kKind, kSplit>, ctas, S::kThreads, kSmem, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel, std::min<int64_t>(rows, ctas) * a.group, kJoinThreads, 0, stream, 1, a);
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
