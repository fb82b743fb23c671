// packed.cu - pages of the bf16 pool to 4 bits and back (locks_pack_pages, locks_unpack_pages).
//
// 8 KB of bf16 on one side of a unit (a page of one kv head), 2432 bytes on the other, so HBM bounds
// both. A warp packs the keys or the values of a unit, or unpacks both. The bf16 side is read and
// written 16 bytes a lane, two tokens to an instruction; the codes go through a staging area in
// shared memory, because the order of the attention's fragments spreads a lane's eight dims over
// four or eight words. Packing takes a warp 800 instructions for 64 values a lane, with most of the
// arithmetic on two values at once, and is bounded by them (64% of the issue slots): 4096 pages of 8 kv heads
// in 68 us (5.1 TB/s of both sides; 73 without the next values on their way meanwhile). Unpacking
// them takes 55 - 57 us, as fast as HBM copies.
#include <algorithm>

#include "pool_internal.h"
#include "two_floats.cuh"

namespace locks {
namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {      // NaN if either is
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Quotients below are rounded as fp32 division rounds them, by Markstein's theorem (IBM J. Res. Dev.
// 34, 1990): with r the correctly rounded 1 / s, q = v r and q + (v - s q) r is the rounded v / s.
// (Newton's step makes r of the approximate reciprocal; for the 8-bit scales here the codes are the
// rounded quotient's for each of the 128 mantissas, which a test goes through.) How a quotient is rounded matters: bf16 values lie on borders between two
// codes often, and there the product with the reciprocal alone may fall to either side.

// Least and greatest of eight values as a pair (least, -greatest): both are then minima.
__device__ __forceinline__ uint32_t extremes(const uint4& x) {
    const uint32_t lo = bf16x2_min(bf16x2_min(x.x, x.y), bf16x2_min(x.z, x.w));
    const uint32_t hi = bf16x2_max(bf16x2_max(x.x, x.y), bf16x2_max(x.z, x.w)) ^ 0x80008000u;
    return bf16x2_min(prmt(lo, hi, 0x5410u), prmt(lo, hi, 0x7632u));
}

// Two groups, of kLanes neighbouring lanes with eight values each: scales and zeros as bf16 bits,
// those of the first group in the low half.
template <int kLanes>
__device__ __forceinline__ void group_scales(const uint4& x0, const uint4& x1, uint32_t& scales, uint32_t& zeros) {
    uint32_t e0 = extremes(x0), e1 = extremes(x1);
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) {
        e0 = bf16x2_min(e0, __shfl_xor_sync(kAll, e0, o));
        e1 = bf16x2_min(e1, __shfl_xor_sync(kAll, e1, o));
    }
    const Two least = two(low_of(e0), low_of(e1)), most = two(-high_of(e0), -high_of(e1));
    const float by = 1.f / 15.f;
    const Two range = fma2(least, two(-1.f, -1.f), most), q = mul2(range, two(by, by));
    float s0, s1;
    parts_of(fma2(fma2(two(-15.f, -15.f), q, range), two(by, by), q), s0, s1);
    scales = pack_bf16x2(s0, s1);
    if ((scales & 0xffffu) < 0x0080u) scales &= 0xffff0000u;      // below 2^-126
    if ((scales >> 16) < 0x0080u) scales &= 0x0000ffffu;
    zeros = prmt(e0, e1, 0x5410u);
}

// The codes of two groups' values, element i of x0 and of x1, as floats kRound + code, whose low bytes
// are the codes. Scales so small or large that the remainder or the reciprocal leave the normal
// numbers divide. The quotient is within [0, 15.06], as the scale is rounded by at most 2^-8 of
// itself, so codes need no bounds: where words are put together, all other bits of a result's two low
// bytes count as 0. A group that is not finite, of NaN scale, gets codes 0.
constexpr float kRound = 12582912.f;              // 1.5 * 2^23
__device__ __noinline__ float divided(float v, float s) { return s > 0.f ? __fdiv_rn(v, s) : 0.f; }
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return __fmaf_rn(__fmaf_rn(-s, r, 1.f), r, r);
}
__device__ __forceinline__ bool ordinary(float s) { return s > 0x1p-90f && s < 0x1p120f; }
__device__ __forceinline__ void codes_of(const uint4& x0, const uint4& x1, uint32_t scales, uint32_t zeros,
                                         uint32_t (&c0)[8], uint32_t (&c1)[8]) {
    const float s0 = low_of(scales), s1 = high_of(scales);
    const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
    const Two z = two(-low_of(zeros), -high_of(zeros));
    if (ordinary(s0) && ordinary(s1)) {
        const Two by = two(reciprocal(s0), reciprocal(s1)), minus = two(-s0, -s1), round = two(kRound, kRound);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = w0[i >> 1], b = w1[i >> 1];
            const Two v = add2(i & 1 ? two(high_of(a), high_of(b)) : two(low_of(a), low_of(b)), z), q = mul2(v, by);
            float y0, y1;
            parts_of(add2(fma2(fma2(minus, q, v), by, q), round), y0, y1);
            c0[i] = __float_as_uint(y0), c1[i] = __float_as_uint(y1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = w0[i >> 1], b = w1[i >> 1];
            float v0, v1;
            parts_of(add2(i & 1 ? two(high_of(a), high_of(b)) : two(low_of(a), low_of(b)), z), v0, v1);
            c0[i] = __float_as_uint(__fadd_rn(divided(v0, s0), kRound));
            c1[i] = __float_as_uint(__fadd_rn(divided(v1, s1), kRound));
        }
    }
}

// Whether there is something to do for an entry of the lists.
__device__ __forceinline__ bool find_pages(const PackArgs& a, int from, int to) {
    if (from < 0 || to < 0) return false;
    if (from < a.num_src && to < a.num_dst) return true;
    report_error(a.st, LOCKS_ERR_BAD_INDEX);
    return false;
}

// A word whose codes of the even half lie four bits below those of the odd one: this lane's half, and the
// other's from the neighbour, which gets `give` in return.
__device__ __forceinline__ uint32_t both_halves(uint32_t keep, uint32_t give, int half) {
    const uint32_t got = __shfl_xor_sync(kAll, give, 1);
    return keep * (half ? 16u : 1u) + got * (half ? 1u : 16u);
}

// Keys: codes at 0 and scales at 1024 of `unit`.
__device__ __forceinline__ void pack_keys(const uint4 (&x)[8], uint8_t* unit) {
    const int lane = threadIdx.x & 31, row = lane >> 4, chunk = lane & 15, half = chunk & 1, w = chunk >> 1;
    uint8_t* const words = unit + 512 * (w >> 2) + 4 * (w & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {                     // tokens t and t + 8
        const int t = 2 * j + row;
        uint32_t c0[8], c1[8], scales, zeros, part[4];
        group_scales<4>(x[j], x[j + 4], scales, zeros);
        codes_of(x[j], x[j + 4], scales, zeros, c0, c1);
#pragma unroll
        for (int p = 0; p < 4; ++p)                   // a pair of dims to a word: the codes' bytes at 0, 8, 16, 24
            part[p] = prmt(c0[2 * p], c1[2 * p], 0x1140u) | prmt(c0[2 * p + 1], c1[2 * p + 1], 0x4011u);
#pragma unroll
        for (int p = 0; p < 2; ++p)                   // the even half keeps words 0, 1
            *reinterpret_cast<uint32_t*>(words + 16 * (4 * t + 2 * half + p)) =
                both_halves(half ? part[p + 2] : part[p], half ? part[p] : part[p + 2], half);
        if ((chunk & 3) == 0) {
            uint16_t* sz = reinterpret_cast<uint16_t*>(unit + 1024 + 16 * t) + (chunk >> 2);
            sz[0] = static_cast<uint16_t>(scales), sz[4] = static_cast<uint16_t>(zeros);
            sz[64] = static_cast<uint16_t>(scales >> 16), sz[68] = static_cast<uint16_t>(zeros >> 16);
        }
    }
}

// Values, the same way.
__device__ __forceinline__ void pack_values(const uint4 (&x)[8], uint8_t* unit) {
    const int lane = threadIdx.x & 31, row = lane >> 4, chunk = lane & 15, half = chunk & 1, w = chunk >> 1;
    uint8_t* const words = unit + 512 * (w >> 2) + 4 * (w & 3);
    const uint32_t place = row ? 0x4011u : 0x1140u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = 2 * j + row;
        uint32_t c0[8], c1[8], scales, zeros, part[8], four[4];
        group_scales<8>(x[j], x[j + 4], scales, zeros);
        codes_of(x[j], x[j + 4], scales, zeros, c0, c1);
#pragma unroll
        for (int d = 0; d < 8; ++d) part[d] = prmt(c0[d], c1[d], place);        // a word a dim: bytes at 0, 8 or 16, 24
#pragma unroll
        for (int d = 0; d < 4; ++d)                   // dims 4 * half .. of both halves
            four[d] = both_halves(half ? part[d + 4] : part[d], half ? part[d] : part[d + 4], half);
#pragma unroll
        for (int d = 0; d < 2; ++d) {                 // ... and 2 * row .. of both tokens
            const uint32_t give = row ? four[d] : four[d + 2], keep = row ? four[d + 2] : four[d];
            *reinterpret_cast<uint32_t*>(words + 16 * (4 * (4 * half + 2 * row + d) + j)) =
                keep | __shfl_xor_sync(kAll, give, 16);
        }
        if ((chunk & 7) == 0) {
            uint16_t* sz = reinterpret_cast<uint16_t*>(unit + 1024 + 8 * t) + (chunk >> 3);
            sz[0] = static_cast<uint16_t>(scales), sz[2] = static_cast<uint16_t>(zeros);
            sz[32] = static_cast<uint16_t>(scales >> 16), sz[34] = static_cast<uint16_t>(zeros >> 16);
        }
    }
}

// A warp's next keys or values are on their way to shared memory while it packs these, and the ids
// of those behind are too. Each lane reads what it has copied itself.
constexpr int kPackCtas = 3;                          // of an SM, by their registers
__global__ void __launch_bounds__(kWarps * 32, kPackCtas) pack_kernel(const __grid_constant__ PackArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][1024 + 256];
    __shared__ uint4 ahead[kWarps][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* const unit = stage[warp];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t items = 2 * static_cast<int64_t>(a.n) * a.hkv;         // a unit's keys, its values
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int heads = __ffs(a.hkv) - 1;               // a power of two
    int src = -1, dst = -1;                           // pages of the next item
    const auto ids = [&](int64_t v) {
        if (v >= items) return;
        const int i = static_cast<int>(v >> (1 + heads));
        src = __ldg(a.src + i);
        dst = a.dst ? __ldg(a.dst + i) : src;
    };
    // Starts on item v; the page that it goes to, or -1.
    const auto fetch = [&](int64_t v) {
        if (v >= items || !find_pages(a, src, dst)) return -1;
        const int h = static_cast<int>(v >> 1) & (a.hkv - 1);
        const uint16_t* in = (v & 1 ? a.v_in : a.k_in) + (static_cast<int64_t>(src) * a.hkv + h) * (kPage * kD) + lane * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) cp_async_16(&ahead[warp][j][lane], in + j * 2 * kD);      // tokens 2j, 2j + 1
        asm volatile("cp.async.commit_group;" ::: "memory");
        return dst;
    };
    ids(u);
    int to = fetch(u);
    ids(u + stride);
    for (; u < items; u += stride) {
        const bool values = u & 1;
        const int h = static_cast<int>(u >> 1) & (a.hkv - 1), here = to;
        uint4 x[8];
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ahead[warp][j][lane];
        __syncwarp();
        to = fetch(u + stride);
        ids(u + 2 * stride);
        if (here < 0) continue;
        if (values) pack_values(x, unit);
        else pack_keys(x, unit);
        __syncwarp();
        uint8_t* const out = a.packed + (static_cast<int64_t>(here) * a.hkv + h) * kUnitBytes + lane * 16;
        uint8_t* const codes = out + (values ? kUnitVCodes : 0);
        uint8_t* const scales = out + (values ? kUnitVScales : kUnitKScales);
        const uint4* const from_stage = reinterpret_cast<const uint4*>(unit) + lane;
        *reinterpret_cast<uint4*>(codes) = from_stage[0];
        *reinterpret_cast<uint4*>(codes + 512) = from_stage[32];
        if (lane < (values ? 8 : 16)) *reinterpret_cast<uint4*>(scales) = from_stage[64];
        __syncwarp();
    }
}

// Whether fp32 holds all bits of zero + scale * code: from the last one of either (8 bits each) to the
// carry of the sum, whose code is below 2^4.
__device__ __forceinline__ bool sums_fit(float s, float z) {
    const int apart = static_cast<int>(__float_as_uint(z) >> 23 & 255u) - static_cast<int>(__float_as_uint(s) >> 23 & 255u);
    return apart >= -11 && apart <= 15;
}
// zero + scale * code rounded to odd: of the two floats next to the exact sum (the product of 8 and 4 bits
// is exact) the one whose last bit is 1, or the sum itself. Rounding that to bf16 is rounding the sum once
// (fp32 has more than two bits on top of bf16's); rounded to nearest here, a sum just off the middle
// between two bf16 values would fall on it.
__device__ __forceinline__ float to_odd(float s, float c, float z) {
    const float down = __fmaf_rd(s, c, z), up = __fmaf_ru(s, c, z);
    return __float_as_uint(down) & 1u ? down : up;
}
// Eight values of a group as bf16, rounded once. (All of them by to_odd: the 64K-token prompt 126 us, packing
// and unpacking, instead of 123.)
__device__ __forceinline__ void put_values(uint16_t* out, const uint32_t (&code)[8], float s, float z) {
    float x[8];
    if (sums_fit(s, z)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(s, static_cast<float>(code[i]), z);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_odd(s, static_cast<float>(code[i]), z);
    }
    *reinterpret_cast<uint4*>(out) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

__global__ void __launch_bounds__(kWarps * 32) unpack_kernel(const __grid_constant__ PackArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kUnitBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* const unit = stage[warp];
    const int row = lane >> 4, chunk = lane & 15, heads = __ffs(a.hkv) - 1;
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t units = static_cast<int64_t>(a.n) * a.hkv;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int i = static_cast<int>(u >> heads), h = static_cast<int>(u) & (a.hkv - 1);
        const int from = __ldg(a.src + i), to = a.dst ? __ldg(a.dst + i) : from;
        if (!find_pages(a, from, to)) continue;
        const uint4* in = reinterpret_cast<const uint4*>(a.packed + (static_cast<int64_t>(from) * a.hkv + h) * kUnitBytes);
        __syncwarp();
        uint4 x[5];
#pragma unroll
        for (int j = 0; j < 5; ++j)
            if (j < 4 || lane < kUnitBytes / 16 - 128) x[j] = __ldcs(in + j * 32 + lane);
#pragma unroll
        for (int j = 0; j < 5; ++j)
            if (j < 4 || lane < kUnitBytes / 16 - 128) reinterpret_cast<uint4*>(unit)[j * 32 + lane] = x[j];
        __syncwarp();
        const int half = chunk & 1, w = chunk >> 1;
        const uint8_t* word = unit + 512 * (w >> 2) + 4 * (w & 3);
        const int64_t at = (static_cast<int64_t>(to) * a.hkv + h) * (kPage * kD) + lane * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = 2 * j + row;
            {
                const uint16_t* sz = reinterpret_cast<const uint16_t*>(unit + kUnitKScales + 16 * t) + (chunk >> 2);
                const float s = low_of(sz[0]), z = low_of(sz[4]);
                uint32_t c[8];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint32_t x = *reinterpret_cast<const uint32_t*>(word + 16 * (4 * (t & 7) + p)) >>
                                       (4 * half + 8 * (t >> 3));
                    c[2 * p] = x & 15, c[2 * p + 1] = x >> 16 & 15;
                }
                put_values(a.k_out + at + j * 2 * kD, c, s, z);
            }
            {
                const uint16_t* sz = reinterpret_cast<const uint16_t*>(unit + kUnitVScales + 8 * t) + (chunk >> 3);
                const float s = low_of(sz[0]), z = low_of(sz[2]);
                uint32_t c[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    c[d] = *reinterpret_cast<const uint32_t*>(word + kUnitVCodes + 16 * (4 * d + (t & 7) / 2)) >>
                               (16 * (t & 1) + 4 * half + 8 * (t >> 3)) &
                           15;
                put_values(a.v_out + at + j * 2 * kD, c, s, z);
            }
        }
    }
}

int grid_of(int64_t items, int num_sms, int per_sm) {
    return static_cast<int>(std::min<int64_t>((items + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms) * per_sm));
}

}  // namespace

cudaError_t launch_pack(const PackArgs& a, int num_sms, cudaStream_t stream) {
    return launch_dependent(pack_kernel, grid_of(2 * static_cast<int64_t>(a.n) * a.hkv, num_sms, kPackCtas), kWarps * 32, 0, stream, 1, a);
}
cudaError_t launch_unpack(const PackArgs& a, int num_sms, cudaStream_t stream) {
    return launch_dependent(unpack_kernel, grid_of(static_cast<int64_t>(a.n) * a.hkv, num_sms, 8), kWarps * 32, 0, stream, 1, a);
}

}  // namespace locks
