// append.cu - head norms, rotary positions and the paged K/V write in one pass
// (locks_append_tokens).
//
// Per head row x of 128: y = x / sqrt(mean(x^2) + eps) * w, then each pair (a, b)
// of y turns by its angle, (a cos - b sin, b cos + a sin), and the row is rounded
// once into q_out or into its cache row. Values are copied (rounded) beside them.
//
// Half a warp holds a row, a lane eight of its elements in two runs of four such that both
// elements of a pair are in one lane: (4l.., rot/2 + 4l..) when pairs lie half the rotated
// part apart, eight in a row when they are neighbours or not rotated. So a row costs four
// shuffles (the mean) and no exchange. A warp takes a token's rows two at a time, several
// loads ahead, and shares nothing with other warps: a token's cosines and sines are computed
// once by its warp, and each lane keeps the four pairs that are its own. The pass reads its
// inputs once and writes its outputs once, so HBM bounds it at prompt lengths and latency at
// decode. 24 warps an SM in CTAs of two: 269 us for 65,536 tokens of 32 + 2 x 8 heads, 88% of
// the copy rate (32 warps of 64 registers spill: 286; CTAs of eight warps: 283).
//
// Angles: a pair turns by position * inv_freq / (2 pi) turns, of which only the
// fraction matters. The host rounds inv_freq / (2 pi) to a multiple of 2^-64 turns;
// the product with the position modulo 2^64 is then that fraction exactly (integer
// overflow drops whole turns), off by at most |position| * 2^-65 <= 2^-34 turns for
// the rounding of the factor. fp32 angles instead would be off by position * 2^-24
// radians, 0.06 at 1M tokens. The nearest quarter turn is taken off in integers and
// sincospi sees at most an eighth of a turn.
#include <algorithm>

#include "cache_internal.h"

namespace locks {
namespace {

constexpr int kThreads = 64;
constexpr int kWarps = kThreads / 32;

// Four consecutive elements; inputs are read once, past L1.
template <typename T>
struct Run4;
template <>
struct Run4<float> {
    uint4 a;
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w)
                     : "l"(p));
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
    }
};
struct Run4Half {
    uint2 a;
    __device__ __forceinline__ void load_raw(const void* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(a.x), "=r"(a.y) : "l"(p));
    }
};
template <>
struct Run4<__nv_bfloat16> : Run4Half {
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { load_raw(p); }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = __uint_as_float(a.x << 16), x[1] = __uint_as_float(a.x & 0xffff0000u);
        x[2] = __uint_as_float(a.y << 16), x[3] = __uint_as_float(a.y & 0xffff0000u);
    }
};
template <>
struct Run4<__half> : Run4Half {
    __device__ __forceinline__ void load(const __half* p) { load_raw(p); }
    __device__ __forceinline__ void get(float* x) const {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a.x));
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&a.y));
        x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
    }
};

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// cos and sin (times scale) of a position's pair.
__device__ __forceinline__ float2 turn(int64_t pos, uint64_t turns, float scale) {
    const uint64_t frac = static_cast<uint64_t>(pos) * turns;         // fraction of a turn, modulo 1
    const uint32_t f = static_cast<uint32_t>((frac + 0x80000000ull) >> 32);
    const uint32_t quarter = (f + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(f - (quarter << 30));   // within an eighth of a turn
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    // a quarter turn on: (cos, sin) -> (-sin, cos)
    float2 r = (quarter & 1) ? make_float2(-s, c) : make_float2(c, s);
    if (quarter & 2) r = make_float2(-r.x, -r.y);
    return make_float2(r.x * scale, r.y * scale);
}

// What a lane does to its eight elements of a row.
struct Lane {
    int o1, o2;                      // its runs of four
    bool turned, neighbours;         // its pairs are rotated; they are (x[2i], x[2i + 1]), else (x[i], x[i + 4])
    float c[4], s[4];
    float w[8];                      // norm weights

    template <bool kNorm>
    __device__ __forceinline__ void apply(float (&x)[8], float eps) const {
        if (kNorm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float scale = rsqrtf(ss * (1.f / kD) + eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * w[e];
        }
        if (turned) {
            if (neighbours) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = x[2 * e], m = x[2 * e + 1];
                    x[2 * e] = p * c[e] - m * s[e];
                    x[2 * e + 1] = m * c[e] + p * s[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = x[e], m = x[e + 4];
                    x[e] = p * c[e] - m * s[e];
                    x[e + 4] = m * c[e] + p * s[e];
                }
            }
        }
    }
};

// Rows first + half, first + half + 2, ... < last of `src` (128 elements apart) through
// `lane` (kTouch) into `dst` (dst_step elements apart), kAhead row pairs in flight.
template <bool kTouch, bool kNorm, typename T, typename TO>
__device__ __forceinline__ void rows(const T* src, TO* dst, int64_t dst_step, int first, int last, const Lane& lane,
                                     float eps) {
    constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;
    const int half = (threadIdx.x >> 4) & 1;
    Run4<T> in[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int r = first + 2 * i + half;
        if (r < last) {
            in[i][0].load(src + r * kD + lane.o1);
            in[i][1].load(src + r * kD + lane.o2);
        }
    }
#pragma unroll 1
    for (int r0 = first; r0 < last; r0 += 2 * kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + 2 * i + half;
            float x[8];
            in[i][0].get(x);
            in[i][1].get(x + 4);
            if (r + 2 * kAhead < last) {
                in[i][0].load(src + (r + 2 * kAhead) * kD + lane.o1);
                in[i][1].load(src + (r + 2 * kAhead) * kD + lane.o2);
            }
            if (kTouch) lane.apply<kNorm>(x, eps);
            if (r < last) {
                store4(dst + r * dst_step + lane.o1, x);
                store4(dst + r * dst_step + lane.o2, x + 4);
            }
        }
    }
}

__device__ __forceinline__ void load_weights(Lane& lane, const float* w) {
    const float4 a = *reinterpret_cast<const float4*>(w + lane.o1), b = *reinterpret_cast<const float4*>(w + lane.o2);
    lane.w[0] = a.x, lane.w[1] = a.y, lane.w[2] = a.z, lane.w[3] = a.w;
    lane.w[4] = b.x, lane.w[5] = b.y, lane.w[6] = b.z, lane.w[7] = b.w;
}

// A unit of work is `per_unit` head rows (even) of one token, heads of q first, then k, then v;
// a warp each.
template <typename T, typename TQ>
__global__ void __launch_bounds__(kThreads, 12) append_kernel(const __grid_constant__ AppendArgs a,
                                                             int units_per_token, int per_unit) {
    __shared__ __align__(16) float turn_s[kWarps][2][64];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (u >= static_cast<int64_t>(a.num_tokens) * units_per_token) return;
    const int t = static_cast<int>(u / units_per_token);
    const int first = static_cast<int>(u - static_cast<int64_t>(t) * units_per_token) * per_unit;
    const int index = a.cache_index[t];
    const int seq = a.token_seq ? a.token_seq[t] : t;
    const int l = threadIdx.x & 31, sub = l & 15;           // rows alternate between half warps
    const int nq = a.q ? a.hq : 0, last = min(first + per_unit, nq + 2 * a.hkv);
    const int pairs = a.rot_dim / 2;
    float* cos_s = turn_s[threadIdx.x >> 5][0];
    float* sin_s = turn_s[threadIdx.x >> 5][1];
    Lane lane;
    lane.neighbours = a.interleaved;
    lane.turned = 8 * sub < a.rot_dim;
    const bool apart = lane.turned && !a.interleaved;       // 4 * sub < pairs, as pairs is a multiple of 8
    lane.o1 = apart ? 4 * sub : 8 * sub;
    lane.o2 = apart ? pairs + 4 * sub : 8 * sub + 4;
    for (int i = l; i < pairs; i += 32) {
        const int64_t pos = a.positions[static_cast<int64_t>(a.axis[i]) * a.num_tokens + t];
        const float2 cs = turn(pos, a.turns[i], a.rope_scale);
        cos_s[i] = cs.x;
        sin_s[i] = cs.y;
    }
    if (index < 0) return;                                  // padding; uniform: the warp has one token
    const int lpage = index / kPage;
    int page = -1;
    if (seq >= 0 && seq < a.batch && lpage < a.max_pages)
        page = a.page_table[static_cast<int64_t>(seq) * a.max_pages + lpage];
    if (page < 0 || page >= a.num_phys) {
        if (l == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        return;
    }
    __syncwarp();
    if (lane.turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) lane.c[e] = cos_s[4 * sub + e], lane.s[e] = sin_s[4 * sub + e];
    }
    if (first < nq) {
        const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(t) * a.q_stride;
        TQ* dst = static_cast<TQ*>(a.q_out) + static_cast<int64_t>(t) * a.hq * kD;
        if (a.q_weight) {
            load_weights(lane, a.q_weight);
            rows<true, true>(src, dst, kD, first, min(last, nq), lane, a.eps);
        } else {
            rows<true, false>(src, dst, kD, first, min(last, nq), lane, a.eps);
        }
    }
    const int64_t at = (static_cast<int64_t>(page) * a.hkv * kPage + index % kPage) * kD;
    if (last > nq && first < nq + a.hkv) {
        const T* src = static_cast<const T*>(a.k) + static_cast<int64_t>(t) * a.k_stride;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.k_cache) + at;
        if (a.k_weight) {
            load_weights(lane, a.k_weight);
            rows<true, true>(src, dst, kPage * kD, max(first - nq, 0), min(last - nq, a.hkv), lane, a.eps);
        } else {
            rows<true, false>(src, dst, kPage * kD, max(first - nq, 0), min(last - nq, a.hkv), lane, a.eps);
        }
    }
    if (last > nq + a.hkv) {
        const T* src = static_cast<const T*>(a.v) + static_cast<int64_t>(t) * a.v_stride;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.v_cache) + at;
        rows<false, false>(src, dst, kPage * kD, max(first - nq - a.hkv, 0), last - nq - a.hkv, lane, a.eps);
    }
}

template <typename T, typename TQ>
cudaError_t launch_t(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    const int total = (a.q ? a.hq : 0) + 2 * a.hkv;
    // Many tokens: a warp per token, which computes the token's angles once. Few: a token's rows
    // spread over as many warps as are resident (a pair of rows each at least), so that the
    // call is one round of loads.
    const int64_t share = static_cast<int64_t>(a.num_tokens) * total / (12 * static_cast<int64_t>(num_sms));
    const int per_unit = static_cast<int>(std::min<int64_t>((share + 3) / 2 * 2, (total + 1) / 2 * 2));
    const int units_per_token = (total + per_unit - 1) / per_unit;
    const int64_t ctas = (static_cast<int64_t>(a.num_tokens) * units_per_token + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<T, TQ>, a, units_per_token, per_unit);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_in(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    return a.q_type == LOCKS_FP32 ? launch_t<T, float>(a, num_sms, stream)
                                  : launch_t<T, __nv_bfloat16>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    switch (a.in_type) {
        case LOCKS_FP32: return launch_in<float>(a, num_sms, stream);
        case LOCKS_FP16: return launch_in<__half>(a, num_sms, stream);
        default: return launch_in<__nv_bfloat16>(a, num_sms, stream);
    }
}

}  // namespace locks
