// append.cu - head norms, rotary positions and the paged K/V write in one pass
// (locks_append_tokens).
//
// Per head row x of 128: y = x / sqrt(mean(x^2) + eps) * w, then each pair (a, b)
// of y turns by its angle, (a cos - b sin, b cos + a sin), and the row is rounded
// once into q_out or into its cache row. Values are copied (rounded) beside them.
//
// Half a warp holds a row, eight consecutive elements a lane: one 16-byte load for
// 16-bit types, the mean by four shuffles, a pair's partner (i, i + rot/2) from the
// lane rot/16 away, one 16-byte cache store. A warp takes a token's rows two at a time,
// four such loads ahead, and shares nothing with other warps: a token's cosines and
// sines are computed once by its warp, and each lane keeps those of its own elements.
// The pass reads its inputs once and writes its outputs once, so HBM bounds it at prompt
// lengths and latency at decode. (A CTA per token that met at a barrier after the angles
// had too few loads in flight: 514 us for 65,536 tokens of 32 + 2 x 8 heads.)
//
// Angles: a pair turns by position * inv_freq / (2 pi) turns, of which only the
// fraction matters. The host rounds inv_freq / (2 pi) to a multiple of 2^-64 turns;
// the product with the position modulo 2^64 is then that fraction exactly (integer
// overflow drops whole turns), off by at most |position| * 2^-65 <= 2^-34 turns for
// the rounding of the factor. fp32 angles instead would be off by position * 2^-24
// radians, 0.06 at 1M tokens. The nearest quarter turn is taken off in integers and
// sincospi sees at most an eighth of a turn.
#include "cache_internal.h"

namespace locks {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;                // row pairs in flight per warp

// Inputs are read once: past L1.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <typename T>
struct Row8;                             // eight consecutive elements of a row

template <>
struct Row8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = load_once(p);
        b = load_once(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z);
        x[3] = __uint_as_float(a.w), x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y);
        x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    }
};
template <>
struct Row8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = load_once(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Row8<__half> {
    uint4 a;
    __device__ __forceinline__ void load(const __half* p) { a = load_once(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

__device__ __forceinline__ void store_row8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_row8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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

// A unit of work is `per_unit` head rows (even) of one token, heads of q first, then k, then v;
// the warps of the grid stride over tokens * units_per_token of them.
template <typename T, typename TQ>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int units_per_token,
                                                          int per_unit) {
    __shared__ __align__(16) float turn_s[kWarps][2][64];
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 15;                              // of the row; rows alternate between half warps
    const int nq = a.q ? a.hq : 0, total = nq + 2 * a.hkv;
    const int half_rot = a.rot_dim / 2, reach = half_rot >> 3;        // lanes per half of the rotated part
    const bool upper = sub >= reach;
    const int pair = a.interleaved ? 4 * sub : 8 * (upper ? sub - reach : sub);   // first pair of this lane
    const bool turned = a.interleaved ? 8 * sub < a.rot_dim : sub < 2 * reach;
    const int partner = (lane & 16) | (turned ? (upper ? sub - reach : sub + reach) : sub);
    float* cos_s = turn_s[warp][0];
    float* sin_s = turn_s[warp][1];
    const int64_t units = static_cast<int64_t>(a.num_tokens) * units_per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units; u += step) {
        const int t = static_cast<int>(u / units_per_token);
        const int first = static_cast<int>(u - static_cast<int64_t>(t) * units_per_token) * per_unit;
        const int last = min(first + per_unit, total);
        const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(t) * a.q_stride + sub * 8;
        const T* k = static_cast<const T*>(a.k) + static_cast<int64_t>(t) * a.k_stride + sub * 8;
        const T* v = static_cast<const T*>(a.v) + static_cast<int64_t>(t) * a.v_stride + sub * 8;
        auto src = [&](int r) {
            return r < nq ? q + r * kD : r < nq + a.hkv ? k + (r - nq) * kD : v + (r - nq - a.hkv) * kD;
        };
        Row8<T> in[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = first + 2 * i + (lane >> 4);
            if (r < last) in[i].load(src(r));
        }
        const int index = a.cache_index[t];
        const int seq = a.token_seq ? a.token_seq[t] : t;
        const int lpage = index / kPage;
        int page = -1;
        if (index >= 0 && seq >= 0 && seq < a.batch && lpage < a.max_pages)
            page = a.page_table[static_cast<int64_t>(seq) * a.max_pages + lpage];
        for (int i = lane; i < half_rot; i += 32) {
            const int64_t pos = a.positions[static_cast<int64_t>(a.axis[i]) * a.num_tokens + t];
            const float2 cs = turn(pos, a.turns[i], a.rope_scale);
            cos_s[i] = cs.x;
            sin_s[i] = cs.y;
        }
        __syncwarp();
        float c[8], s[8];
        if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool used = e < 4 || !a.interleaved;
                c[e] = used ? cos_s[pair + e] : 0.f;
                s[e] = used ? sin_s[pair + e] : 0.f;
            }
        }
        __syncwarp();
        if (page < 0 || page >= a.num_phys) {               // uniform: the warp has one token
            if (index >= 0 && lane == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            continue;
        }
        const int64_t cache_row = static_cast<int64_t>(page) * a.hkv * kPage + index % kPage;
#pragma unroll 1
        for (int r0 = first; r0 < last; r0 += 2 * kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (r0 + 2 * i >= last) break;              // uniform
                const int r = r0 + 2 * i + (lane >> 4);
                const bool live = r < last;
                const bool is_q = r < nq, is_v = r >= nq + a.hkv;
                float x[8];
                in[i].get(x);
                {
                    const int next = r + 2 * kAhead;
                    if (next < last) in[i].load(src(next));
                }
                const float* w = is_q ? a.q_weight : a.k_weight;
                const bool normed = live && !is_v && w;
                if (__any_sync(0xffffffffu, normed)) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (normed) {
                        const float scale = rsqrtf(ss * (1.f / kD) + a.eps);
                        const float4 w0 = reinterpret_cast<const float4*>(w + sub * 8)[0];
                        const float4 w1 = reinterpret_cast<const float4*>(w + sub * 8)[1];
                        const float we[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * we[e];
                    }
                }
                if (half_rot > 0 && __any_sync(0xffffffffu, live && !is_v)) {
                    if (a.interleaved) {
                        if (!is_v && turned) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float p = x[2 * e], m = x[2 * e + 1];
                                x[2 * e] = p * c[e] - m * s[e];
                                x[2 * e + 1] = m * c[e] + p * s[e];
                            }
                        }
                    } else {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
                        if (!is_v && turned) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = x[e] * c[e] + (upper ? y[e] : -y[e]) * s[e];
                        }
                    }
                }
                if (live) {
                    if (is_q) {
                        store_row8(static_cast<TQ*>(a.q_out) + (static_cast<int64_t>(t) * a.hq + r) * kD + sub * 8, x);
                    } else {
                        const int h = is_v ? r - nq - a.hkv : r - nq;
                        __nv_bfloat16* cache = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache);
                        store_row8(cache + (cache_row + h * kPage) * kD + sub * 8, x);
                    }
                }
            }
        }
    }
}

template <typename T, typename TQ>
cudaError_t launch_t(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    const int total = (a.q ? a.hq : 0) + 2 * a.hkv;
    // Few tokens: a warp per pair of rows, so that the call is one round of loads. Many: a warp
    // per token, which computes the token's angles once.
    const bool few = static_cast<int64_t>(a.num_tokens) * total <= static_cast<int64_t>(num_sms) * 8 * kWarps;
    const int per_unit = few ? 2 : (total + 1) / 2 * 2;
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
