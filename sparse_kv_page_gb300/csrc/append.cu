// append.cu - head norms, rotary positions and the paged K/V write in one pass
// (locks_append_tokens).
//
// Per head row x of 128: y = x / sqrt(mean(x^2) + eps) * w, then each pair (a, b)
// of y turns by its angle, (a cos - b sin, b cos + a sin), and the row is rounded
// once into q_out or into its cache row. Values are copied (rounded) beside them.
//
// Half a warp holds a row, eight consecutive elements a lane: one 16-byte load for
// 16-bit types, the mean by four shuffles, a pair's partner (i, i + rot/2) from the
// lane rot/16 away, one 16-byte cache store. Nothing is staged; the pass reads its
// inputs once and writes its outputs once, so HBM bounds it at prompt lengths and
// latency at decode.
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
constexpr int kRows = kThreads / 16;     // head rows in flight per CTA
constexpr int kBatch = 3;                // rows a half warp loads before it uses the first

template <typename T>
struct Row8;                             // eight consecutive elements of a row

template <>
struct Row8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Row8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
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
    __device__ __forceinline__ void load(const __half* p) { a = *reinterpret_cast<const uint4*>(p); }
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

// Grid: (tokens, row blocks): a CTA takes the rows blockIdx.y * kRows * per_block ... of
// its token, heads of q first, then k, then v.
template <typename T, typename TQ>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int rows_per_cta) {
    __shared__ __align__(16) float cos_s[64], sin_s[64];
    grid_dependency_wait();
    allow_dependent_launch();
    const int t = blockIdx.x, tid = threadIdx.x;
    const int index = a.cache_index[t];
    if (index < 0) return;                                  // padding
    const int seq = a.token_seq ? a.token_seq[t] : t;
    const int lpage = index / kPage;
    int page = -1;
    if (seq >= 0 && seq < a.batch && lpage < a.max_pages)
        page = a.page_table[static_cast<int64_t>(seq) * a.max_pages + lpage];
    if (page < 0 || page >= a.num_phys) {
        if (tid == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
        return;
    }
    const int half_rot = a.rot_dim / 2;
    if (tid < half_rot) {
        const int64_t pos = a.positions[static_cast<int64_t>(a.axis[tid]) * a.num_tokens + t];
        const uint64_t frac = static_cast<uint64_t>(pos) * a.turns[tid];   // fraction of a turn, modulo 1
        const uint32_t f = static_cast<uint32_t>((frac + 0x80000000ull) >> 32);
        const uint32_t quarter = (f + 0x20000000u) >> 30;
        const int32_t rest = static_cast<int32_t>(f - (quarter << 30));    // within an eighth of a turn
        float s, c;
        sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
        // a quarter turn on: (cos, sin) -> (-sin, cos)
        float co = (quarter & 1) ? -s : c, si = (quarter & 1) ? c : s;
        if (quarter & 2) co = -co, si = -si;
        cos_s[tid] = co * a.rope_scale;
        sin_s[tid] = si * a.rope_scale;
    }
    __syncthreads();

    const int lane = tid & 15, slot = tid >> 4;
    const int nq = a.q ? a.hq : 0;
    const int total = nq + 2 * a.hkv;
    const int first = blockIdx.y * rows_per_cta;
    const int last = min(first + rows_per_cta, total);
    const int64_t cache_row = static_cast<int64_t>(page) * a.hkv * kPage + index % kPage;
    const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(t) * a.q_stride + lane * 8;
    const T* k = static_cast<const T*>(a.k) + static_cast<int64_t>(t) * a.k_stride + lane * 8;
    const T* v = static_cast<const T*>(a.v) + static_cast<int64_t>(t) * a.v_stride + lane * 8;
    for (int r0 = first; r0 < last; r0 += kRows * kBatch) {
        Row8<T> in[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRows + slot;
            if (r < last)
                in[i].load(r < nq ? q + r * kD : r < nq + a.hkv ? k + (r - nq) * kD : v + (r - nq - a.hkv) * kD);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (r0 + i * kRows >= last) break;              // uniform in the CTA
            const int r = r0 + i * kRows + slot;
            const bool live = r < last;
            const bool is_q = r < nq, is_v = r >= nq + a.hkv;
            float x[8];
            if (live) {
                in[i].get(x);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
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
                    Row8<float> wv;
                    wv.load(w + lane * 8);
                    float we[8];
                    wv.get(we);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * we[e];
                }
            }
            if (half_rot > 0 && __any_sync(0xffffffffu, live && !is_v)) {
                if (a.interleaved) {
                    if (!is_v && lane * 8 < a.rot_dim) {
                        const float4 c = *reinterpret_cast<const float4*>(&cos_s[lane * 4]);
                        const float4 s = *reinterpret_cast<const float4*>(&sin_s[lane * 4]);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = x[2 * e], m = x[2 * e + 1];
                            x[2 * e] = p * cc[e] - m * sn[e];
                            x[2 * e + 1] = m * cc[e] + p * sn[e];
                        }
                    }
                } else {
                    const int n = half_rot >> 3;             // lanes per half
                    const bool upper = lane >= n;
                    const int at = upper ? lane - n : lane;  // the pair's lane in the lower half
                    const int from = (tid & 16) | (lane < 2 * n ? (upper ? lane - n : lane + n) : lane);
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], from);
                    if (!is_v && lane < 2 * n) {
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(&cos_s[at * 8 + e]);
                            const float4 s = *reinterpret_cast<const float4*>(&sin_s[at * 8 + e]);
                            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                x[e + f] = x[e + f] * cc[f] + (upper ? y[e + f] : -y[e + f]) * sn[f];
                        }
                    }
                }
            }
            if (!live) continue;
            if (is_q) {
                store_row8(static_cast<TQ*>(a.q_out) + (static_cast<int64_t>(t) * a.hq + r) * kD + lane * 8, x);
            } else {
                const int h = is_v ? r - nq - a.hkv : r - nq;
                __nv_bfloat16* cache = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache);
                store_row8(cache + (cache_row + h * kPage) * kD + lane * 8, x);
            }
        }
    }
}

template <typename T, typename TQ>
cudaError_t launch_t(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    const int total = (a.q ? a.hq : 0) + 2 * a.hkv;
    // Few tokens: a CTA per kRows rows, so that each half warp has one row and the call
    // is one round of loads. Many: a CTA per token, whose angles are computed once.
    const bool few = static_cast<int64_t>(a.num_tokens) * total <= static_cast<int64_t>(num_sms) * 8 * kRows;
    const int rows = few ? kRows : total;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_tokens, (total + rows - 1) / rows, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<T, TQ>, a, rows);
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
