// packed_units.cuh - what the kernels of the packed attention share: the rows' lengths, the line of
// steps that long rows are cut on, packed arithmetic and the stores of results.
#pragma once

#include "pool_internal.h"
#include "two_floats.cuh"

namespace locks {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRecentSteps = 3;                       // of a recent bf16 page: 8 KB against 2.4
constexpr float kScaleLog2 = kInvSqrtD * kLog2e;
// Queries are scaled by 2^(14 - e), e the exponent of the row's largest (within -100..100, so that
// the factors are numbers); with codes of 2^-24 scores are in units of 2^(e + 10).
constexpr float kQueryTop = 0x1p14f, kScoreUnit = 0x1p10f * kScaleLog2;
constexpr float kCode = 0x1p-24f, kMiddle = 7.5f;
constexpr float kSlack = 8.f;                         // log2 that a score may pass the maximum by
// Weights times a value's scale are fp16 (11 bits, rounded: 2^-11 of a weight at most, up or down;
// the output has 8). All weights carry a factor 2^lift that brings the largest scale so far to
// 2^5..2^6, and is set anew when a scale times it passes 2^7: with kSlack they stay below 2^15.
// fp16 ends at 2^-25, which is 2^-21 of a weight of 1 where a scale times the factor is 2^-4. For a
// pair of pages with a scale below that (or below 0) weights enter in two bf16 parts, 16 bits
// whatever the scale: they carry kWide, as codes are 2^-133 in bf16.
// Scales below 2^kScaleLeast count as that large, for the zeros, of up to 2^50, take the factor too:
// 2^(54 + kSlack + 50) and the sums of it are numbers.
constexpr int kScaleTop = 5, kScaleLimit = 7, kScaleLow = -4, kScaleLeast = -49;
constexpr float kWide = 0x1p109f;

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Whether either half of a is greater than (less than) b's.
__device__ __forceinline__ bool any_greater(uint32_t a, uint32_t b) {
    return !__hbleu2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
}
__device__ __forceinline__ bool any_less(uint32_t a, uint32_t b) { return any_greater(b, a); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 f16x2_of(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
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
    const int pages = a.selected ? __ldcg(a.n_selected + static_cast<int64_t>(b) * a.hkv + h) : __ldcg(a.seq_pages + b);
    const int recent = a.max_recent > 0 ? __ldcg(a.recent_tokens + b) : 0;
    r.pages = checked(a, pages, a.selected ? a.k_cap : a.max_pages, report);
    r.recent = checked(a, recent, static_cast<int64_t>(a.max_recent) * kPage, report);
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

// CTA c of n holds steps first(c) .. first(c + 1) of the line. (A 64-bit division is a long routine,
// kept in one place.)
static __device__ __noinline__ int64_t divide64(int64_t x, int64_t y) { return x / y; }
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    if (x < (1ll << 32) && y < (1ll << 32)) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return divide64(x, y);
}
__device__ __forceinline__ int64_t first_step(int64_t total, int c, int n) { return divide(total * c, n); }
__device__ __forceinline__ int cta_of(int64_t total, int64_t step, int n) {
    return static_cast<int>(divide((step + 1) * n - 1, total));
}

__device__ __forceinline__ void store_row(const PackedArgs& a, int64_t row, float value, float sum, int dim) {
    a.out[row * kD + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : __fdividef(value, sum)));
}
__device__ __forceinline__ void store_lse(const PackedArgs& a, int64_t row, float m, float sum) {
    if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
}

// Steps off .. off + steps of a row.
struct Part {
    int b, h, off, steps;
    Len len;
};

// ----------------------------------------------------------------- the line of steps

template <int kThreads>
struct LineShared {
    int64_t upto[kThreads], warp_sum[kThreads / 32];      // steps of the sequences up to each thread's last
    int2 len[kThreads];                                   // pages and recent tokens of sequence i, where that is enough
};

// All rows' steps one after the other, by a CTA of kThreads threads.
template <int kThreads>
struct Line {
    const PackedArgs& a;
    LineShared<kThreads>& s;

    __device__ __forceinline__ int per() const { return (a.batch + kThreads - 1) / kThreads; }
    // Lengths are kept where they are the same for all kv heads and there is a thread for each sequence.
    __device__ __forceinline__ bool kept() const { return !a.selected && a.batch <= kThreads; }
    __device__ __forceinline__ Len length(int b, int h) const {
        if (!kept()) return row_len(a, b, h, false);
        const int2 x = s.len[b];
        return Len{x.x, x.y};
    }
    __device__ __forceinline__ int64_t total() const { return s.upto[kThreads - 1]; }

    // All of the CTA. Writes the results of rows without tokens, which are nobody's.
    __device__ __forceinline__ void scan(bool by_row) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        int64_t sum = 0;
        if (kept()) {
            Len len = {0, 0};
            if (tid < a.batch) len = row_len(a, tid, 0, blockIdx.x == 0);
            s.len[tid] = make_int2(len.pages, len.recent);
            sum = static_cast<int64_t>(len.steps()) * a.hkv;
        } else {
            for (int i = 0; i < per(); ++i) {
                const int b = tid * per() + i;
                if (b < a.batch) sum += seq_steps(a, b, blockIdx.x == 0);
            }
        }
        int64_t upto = sum;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
            const int64_t y = __shfl_up_sync(kAll, upto, x);
            if (lane >= x) upto += y;
        }
        if (lane == 31) s.warp_sum[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += s.warp_sum[w];
        s.upto[tid] = upto;
        for (int r = blockIdx.x * kThreads + tid; r < a.batch * a.hkv; r += gridDim.x * kThreads) {
            const int b = r / a.hkv, h = r % a.hkv;
            if (length(b, h).steps() != 0) continue;
            for (int q = 0; q < a.group; ++q) {
                const int64_t row = static_cast<int64_t>(b) * a.hq + h * a.group + q;
                for (int d = 0; d < kD; d += 8) *reinterpret_cast<uint4*>(a.out + row * kD + d) = make_uint4(0, 0, 0, 0);
                store_lse(a, row, 0.f, 0.f);
            }
            if (by_row) a.cuts[r] = {-1, 0, 0};
        }
        __syncthreads();
    }
    // The row at step `pos` of the line. Whole warps.
    __device__ __forceinline__ Part at(int64_t pos) const {
        Part p;
        int before = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i)
            before += __popc(__ballot_sync(kAll, s.upto[i * 32 + (threadIdx.x & 31)] <= pos));
        int64_t at = pos - (before > 0 ? s.upto[before - 1] : 0);
        p.b = before * per();
        if (kept()) {
            p.len = length(p.b, 0);
            p.h = static_cast<int>(divide(at, p.len.steps()));
            p.off = static_cast<int>(at - static_cast<int64_t>(p.h) * p.len.steps());
        } else {
            for (int64_t n; p.b < a.batch - 1 && at >= (n = seq_steps(a, p.b, false)); ++p.b) at -= n;
            p.h = 0;
            for (p.len = length(p.b, 0); p.h < a.hkv - 1 && at >= p.len.steps(); p.len = length(p.b, ++p.h)) at -= p.len.steps();
            p.off = static_cast<int>(at);
        }
        p.steps = 0;
        return p;
    }
    // The row behind p's with any steps, which begins at `pos` (there is one as long as steps are left). The
    // very next one where that has some, else by the sums: two of 4096 sequences in use, at the ends, with the
    // rows between them gone through one by one 8.6 ms.
    __device__ __forceinline__ Part next(const Part& p, int64_t pos) const {
        Part r = p;
        if (++r.h == a.hkv) ++r.b, r.h = 0;
        r.len = length(r.b, r.h);
        if (r.len.steps() == 0) return at(pos);
        r.off = 0;
        return r;
    }
};

}  // namespace
}  // namespace locks
