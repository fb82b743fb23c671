// packed_tiles.cu - decode attention over packed pages on tcgen05, for long rows of more than eight
// queries to a kv head.
//
// On mma.sync such a row is bound by the instructions of its warps: fragments and accumulators of
// sixteen queries fill the registers, and a page costs a warp 450 instructions. Here a tile is eight
// pages (128 tokens), and the products run on their own out of tensor memory:
//   S = K Q^T      A: the tile's key codes as fp16, a token a lane; B: the queries, in a high and a low
//                  part (fp32 queries); a 128 x 16 accumulator for each group of 32 dims
//   O^T = V^T P^T  A: the value codes, a dim a lane; B: the weights times the scales of either group of
//                  64 dims, 32 columns (a dim uses its own group's 16)
// The codes' 4-bit fields become fp16 numbers by masks as on mma.sync (packed_attend.cu), and their order
// in a page is that of tcgen05.st's 16 x 256-bit shape too, so a warp brings a page's keys into tensor
// memory with one store. Zeros of keys are a product of their own with the queries' sums; the values'
// middle code is taken off by a product of the weights with a constant. A thread weighs a token for
// eight queries. What a warp does for a page falls to about 300 instructions, two CTAs an SM fill each
// other's waits, and HBM bounds the call again.
#include <algorithm>

#include "packed_units.cuh"
#include "tcgen05.cuh"

namespace locks {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kTilePages = 8, kStages = 4;
constexpr int kStageBytes = kTilePages * kUnitBytes;
constexpr int kQueries = 16, kHalf = 8;               // columns; queries of a thread
// Tensor-memory columns (256): key codes, value codes, key zeros, the constant, scores of the 4 groups
// and of the zeros, outputs.
constexpr uint32_t kKeys = 0, kValues = 64, kZeros = 128, kConst = 136, kScores = 144, kOut = 224, kColumns = 256;
constexpr int kMiddleCode = 8;

struct __align__(1024) Shared {
    uint8_t weights[128 * 128];                       // [token][group * 16 + query] fp16, rows of 128 bytes, swizzled
    uint8_t queries[2][2][16 * 128];                  // [high, low][64 dims][query][64] fp16, swizzled
    uint8_t sums[16 * 128];                           // [query][16] bf16 of the groups' sums, swizzled
    uint8_t stage[kStages][kStageBytes];
    uint64_t scored, added;                           // products with keys; with values
    uint32_t tmem;
    int abort;
    float unit[kQueries];
    float top[kWarps][kHalf], scale[kWarps];          // a warp's largest score of each query; its largest scale
    float l[kWarps][kHalf], z[kWarps][kHalf][2];      // a warp's sums
    float m[kQueries], sum[kQueries], zero[kQueries][2];
    float recent_m[kQueries], recent_l[kQueries];
    LineShared<kThreads> line;
};
// Recent tokens, in the stages: the queries, a page's keys and values, the output.
struct Recent {
    float q[kQueries][kD];
    uint16_t k[kPage][kD + 8], v[kPage][kD];
    float s[kQueries][kPage + 1];
    float o[kQueries][kD];
};
static_assert(sizeof(Recent) <= kStages * kStageBytes, "recent tokens lie in the stages");
constexpr uint64_t kDrainNs = 500000000ull;           // what is in flight ends by itself

// fp16 x fp16 -> fp32 products, 128 rows; bf16_idesc is tcgen05.cuh's.
constexpr uint32_t f16_idesc(int n, bool mn_major_b) { return bf16_idesc(128, n, mn_major_b) & ~((1u << 7) | (1u << 10)); }

__device__ __forceinline__ void store_16x256(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void store_16x256(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// Eight columns of this thread's lane; load_wait before they are used.
__device__ __forceinline__ void load_8(float (&r)[8], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(addr)
                 : "memory");
}
// ... which takes the registers along, so that no use of them moves ahead of the wait.
template <typename... R>
__device__ __forceinline__ void load_wait(R&... r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    ((void)[](float(&x)[8]) {
        asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]));
    }(r), ...);
}
__device__ __forceinline__ void store_8(uint32_t addr, const float (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "f"(r[0]),
                 "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ bool any_thread(bool x) { return __syncthreads_or(x); }

// Place of token i of a page, and of dim d of a 16-dim step, along K: the order in which
// tcgen05.st takes a lane's pairs (2t, 2t + 1) and (8 + 2t, 8 + 2t + 1) of sixteen.
__device__ __forceinline__ int k_place(int i) { return (i & 7) / 2 * 4 + (i >> 3) * 2 + (i & 1); }
// Byte of 16-byte chunk c of a swizzled 128-byte row.
__device__ __forceinline__ int chunk_of(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// A row's queries as operands: 16 threads a query, eight dims each.
template <bool kSplit>
__device__ __forceinline__ void put_queries(const PackedArgs& a, int b, int h, Shared& sh) {
    const int query = threadIdx.x / 16, part = threadIdx.x % 16;
    const bool on = query < a.group;
    const int64_t at = (static_cast<int64_t>(b) * a.hq + h * a.group + (on ? query : 0)) * kD + 8 * part;
    float x[8], big = 0.f;
    if (a.q_type == LOCKS_FP32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i & 1 ? high_of(w[i >> 1]) : low_of(w[i >> 1]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!on) x[i] = 0.f;
        big = fmaxf(big, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 1; o < 16; o *= 2) big = fmaxf(big, __shfl_xor_sync(kAll, big, o));
    const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * kQueryTop;
    const float by = part & 1 ? up * 0.0625f : up;            // fields 4 bits up count 16 times
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = 8 * part + i, step = d / 16, place = step % 4 * 16 + k_place(d % 16);
        const float y = x[i] * by;
        const __half hi = __float2half_rn(y);
        float used = __half2float(hi);
        uint8_t* const row = &sh.queries[0][step / 4][chunk_of(query, place / 8) + place % 8 * 2];
        *reinterpret_cast<__half*>(row) = hi;
        if (kSplit) {
            const __half lo = __float2half_rn(y - used);
            used += __half2float(lo);
            *reinterpret_cast<__half*>(row + sizeof(sh.queries[0])) = lo;
        }
        sum += used;
    }
    if (part & 1) sum *= 16.f;
    sum += __shfl_xor_sync(kAll, sum, 1);
    sum += __shfl_xor_sync(kAll, sum, 2);
    sum *= kCode;
    // the sum's rows k = g, 4 + g and 8 + g are its first 8 bits, the next 8, and the next; 12 + g is 0
    {
        const int g = part / 4, i = part % 4, k = 4 * i + g;
        const float s0 = __bfloat162float(__float2bfloat16_rn(sum)), s1 = __bfloat162float(__float2bfloat16_rn(sum - s0));
        const float mine = i == 0 ? s0 : i == 1 ? s1 : i == 2 ? sum - s0 - s1 : 0.f;
        *reinterpret_cast<__nv_bfloat16*>(&sh.sums[chunk_of(query, k / 8) + k % 8 * 2]) = __float2bfloat16_rn(mine);
    }
    if (part == 0) sh.unit[query] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * kScoreUnit;
}

// What a thread keeps of its token lane: sums over its tokens, for queries 8 * half .. + 7. The maxima
// are the same in all threads of a half.
struct Sums {
    float m[kHalf], l[kHalf];
    Two z[kHalf];                                     // of both groups: of weights times centred zeros
    float lift, scale_limit;
};

// Recent tokens r0 .. r1 (pages) of a row in fp32, by the whole CTA: 16 threads a query. Leaves the
// output in the stages, m and l in shared memory.
__device__ __forceinline__ void attend_recent(const PackedArgs& a, int b, int h, int r0, int r1, int tokens, Shared& sh) {
    Recent& r = *reinterpret_cast<Recent*>(sh.stage);
    const int query = threadIdx.x / 16, part = threadIdx.x % 16;
    const int64_t at = (static_cast<int64_t>(b) * a.hq + h * a.group + (query < a.group ? query : 0)) * kD + 8 * part;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r.q[query][8 * part + i] = a.q_type == LOCKS_FP32 ? static_cast<const float*>(a.q)[at + i]
                                                          : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.q)[at + i]) << 16);
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int page = r0; page < r1; ++page) {
        const int valid = min(kPage, tokens - page * kPage);
        int id = __ldcg(a.recent_table + static_cast<int64_t>(b) * a.max_recent + page);
        if (id < 0 || id >= a.num_cache) {
            if (threadIdx.x == 0) report_error(a.st, LOCKS_ERR_BAD_INDEX);
            id = 0;
        }
        const int token = threadIdx.x / 16;               // 16 threads a token, 16 bytes each
        const int64_t from = (static_cast<int64_t>(id) * a.hkv + h) * (kPage * kD) + token * kD + 8 * part;
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (token < valid) {
            k = __ldcg(reinterpret_cast<const uint4*>(a.k_cache + from));
            v = __ldcg(reinterpret_cast<const uint4*>(a.v_cache + from));
        }
        __syncthreads();
        *reinterpret_cast<uint4*>(&r.k[token][8 * part]) = k;
        *reinterpret_cast<uint4*>(&r.v[token][8 * part]) = v;
        __syncthreads();
        float s = 0.f;                                    // query, token `part`
        for (int d = 0; d < kD; d += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&r.k[part][d]);
            s = fmaf(r.q[query][d], low_of(w), fmaf(r.q[query][d + 1], high_of(w), s));
        }
        s = part < valid ? s * kScaleLog2 : -INFINITY;
        float top = s;
#pragma unroll
        for (int x = 1; x < 16; x *= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
        top = fmaxf(top, m);
        const float f = m == -INFINITY ? 0.f : fast_exp2(m - top);
        const float p = part < valid ? fast_exp2(s - (top == -INFINITY ? 0.f : top)) : 0.f;
        m = top;
        float sum = p;
#pragma unroll
        for (int x = 1; x < 16; x *= 2) sum += __shfl_xor_sync(kAll, sum, x);
        l = l * f + sum;
        r.s[query][part] = p;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= f;
        for (int t = 0; t < valid; ++t) {
            const float w = r.s[query][t];
            const uint4 x = *reinterpret_cast<const uint4*>(&r.v[t][8 * part]);
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(w, i & 1 ? high_of(y[i >> 1]) : low_of(y[i >> 1]), o[i]);
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r.o[query][8 * part + i] = o[i];
    if (part == 0) sh.recent_m[query] = m, sh.recent_l[query] = l;
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) tiles_kernel(const __grid_constant__ PackedArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // tensor memory is reached by quarters of 32 lanes: warps q and q + 4 have quarter q. In a tile they
    // take the keys of pages 2q and 2q + 1, the values' dims 32q .. and 32q + 16 .. of all pages, and
    // weigh the tokens of quarter q for queries 0 .. 7 and 8 .. 15.
    const int quarter = warp & 3, half = warp >> 2, gid = lane >> 2, tig = lane & 3;
    const bool by_row = cuts_by_row(a, gridDim.x);
    if (tid == 0) {
        mbar_init(&sh.scored, 1);
        mbar_init(&sh.added, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&sh.tmem, kColumns);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem, mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    grid_dependency_wait();
    allow_dependent_launch();

    Line<kThreads> line{a, sh.line};
    line.scan(by_row);
    const int64_t total = line.total();
    const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kTilePages - 1) / kTilePages));
    int64_t pos = 0, end = 0;
    if (static_cast<int>(blockIdx.x) < ctas) {
        pos = first_step(total, blockIdx.x, ctas);
        end = first_step(total, blockIdx.x + 1, ctas);
    }
    if (!by_row && tid == 0) a.cuts[blockIdx.x] = {-1, 0, 0};
    // the constant: minus the middle code, in the units of either kind of dims
    if (half == 0) {
        const uint32_t c = (lane & 8) ? 0x80008000u | (kMiddleCode * 16 * 0x10001u) : 0x80008000u | (kMiddleCode * 0x10001u);
        const float f = __uint_as_float(c);
        const float r[8] = {f, f, f, f, f, f, f, f};
        store_8(mine + kConst, r);
        tmem_wait_store();
    }
    uint32_t tiles = 0;                               // so far: phases of `scored`
    uint32_t adds = 0;                                // ... of `added`
    Part part;
    if (pos < end) part = line.at(pos);
    bool ok = true;
#pragma unroll 1
    while (ok && pos < end) {
        part.steps = static_cast<int>(min(end - pos, static_cast<int64_t>(part.len.steps() - part.off)));
        const int b = part.b, h = part.h;
        const int page0 = min(part.off, part.len.pages), page1 = min(part.off + part.steps, part.len.pages);
        const int n = (page1 - page0 + kTilePages - 1) / kTilePages;
        const uint8_t* const base = a.packed + static_cast<int64_t>(h) * kUnitBytes + lane * 16;
        const uint32_t stride = static_cast<uint32_t>(a.hkv) * kUnitBytes;
        // this warp fetches the page that it takes the keys of; past the part's end the last one again
        const int slot = 2 * quarter + half;
        uint32_t ids = 0, next = 0;
        const auto id_of = [&](int t) { return packed_id(a, b, h, min(page0 + t * kTilePages + slot, page1 - 1)); };
        if (lane < n) ids = id_of(lane);
        const auto load = [&](int t) {
            if (t < n) {
                if ((t & 31) == 0) {
                    if (t > 0) ids = next;
                    if (t + 32 + lane < n) next = id_of(t + 32 + lane);
                }
                const uint8_t* from = base + static_cast<uint64_t>(__shfl_sync(kAll, ids, t & 31)) * stride;
                uint8_t* to = sh.stage[t % kStages] + slot * kUnitBytes + lane * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) cp_async_16(to + j * 512, from + j * 512);
                if (lane < kUnitBytes / 16 - 128) cp_async_16(to + 2048, from + 2048);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int t = 0; t < kStages - 1; ++t) load(t);
        put_queries<kSplit>(a, b, h, sh);
        fence_proxy_async_smem();
        Sums run;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) run.m[j] = -INFINITY, run.l[j] = 0.f, run.z[j] = two(0.f, 0.f);
        run.lift = run.scale_limit = 0.f;

#pragma unroll 1
        for (int t = 0; t < n; ++t, ++tiles) {
            const uint8_t* const stage = sh.stage[t % kStages];
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            {                                         // keys, and their zeros
                const uint8_t* const unit = stage + slot * kUnitBytes;
                const uint32_t to = mine + (static_cast<uint32_t>(half * 16) << 16);
                const uint4 k0 = *reinterpret_cast<const uint4*>(unit + 16 * lane);
                const uint4 k1 = *reinterpret_cast<const uint4*>(unit + 512 + 16 * lane);
                const uint2 z0 = *reinterpret_cast<const uint2*>(unit + kUnitKScales + 16 * gid + 8);
                const uint2 z1 = *reinterpret_cast<const uint2*>(unit + kUnitKScales + 16 * (gid + 8) + 8);
                const uint32_t w[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
                uint32_t r[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {         // token gid: pairs 2 tig and 8 + 2 tig; token gid + 8
                    const uint32_t up = w[k] >> 8;
                    r[4 * k] = w[k] & 0x000f000fu, r[4 * k + 1] = w[k] & 0x00f000f0u;
                    r[4 * k + 2] = up & 0x000f000fu, r[4 * k + 3] = up & 0x00f000f0u;
                }
                store_16x256(to + kKeys, r);
                const bool some = tig < 3;
                store_16x256(to + kZeros, some ? z0.x : 0u, some ? z0.y : 0u, some ? z1.x : 0u, some ? z1.y : 0u);
                tmem_wait_store();
            }
            tc_fence_before_sync();
            __syncthreads();                          // keys are there, and everyone's copies
            if (tid == 0 && ok) {
                tc_fence_after_sync();
                const uint64_t sums = sw128_desc(smem_u32(sh.sums), 16, 1024);
                mma_ts(tmem + kScores + 64, tmem + kZeros, sums, bf16_idesc(128, 16, false), false);
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int p = 0; p < (kSplit ? 2 : 1); ++p) {
                        const uint64_t q = sw128_desc(smem_u32(sh.queries[p][k / 4]), 16, 1024) + ((k % 4 * 32) >> 4);
                        mma_ts(tmem + kScores + 16 * (k / 2), tmem + kKeys + 8 * k, q, f16_idesc(16, false), k % 2 + p > 0);
                    }
                mma_commit(&sh.scored);
            }
            // values, once those of the tile before are used up
            if (adds > 0) ok = ok && mbar_wait_bounded(&sh.added, (adds - 1) & 1, a.st.wait_limit_ns);
            tc_fence_after_sync();
            {
                const int db = 2 * quarter + half;
                const uint8_t* const word = stage + kUnitVCodes + 512 * (db >> 2) + 16 * lane + 4 * (db & 3);
                uint32_t r[32];
#pragma unroll
                for (int p = 0; p < kTilePages; ++p) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(word + p * kUnitBytes), up = w >> 8;
                    r[4 * p] = w & 0x000f000fu, r[4 * p + 1] = up & 0x000f000fu;              // dim gid: tokens, tokens + 8
                    r[4 * p + 2] = w & 0x00f000f0u, r[4 * p + 3] = up & 0x00f000f0u;          // dim gid + 8
                }
                store_16x256(mine + (static_cast<uint32_t>(half * 16) << 16) + kValues, r);
                tmem_wait_store();
            }
            // scores of this thread's token
            const int page = 2 * quarter + (lane >> 4), token = lane & 15;
            const uint8_t* const unit = stage + page * kUnitBytes;
            const uint4 ks = *reinterpret_cast<const uint4*>(unit + kUnitKScales + 16 * token);
            const uint2 vs = *reinterpret_cast<const uint2*>(unit + kUnitVScales + 8 * token);
            ok = ok && mbar_wait_bounded(&sh.scored, tiles & 1, a.st.wait_limit_ns);
            tc_fence_after_sync();
            float s[kHalf];
            {
                float g0[8], g1[8];
                load_8(s, mine + kScores + 64 + 8 * half);
                load_8(g0, mine + kScores + 8 * half);
                load_8(g1, mine + kScores + 16 + 8 * half);
                load_wait(s, g0, g1);
                const float a0 = low_of(ks.x), a1 = high_of(ks.x), a2 = low_of(ks.y), a3 = high_of(ks.y);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) s[j] = fmaf(a1, g1[j], fmaf(a0, g0[j], s[j]));
                load_8(g0, mine + kScores + 32 + 8 * half);
                load_8(g1, mine + kScores + 48 + 8 * half);
                load_wait(g0, g1);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) s[j] = fmaf(a3, g1[j], fmaf(a2, g0[j], s[j]));
            }
            const bool on = page0 + t * kTilePages + page < page1;
            const float largest = fmaxf(low_of(vs.x), high_of(vs.x));
            bool over = largest > run.scale_limit;
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                s[j] = on ? s[j] * sh.unit[8 * half + j] : -INFINITY;
                over |= s[j] > run.m[j] + kSlack;
            }
            tc_fence_before_sync();
            if (any_thread(over)) {                   // see packed_attend.cu
                float top[kHalf], scale = largest;
#pragma unroll
                for (int j = 0; j < kHalf; ++j) {
                    top[j] = s[j];
#pragma unroll
                    for (int x = 1; x < 32; x *= 2) top[j] = fmaxf(top[j], __shfl_xor_sync(kAll, top[j], x));
                    if (lane == 0) sh.top[warp][j] = top[j];
                }
#pragma unroll
                for (int x = 1; x < 32; x *= 2) scale = fmaxf(scale, __shfl_xor_sync(kAll, scale, x));
                if (lane == 0) sh.scale[warp] = scale;
                __syncthreads();
                float change = 0.f;
                for (int w = 0; w < kWarps; ++w) scale = fmaxf(scale, sh.scale[w]);
                if (scale > run.scale_limit) {
                    const int e = kScaleTop - min(max(static_cast<int>(__float_as_uint(scale) >> 23) - 127, -95), 105);
                    change = static_cast<float>(e) - run.lift;
                    run.lift += change;
                    run.scale_limit = kScaleLimit * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                }
                float f[kHalf], o[kHalf];
#pragma unroll
                for (int j = 0; j < kHalf; ++j) {
                    float to = run.m[j];
#pragma unroll
                    for (int w = 0; w < 4; ++w) to = fmaxf(to, sh.top[half * 4 + w][j]);
                    f[j] = run.m[j] == -INFINITY ? 0.f : fast_exp2(run.m[j] - to + change);
                    run.m[j] = to;
                    run.l[j] *= f[j];
                    run.z[j] = mul2(run.z[j], two(f[j], f[j]));
                }
                if (t > 0) {                          // the output so far: all its products are done
                    const uint32_t at = mine + kOut + 16 * (quarter / 2) + 8 * half;
                    load_8(o, at);
                    load_wait(o);
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) o[j] *= f[j];
                    store_8(at, o);
                    tmem_wait_store();
                }
                __syncthreads();                      // the warps' maxima are read
            }
            // weights, and weights times scales as fp16
            {
                const float v0 = low_of(vs.x), v1 = high_of(vs.x);
                const Two scales = two(v0, v1);
                const Two zeros = two(fmaf(static_cast<float>(kMiddleCode), v0, low_of(vs.y)),
                                      fmaf(static_cast<float>(kMiddleCode), v1, high_of(vs.y)));
                float x[kHalf][2];
#pragma unroll
                for (int j = 0; j < kHalf; ++j) {
                    const float p = fast_exp2(s[j] + (run.m[j] == -INFINITY ? run.lift : run.lift - run.m[j]));
                    run.l[j] += p;
                    const Two weight = two(p, p);
                    run.z[j] = fma2(weight, zeros, run.z[j]);
                    parts_of(mul2(weight, scales), x[j][0], x[j][1]);
                }
                const int row = 16 * page + k_place(token);
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    *reinterpret_cast<uint4*>(&sh.weights[chunk_of(row, 2 * g + half)]) =
                        make_uint4(pack_f16x2(x[0][g], x[1][g]), pack_f16x2(x[2][g], x[3][g]), pack_f16x2(x[4][g], x[5][g]),
                                   pack_f16x2(x[6][g], x[7][g]));
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            if (!ok) sh.abort = 1;
            __syncthreads();
            ok = !sh.abort;
            if (tid == 0 && ok) {
                tc_fence_after_sync();
                const uint64_t w = sw128_desc(smem_u32(sh.weights), 16, 1024);
                constexpr uint32_t kKind = f16_idesc(32, true);
#pragma unroll
                for (int p = 0; p < kTilePages; ++p) {
                    mma_ts(tmem + kOut, tmem + kValues + 8 * p, w + p * (2048 >> 4), kKind, t + p > 0);
                    mma_ts(tmem + kOut, tmem + kConst, w + p * (2048 >> 4), kKind, true);
                }
                mma_commit(&sh.added);
            }
            if (!ok) break;
            ++adds;
            load(t + kStages - 1);                    // into the stage of the tile before, which all have read
        }
        if (ok && n > 0) ok = mbar_wait_bounded(&sh.added, (adds - 1) & 1, a.st.wait_limit_ns);
        tc_fence_after_sync();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (any_thread(!ok)) {
            ok = false;
            break;
        }
        // the warps' sums, and the part's
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
            float l = run.l[j], z0, z1;
            parts_of(run.z[j], z0, z1);
#pragma unroll
            for (int x = 1; x < 32; x *= 2) {
                l += __shfl_xor_sync(kAll, l, x);
                z0 += __shfl_xor_sync(kAll, z0, x);
                z1 += __shfl_xor_sync(kAll, z1, x);
            }
            if (lane == 0) {
                sh.l[warp][j] = l, sh.z[warp][j][0] = z0, sh.z[warp][j][1] = z1;
                if (quarter == 0) sh.m[8 * half + j] = run.m[j];
            }
        }
        __syncthreads();
        const float down = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(run.lift)) << 23);
        if (tid < kQueries) {
            const int hf = tid / 8, j = tid % 8;
            float l = 0.f, z0 = 0.f, z1 = 0.f;
            for (int w = 0; w < 4; ++w) l += sh.l[4 * hf + w][j], z0 += sh.z[4 * hf + w][j][0], z1 += sh.z[4 * hf + w][j][1];
            sh.sum[tid] = l * down, sh.zero[tid][0] = z0 * down, sh.zero[tid][1] = z1 * down;
        }
        const int behind = part.off - part.len.pages + kRecentSteps - 1;
        const int recent0 = max(0, behind / kRecentSteps);
        const int recent1 = min(part.len.recent_pages(), max(0, (behind + part.steps) / kRecentSteps));
        const bool recent = recent0 < recent1;
        if (recent) attend_recent(a, b, h, recent0, recent1, part.len.recent, sh);
        __syncthreads();
        // a dim a thread, eight queries
        const bool begins = part.off == 0, whole = begins && part.steps == part.len.steps();
        const int dim = 32 * quarter + lane, to = 2 * blockIdx.x + (begins ? 1 : 0);
        const int64_t row = static_cast<int64_t>(b) * a.hq + h * a.group;
        float o[kHalf] = {};
        if (n > 0) {
            load_8(o, mine + kOut + 16 * (quarter / 2) + 8 * half);
            load_wait(o);
        }
        const float back = (dim & 8 ? 0.0625f / kCode : 1.f / kCode) * down;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
            const int query = 8 * half + j;
            if (query >= a.group) continue;
            float x = n > 0 ? fmaf(o[j], back, sh.zero[query][quarter / 2]) : 0.f;
            float m = n > 0 ? sh.m[query] : -INFINITY, l = n > 0 ? sh.sum[query] : 0.f;
            if (recent) {
                const float top = fmaxf(m, sh.recent_m[query]), from = top == -INFINITY ? 0.f : top;
                const float f = fast_exp2(m - from), g = fast_exp2(sh.recent_m[query] - from);
                x = fmaf(f, x, g * reinterpret_cast<const Recent*>(sh.stage)->o[query][dim]);
                l = fmaf(f, l, g * sh.recent_l[query]);
                m = top;
            }
            if (whole) {
                store_row(a, row + query, x, l, dim);
                if (dim == 0) store_lse(a, row + query, m, l);
            } else {
                a.part_o[(static_cast<int64_t>(to) * a.group + query) * kD + dim] = x;
                if (dim == 0) a.part_ml[to * a.group + query] = make_float2(m, l);
            }
        }
        if (begins && tid == 0 && (by_row || !whole)) {
            const int r = b * a.hkv + h;
            const int last = cta_of(total, pos + part.len.steps() - 1, ctas);
            a.cuts[by_row ? r : static_cast<int>(blockIdx.x)] = {whole ? -1 : r, static_cast<int>(blockIdx.x), last};
        }
        pos += part.steps;
        if (pos < end) part = line.next(part);
        tc_fence_before_sync();
        __syncthreads();                              // stages, sums and the output are read
        tc_fence_after_sync();
    }
    // a wait that ran out: what was issued is waited for all the same, and the error recorded
    if (!ok) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        mbar_wait_bounded(&sh.scored, tiles & 1, kDrainNs);
        if (adds > 0) mbar_wait_bounded(&sh.added, (adds - 1) & 1, kDrainNs);
        if (tid == 0) report_error(a.st, LOCKS_ERR_TIMEOUT);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_free(tmem, kColumns);
}

}  // namespace

template <bool kSplit>
static cudaError_t launch_tiles_t(const PackedArgs& a, int ctas, cudaStream_t stream) {
    const cudaError_t e = ensure_kernel_attrs<tiles_kernel<kSplit>>(sizeof(Shared));
    return e != cudaSuccess ? e : launch_dependent(tiles_kernel<kSplit>, ctas, kThreads, sizeof(Shared), stream, 1, a);
}
static_assert(2 * (sizeof(Shared) + 1024) <= 228 * 1024, "two CTAs an SM");

int packed_tiles_ctas(int num_sms) { return std::min(2 * num_sms, kMaxPackedCtas); }

cudaError_t launch_packed_tiles(const PackedArgs& a, int ctas, cudaStream_t stream) {
    return a.q_type == LOCKS_FP32 ? launch_tiles_t<true>(a, ctas, stream) : launch_tiles_t<false>(a, ctas, stream);
}

}  // namespace locks
