// pool_internal.h - launchers of the packed cache and the page pool (locks_pool.h).
#pragma once

#include "../../include/locks_pool.h"
#include "cache_internal.h"

namespace locks {

constexpr int kUnitBytes = LOCKS_PACKED_BYTES;     // a page of one kv head
constexpr int kUnitVCodes = 1024;                  // offsets within it
constexpr int kUnitKScales = 2048;                 // 16 bytes a token: 4 scales, 4 zeros
constexpr int kUnitVScales = 2304;                 // 8 bytes a token: 2 scales, 2 zeros

struct PackArgs {
    const uint16_t* k_in;          // packing reads these
    const uint16_t* v_in;
    uint16_t* k_out;               // unpacking writes these
    uint16_t* v_out;
    uint8_t* packed;
    const int32_t* src;
    const int32_t* dst;            // nullable: src
    int n, hkv, num_src, num_dst;
    DeviceStatus st;
};
cudaError_t launch_pack(const PackArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_unpack(const PackArgs& a, int num_sms, cudaStream_t stream);

struct PackedArgs {
    const void* q;                 // fp32 or bf16 [batch][hq][128]
    const uint8_t* packed;         // [num_packed][hkv][kUnitBytes]
    const int32_t* page_table;     // [batch][max_pages]
    const int32_t* seq_pages;      // [batch]
    const int32_t* selected;       // nullable [batch][hkv][k_cap]
    const int32_t* n_selected;
    const uint16_t* k_cache;       // bf16 pool of num_cache pages
    const uint16_t* v_cache;
    const int32_t* recent_table;   // [batch][max_recent], not read when max_recent is 0
    const int32_t* recent_tokens;  // [batch]
    uint16_t* out;
    float* lse;                    // nullable
    int q_type, k_cap, max_recent, batch, hq, hkv, group, max_pages, num_packed, num_cache;
    // workspace regions (packed_layout)
    struct PackedCut* cuts;        // [kMaxPackedCtas]: of each row, or where there are more rows of each CTA
    float2* part_ml;               // [2 * kMaxPackedCtas][group] (max, sum)
    float* part_o;                 // [2 * kMaxPackedCtas][group][128]
    DeviceStatus st;
};
// A row (sequence, kv head) that lies in several CTAs of the line, with the first and last of them.
struct PackedCut {
    int32_t row, first, last;      // row -1: none
};
constexpr int kMaxPackedCtas = 512;
struct PackedLayout {
    size_t ml, o, bytes;           // offsets from the workspace (cuts at 256)
};
PackedLayout packed_layout(int group);
__host__ __device__ inline bool cuts_by_row(const PackedArgs& a, int ctas) {
    return static_cast<int64_t>(a.batch) * a.hkv <= ctas;
}
cudaError_t launch_packed_attention(const PackedArgs& a, int num_sms, cudaStream_t stream);

struct CopyArgs {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* n_pairs;        // nullable: max_pairs
    int max_pairs, num_pages, num_planes;
    DeviceStatus st;
    uint8_t* base[LOCKS_MAX_PLANES];
    int64_t page_bytes[LOCKS_MAX_PLANES];
};
cudaError_t launch_copy_pages(const CopyArgs& a, int num_sms, cudaStream_t stream);

// The page calls share one argument block; each uses the fields its comment names.
struct PoolArgs {
    const int32_t* page_table;     // fork, compact
    int32_t* page_table_out;       // fork, compact; take: the table itself
    const int32_t* seq_tokens;     // fork, take, compact
    const int32_t* new_tokens;     // take
    const int32_t* parents;        // fork
    int32_t* seq_tokens_out;       // fork, take
    const int32_t* refs;
    int32_t* refs_out;
    int32_t* list_src;             // fork: copy_src; compact: move_src
    int32_t* list_dst;
    int32_t* n_list;
    int32_t* n_free;               // take, nullable
    int32_t* new_page;             // compact
    const int32_t* lists;          // free: [rows][stride]
    const int32_t* counts;         // free
    int rows, stride;              // free
    int batch, max_pages, num_pages;
    // workspace regions (pool_layout)
    int32_t* needed;               // fork: fresh pages
    int32_t* block_counts;         // [kMaxPoolBlocks] free or used pages of each block of the pool
    int32_t* scan;                 // [batch] pages needed by rows 0..b
    int32_t* shift;                // take: [batch] from a page's rank to its place in the row
    int32_t* children;             // fork: [batch] rows that continue row p (the same region)
    int32_t* keeper;               // fork: [batch] the child that keeps p's last page
    int32_t* fresh;                // fork: [batch] row of the i-th fresh page
    uint8_t* flags;                // [pages / 4]: bits of the free pages
    DeviceStatus st;
};
constexpr int kMaxPoolBlocks = 512;
struct PoolLayout {
    size_t needed, block_counts, scan, shift, keeper, fresh, flags, bytes;
};
PoolLayout pool_layout(int batch, int pages);
cudaError_t launch_fork(const PoolArgs& a, cudaStream_t stream);
cudaError_t launch_take(const PoolArgs& a, cudaStream_t stream);
cudaError_t launch_compact(const PoolArgs& a, cudaStream_t stream);
cudaError_t launch_free(const PoolArgs& a, int num_sms, cudaStream_t stream);

// kernel<<<ctas, threads, smem>>> that may start while the kernel before it on the stream is
// still running (it has to call grid_dependency_wait before its first global access), in
// clusters of `cluster` CTAs where that is not 1.
template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel kernel, int64_t ctas, int threads, size_t smem, cudaStream_t stream, int cluster,
                             const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace locks
