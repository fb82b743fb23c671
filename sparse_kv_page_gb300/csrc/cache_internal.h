// cache_internal.h - launchers of the paged-cache operators (locks_cache.h), and the
// argument checks of the C ABI that their entry points share with api.cu.
#pragma once

#include "../../include/locks_cache.h"
#include "locks_internal.h"

namespace locks {

// ------------------------------------------------- shared argument checks (api.cu)
int check_dims(const locks_dims_t* d);
int check_workspace(void* ws, size_t bytes, size_t need);
int current_sms();                       // SMs of the current device; 0: no device
DeviceStatus device_status(void* ws);    // with the process's wait limit
// Where locks_score_pages puts its (max, sum exp) pairs, on a device of `sms` SMs: [batch][query
// head][grid][warps]. A sequence is `chunks` items (sequence b the items from b * chunks on), and
// scorer CTA c has items c * per .. (c + 1) * per and writes the pairs of the sequences they
// belong to, no others.
struct ScorerSlots {
    int grid, warps, chunks, per;
};
ScorerSlots scorer_slots(const locks_dims_t* d, int sms);

// ------------------------------------------------------------------ launchers
struct AppendArgs {
    const void* q;               // nullable, with q_out
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;   // elements per token
    const int32_t* positions;    // [axes][num_tokens]
    const int32_t* token_seq;    // nullable
    const int32_t* cache_index;
    const int32_t* page_table;
    const float* q_weight;       // nullable
    const float* k_weight;       // nullable
    float eps;
    void* q_out;
    uint16_t* k_cache;
    uint16_t* v_cache;
    int num_tokens, batch, hq, hkv, max_pages, num_phys;
    int in_type, q_type;
    int rot_dim, interleaved;    // rot_dim 0: no rotation
    float rope_scale;
    uint64_t turns[64];          // pair i: inv_freq / (2 pi) turns per position, as a fraction of 2^64 (wraps)
    uint8_t axis[64];
    DeviceStatus st;
};
cudaError_t launch_append(const AppendArgs& a, int num_sms, cudaStream_t stream);

struct MassArgs {
    const float* scores;
    const int32_t* seq_pages;
    const float* mass;
    float* mass_out;
    float decay;
    int batch, hq, max_pages;
    const float2* partials;      // [batch][hq][row]
    int row;
    DeviceStatus st;
};
// Pairs per (sequence, query head) that launch_mass_partials writes.
int mass_partials_row(int max_pages);
cudaError_t launch_mass_partials(const MassArgs& a, float2* partials, cudaStream_t stream);
// Joins the scorer's pairs of each (sequence, query head) to one.
cudaError_t launch_mass_reduce(const float2* in, const ScorerSlots& slots, const MassArgs& a, float2* out,
                               cudaStream_t stream);
// Follows one of the two on the same stream.
cudaError_t launch_mass(const MassArgs& a, cudaStream_t stream);

struct EvictArgs {
    const float* mass;
    const int32_t* page_table;
    const int32_t* seq_pages;
    float* mass_out;
    int32_t* page_table_out;
    int32_t* seq_pages_out;
    int32_t* evicted;
    int32_t* n_evicted;
    int batch, max_pages, keep, sink, recent, extra, evict_cap;
    DeviceStatus st;
};
constexpr int kMaxEvictPages = 393216;
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace locks

namespace locks {

struct PrefixArgs {
    const void* q;                 // fp32 or bf16 [batch][hq][128]
    const uint16_t* k_cache;
    const uint16_t* v_cache;
    const int32_t* prefix_table;   // [num_groups][max_prefix_pages]
    const int32_t* prefix_tokens;  // [num_groups]
    const int32_t* group_start;    // [num_groups + 1]
    const int32_t* page_table;     // [batch][max_pages]
    const int32_t* seq_tokens;     // [batch]
    uint16_t* out;
    float* lse;                    // nullable
    int num_groups, max_prefix_pages, batch, hq, hkv, max_pages, num_phys, q_type;
    int group;                     // hq / hkv
    bool own_apart;                // the second launch attends to the sequences' own tokens
    bool own_alone;                // ... and to the prefixes: there is no first
    // workspace regions (prefix_layout)
    int64_t* total;                // steps of the whole call
    struct PrefixSeq* seqs;        // [batch]
    float2* part_ml;               // (max, sum) of either softmax group per partial row
    float* part_o;                 // [partial row][128]
    DeviceStatus st;
    CUtensorMap tm_k, tm_v;        // 64 x 16 boxes with 128-byte swizzle (filled by the launcher)
};
// Where a sequence's own tokens and its group's prefix lie on the line of all steps and on
// the line of all partial rows (written by the first launch for the second).
struct PrefixSeq {
    int64_t own_step0, pre_step0;
    int32_t own_row0, own_tiles;
    int32_t pre_row0, pre_tiles, pre_seq0, pre_num_seqs;   // pre_tiles 0: no prefix
};
constexpr int kMaxPrefixCtas = 256;
struct PrefixLayout {
    size_t seqs, ml, o, bytes;    // offsets from the workspace (total at 256)
};
PrefixLayout prefix_layout(int batch, int hq);
cudaError_t launch_prefix(const PrefixArgs& a, int num_sms, cudaStream_t stream);
// A cache [num_phys][hkv][16][128] as num_phys * hkv * 16 rows, in 64 x 16 boxes with 128-byte
// swizzle.
cudaError_t cache_map(CUtensorMap* map, const uint16_t* base, int64_t rows);
// By pages (prefix_pages.cu): one launch of clusters for few sequences, one of single CTAs for
// short lists, and a second launch that attends to own tokens and joins the prefix's partials
// to them.
bool prefix_is_small(const PrefixArgs& a, int num_sms);
cudaError_t launch_prefix_small(const PrefixArgs& a, int num_sms, cudaStream_t stream);
bool list_by_pages(const PrefixArgs& a, int num_sms);
bool own_by_pages(const PrefixArgs& a, int num_sms);
cudaError_t launch_own(const PrefixArgs& a, int grid, cudaStream_t stream);

}  // namespace locks
