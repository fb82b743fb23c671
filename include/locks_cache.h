/*
 * locks_cache.h - C ABI of the paged-cache operators that surround the LOCKS
 * decode step (locks.h): filling the cache from a projection's output,
 * attention of a batch that shares prefixes, the attention mass kept per page,
 * and eviction of the pages of least mass.
 *
 * The conventions of locks.h hold for every call below: raw device pointers
 * that the caller owns, dims on the host, a cudaStream_t passed as void*, no
 * allocation and no host synchronisation (every call may be captured in a CUDA
 * graph), LOCKS_OK or a negative LOCKS_ERR_* code with argument errors found
 * before anything is launched, and device-side errors recorded in the status
 * word at the start of the workspace (locks_get_device_status). Where the
 * workspace is optional it may be NULL; device-side errors are then not recorded.
 * A workspace is scratch of one call at a time: calls that may overlap on the
 * GPU (other streams, other captured graphs) need one each. Pointers and
 * workspaces belong to the current device of the calling thread.
 */
#ifndef LOCKS_CACHE_H
#define LOCKS_CACHE_H

#include "locks.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOCKS_MAX_AXES 4

/* Element types of activations. */
enum { LOCKS_BF16 = 0, LOCKS_FP16 = 1, LOCKS_FP32 = 2 };

/*
 * Rotary positions. Pair i (0 <= i < rot_dim / 2) of a head is its elements
 * (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved is not 0; elements
 * from rot_dim on are not rotated. Pair i of token t turns by the angle
 * positions[axis[i]][t] * inv_freq[i]: one axis for plain text, several (time,
 * height, width) for images and video, in any assignment of pairs to axes.
 */
typedef struct {
    int32_t rot_dim;       /* 0, 16, 32, ... 128 */
    int32_t interleaved;   /* 0 or 1 */
    int32_t num_axes;      /* rows of positions, 1..LOCKS_MAX_AXES */
    float scale;           /* multiplies cos and sin (1: a plain rotation) */
    double inv_freq[64];   /* radians per position, from -4096 to 4096 */
    int32_t axis[64];      /* 0 <= axis[i] < num_axes */
} locks_rope_t;

/*
 * Fills the paged cache from a projection's output, with the norms of queries
 * and keys and the rotation of both on the way. For every token t < num_tokens
 * with cache_index[t] >= 0, with s = token_seq[t] (s = t when token_seq is
 * NULL; num_tokens <= batch then) and page = page_table[s][cache_index[t] / 16]:
 *   q_out[t][h]                       = rot(norm(q[t][h], q_weight))   h < num_q_heads
 *   k_cache[page][h][cache_index % 16] = bf16(rot(norm(k[t][h], k_weight)))  h < num_kv_heads
 *   v_cache[page][h][cache_index % 16] = bf16(v[t][h])
 *   norm(x, w) = x / sqrt(mean(x^2) + eps) * w; x itself where w is NULL
 * computed in fp32 and rounded once (nearest even); angles are reduced exactly,
 * so positions up to 2^31 - 1 lose nothing. It serves one token per sequence
 * (decode) and prompts of any length (prefill) alike.
 * - q, k, v: in_type, [num_tokens][heads][128] with q_stride / k_stride /
 *   v_stride elements from one token to the next (not negative), so that all
 *   three may be slices of one projection's output; 16-byte aligned rows.
 * - positions int32 [num_axes][num_tokens]; rope NULL: no rotation, positions
 *   are not read. rope is a HOST pointer, read during the call.
 * - q_weight, k_weight fp32 [128], 16-byte aligned, each may be NULL.
 * - q_out: q_type LOCKS_FP32 (as locks_decode_step takes it) or LOCKS_BF16,
 *   contiguous [num_tokens][num_q_heads][128], 16-byte aligned; it may not
 *   overlap q, k or v. q and q_out may both be NULL (keys and values only).
 * - A negative cache_index marks a row of padding: nothing is written for it,
 *   whatever it holds. A token_seq, cache_index or page id out of range records
 *   LOCKS_ERR_BAD_INDEX and nothing is written for that token.
 * - No two tokens of a call may name the same cache row: each of its 16-byte
 *   pieces would hold either token's values.
 * - workspace: optional, 256 bytes (status only).
 */
LOCKS_API int locks_append_tokens(const locks_dims_t* dims, const locks_rope_t* rope, const void* q, const void* k,
                                  const void* v, int32_t in_type, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, int32_t num_tokens, const int32_t* positions,
                                  const int32_t* token_seq, const int32_t* cache_index, const int32_t* page_table,
                                  const float* q_weight, const float* k_weight, float eps, void* q_out,
                                  int32_t q_type, uint16_t* k_cache, uint16_t* v_cache, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Workspace bytes of locks_prefix_attention for these dims and num_groups (256-byte aligned). */
LOCKS_API int locks_prefix_workspace_size(const locks_dims_t* dims, int32_t num_groups, size_t* bytes);

/*
 * Decode attention of a batch whose sequences share prefixes; each prefix is
 * read once for all its sequences. The sequences b of group i, group_start[i]
 * <= b < group_start[i + 1], attend to that group's prefix and then to tokens
 * of their own, in one softmax with scale 1/sqrt(128):
 *   T_b       = prefix tokens 0..prefix_tokens[i) through prefix_table[i],
 *               then own tokens 0..seq_tokens[b) through page_table[b]
 *   out[b][h] = sum_{t in T_b} softmax_t(q[b][h] . k_t / sqrt(128)) v_t
 *   lse[b][h] = log sum_t exp(q[b][h] . k_t / sqrt(128))
 * Sequences outside every group attend to their own tokens only. Both kinds of
 * tokens may end inside a page; rows behind the end are never used, whatever
 * they hold. No tokens at all: out = 0, lse = -inf.
 * - q: q_type LOCKS_FP32 or LOCKS_BF16, contiguous [batch][num_q_heads][128],
 *   16-byte aligned. fp32 queries, and the softmax weights where they meet the
 *   values, enter the products as a bf16 high and low part (about 16 significant
 *   bits); sums and softmax statistics are fp32.
 * - prefix_table int32 [num_groups][max_prefix_pages], prefix_tokens int32
 *   [num_groups] in [0, 16 * max_prefix_pages], group_start int32
 *   [num_groups + 1], not falling, in [0, batch]; seq_tokens int32 [batch] in
 *   [0, 16 * max_pages_per_seq]. All are read on the device, so a captured
 *   graph may be replayed after they change. A length out of range counts as
 *   0 and a group whose bounds fall, overlap an earlier group or leave
 *   [0, batch] as empty; an out-of-range page id is read as page 0; each
 *   records LOCKS_ERR_BAD_INDEX.
 * - num_groups >= 0 (0: no prefixes; the group arrays are not read) and at
 *   most 65536, batch at most 65536.
 * - page_table int32 [batch][max_pages_per_seq], not read when
 *   max_pages_per_seq is 0.
 * - out bf16 bits [batch][num_q_heads][128], 16-byte aligned; lse fp32, may be
 *   NULL.
 * One kernel launch, or two for long lists. Which form runs follows the batch,
 * the heads and the widths of the tables (max_prefix_pages and
 * max_pages_per_seq), so tables not much wider than the lists in them serve
 * best.
 * The result depends on which sequences share a prefix, on the batch and on
 * those widths through rounding alone (the order in which parts of the softmax
 * are joined), and repeats exactly for the same arguments.
 */
LOCKS_API int locks_prefix_attention(const locks_dims_t* dims, const void* q, int32_t q_type,
                                     const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* prefix_table,
                                     const int32_t* prefix_tokens, const int32_t* group_start, int32_t num_groups,
                                     int32_t max_prefix_pages, const int32_t* page_table, const int32_t* seq_tokens,
                                     uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Workspace bytes of locks_accumulate_mass for these dims (256-byte aligned). */
LOCKS_API int locks_mass_workspace_size(const locks_dims_t* dims, size_t* bytes);

/*
 * Adds one decode step's attention mass to the mass kept per page, from the
 * step's page scores (locks_score_pages, or locks_exact_scores for exact mass):
 *   L_bh           = log sum_{j < seq_pages[b]} exp(scores[b][h][j])
 *   mass_out[b][j] = decay * mass[b][j] + (1/Hq) sum_h exp(scores[b][h][j] - L_bh)
 * for j < seq_pages[b]; other entries are not written. A score that is NaN or
 * +inf adds nothing, neither to its page nor to L_bh; a head without any score
 * above -inf adds nothing.
 * - mass, mass_out: fp32 [batch][max_pages_per_seq]; mass_out may be mass itself
 *   (but may not overlap it otherwise). decay: finite; 1 sums, less forgets.
 *   With decay 0 the old mass is not read.
 * - lse_partials (may be NULL): the partials locks_score_pages wrote for these
 *   same scores, dims and seq_pages on this device; L_bh is then joined from them
 *   and the scores are read once instead of twice. What that call left of the
 *   buffer as it was is not read. (The scorer leaves a +inf score out of its sums
 *   together with the eight pages 8i .. 8i + 7 it lies among, so L_bh lacks those.)
 * - seq_pages[b] out of [0, max_pages_per_seq] records LOCKS_ERR_BAD_INDEX and
 *   the sequence is skipped. batch at most 65535, else LOCKS_ERR_UNSUPPORTED. Two
 *   kernel launches.
 */
LOCKS_API int locks_accumulate_mass(const locks_dims_t* dims, const float* scores, const float* lse_partials,
                                    const int32_t* seq_pages, const float* mass, float* mass_out, float decay,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Evicts the pages of least mass until keep_pages are left. For every sequence
 * with n = seq_pages[b] > keep_pages, the e = n - keep_pages pages of least
 * mass among sink_pages <= j < n - recent_pages leave (equal masses: the lower
 * page first; NaN counts as less than any number; -0 equals 0), e = 0
 * otherwise. The others keep their order and close up, with the extra_pages
 * table entries behind them (the pages of a tail without summaries, which are
 * never evicted; entries past max_pages_per_seq do not exist):
 *   page_table_out[b][i], mass_out[b][i] = the i-th kept page's entries,
 *       i < min(n + extra_pages, max_pages_per_seq) - e (others not written)
 *   evicted[b][i]    = physical page of the i-th evicted page, in ascending
 *                      logical order, i < e (others not written)
 *   n_evicted[b] = e,  seq_pages_out[b] = n - e
 * Summaries and cache rows belong to physical pages and stay where they are;
 * the caller may reuse the evicted ones. Keys keep the positions they were
 * rotated by.
 * - evicted: int32 [batch][evict_cap], evict_cap >= max_pages_per_seq -
 *   keep_pages, at least 1.
 * - page_table_out, mass_out and seq_pages_out may each be the input itself (in
 *   place) but may not overlap it otherwise.
 * - keep_pages >= sink_pages + recent_pages, none of them negative; 0 <=
 *   extra_pages. max_pages_per_seq at most 393216, else LOCKS_ERR_UNSUPPORTED.
 * - seq_pages[b] out of [0, max_pages_per_seq] records LOCKS_ERR_BAD_INDEX;
 *   n_evicted[b] is then 0 and nothing else is written for the sequence.
 * - workspace: optional, 256 bytes (status only). One launch.
 */
LOCKS_API int locks_evict_pages(const locks_dims_t* dims, const float* mass, const int32_t* page_table,
                                const int32_t* seq_pages, int32_t keep_pages, int32_t sink_pages,
                                int32_t recent_pages, int32_t extra_pages, float* mass_out,
                                int32_t* page_table_out, int32_t* seq_pages_out, int32_t* evicted,
                                int32_t evict_cap, int32_t* n_evicted, void* workspace, size_t workspace_bytes,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOCKS_CACHE_H */
