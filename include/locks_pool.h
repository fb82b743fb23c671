/*
 * locks_pool.h - C ABI of a cache in 4 bits and of the page pool around it: packing full
 * pages to 4 bits and back, decode attention over packed pages (all of them, or the ones
 * locks_select_pages chose) with recent bf16 tokens behind them, and the pool's page calls:
 * copying pages, forking sequences, taking and freeing pages, compacting the pool.
 *
 * The conventions of locks.h and locks_cache.h hold for every call below: raw device
 * pointers that the caller owns, dims on the host, a cudaStream_t passed as void*, no
 * allocation and no host synchronisation (every call may be captured in a CUDA graph),
 * LOCKS_OK or a negative LOCKS_ERR_* code with argument errors found before anything is
 * launched, and device-side errors recorded in the status word at the start of the
 * workspace. Where the workspace is optional it may be NULL; device-side errors are then
 * not recorded. A workspace is scratch of one call at a time: calls that may overlap on the
 * GPU (other streams, other captured graphs) need one each.
 *
 * Two pools
 * ---------
 * The bf16 pool, k_cache and v_cache of dims->num_phys_pages pages, holds the pages that
 * are being filled. The packed pool holds full pages:
 *   packed  uint8 [num_packed_pages][num_kv_heads][LOCKS_PACKED_BYTES], 16-byte aligned
 * A sequence's full pages are entries of page_table that name packed pages, and its last
 * tokens lie in pages of the bf16 pool (recent_table). A page that fills is packed and its
 * bf16 page used again; summaries, being indexed by physical page, are those of the packed
 * page. Scoring, selection, mass and eviction go by the tables and take a packed pool's as
 * they are, with dims whose num_phys_pages is num_packed_pages.
 *
 * locks_build_summaries reads bf16 pages and writes at their ids. For summaries at the packed
 * pages' ids, the four summary arrays have num_packed_pages + num_phys_pages pages, first those
 * of the packed pool, then those of the bf16 pool:
 * - locks_build_summaries with the bf16 pool's dims and ids, and a locks_summaries_t of pointers
 *   num_packed_pages pages into the arrays;
 * - locks_copy_pages with the four whole arrays as planes, from num_packed_pages + bf16 page to
 *   packed page, and locks_pack_pages from and to the same pages;
 * - the arrays' fronts are what scoring and selection read, and what goes into the planes, beside
 *   the packed pages, when a fork or a compaction moves packed pages.
 *
 * Packed unit: one page of one kv head, LOCKS_PACKED_BYTES = 2432 bytes
 *   0     codes of the keys, 4 bits each      1024  codes of the values
 *   2048  for token t: bf16 scales of its key's 4 groups of 32 dims, then their zeros
 *   2304  for token t: bf16 scales of its value's 2 groups of 64 dims, then their zeros
 * value = zero + scale * code, code 0..15; scales may be of either sign. Codes lie in the order
 * in which the attention's tensor-core fragments read them. That of token t and dim d lies in the
 * four bits from bit b of the 32-bit word at byte 512 * (w / 4) + 16 * l + 4 * (w % 4) of its 1024,
 * w = d / 16:
 *   keys    l = 4 * (t % 8) + d % 8 / 2,  b = 16 * (d % 2) + 4 * (d / 8 % 2) + 8 * (t / 8)
 *   values  l = 4 * (d % 8) + t % 8 / 2,  b = 16 * (t % 2) + 4 * (d / 8 % 2) + 8 * (t / 8)
 *
 * Reference counts
 * ----------------
 *   refs  int32 [pages], 16-byte aligned: how many holders (rows of tables and whoever else)
 *         a page of a pool has, from -2^30 to 2^30. A page with refs <= 0 is free; there is no list
 *         of free pages.
 * A sequence of n tokens holds the first ceil(n / 16) pages of its row. Its full pages may be
 * shared with other rows, a page that is not full never is. The calls below keep it so.
 * Pages are always taken in ascending order of their ids, so that results repeat exactly.
 */
#ifndef LOCKS_POOL_H
#define LOCKS_POOL_H

#include "locks_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOCKS_PACKED_BYTES 2432
#define LOCKS_MAX_PLANES 128

enum {
    LOCKS_ERR_NO_PAGES = -7,           /* device: a pool has too few free pages */
};

/*
 * Packs pages: unit (dst_pages[i], h) of the packed pool from page src_pages[i] of the bf16
 * pool, i < n_pages, h < num_kv_heads. For every group (32 dims of a key, 64 of a value):
 *   zero  = the group's least value
 *   scale = bf16((greatest - least) / 15), 0 where that is below 2^-126
 *   code  = round((x - zero) / scale), ties to even; 0 where scale is 0
 * with the quotients rounded as fp32 division rounds them. A group with a NaN or an infinity
 * (or whose range overflows fp32) has a NaN for its scale and codes 0, and unpacks to no finite
 * value; other groups are not touched by it. dst_pages NULL: the same ids as src_pages. A negative
 * id in either list skips the entry; one out of range does too and records LOCKS_ERR_BAD_INDEX. No
 * packed page may be named twice in dst_pages.
 * workspace: optional, 256 bytes (status only). One launch.
 */
LOCKS_API int locks_pack_pages(const locks_dims_t* dims, const uint16_t* k_cache, const uint16_t* v_cache,
                               const int32_t* src_pages, const int32_t* dst_pages, int32_t n_pages, uint8_t* packed,
                               int32_t num_packed_pages, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Unpacks pages: page dst_pages[i] of the bf16 pool from page src_pages[i] of the packed pool,
 * bf16(zero + scale * code), rounded once, for pages that go on being read as bf16 ones (summaries
 * of another kind, shared-prefix attention). Lists, errors and workspace as for packing.
 */
LOCKS_API int locks_unpack_pages(const locks_dims_t* dims, const uint8_t* packed, int32_t num_packed_pages,
                                 const int32_t* src_pages, const int32_t* dst_pages, int32_t n_pages,
                                 uint16_t* k_cache, uint16_t* v_cache, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Workspace bytes of locks_packed_attention for these dims (256-byte aligned). */
LOCKS_API int locks_packed_workspace_size(const locks_dims_t* dims, size_t* bytes);

/*
 * Decode attention over packed pages and then recent bf16 tokens, in one softmax with scale
 * 1/sqrt(128). The tokens T_bh of sequence b for the query heads of kv head h are
 *   the 16 tokens of each packed page page_table[b][j], j < seq_pages[b], or, with
 *   `selected`, of pages page_table[b][selected[b][h][i]], i < n_selected[b][h];
 *   then recent tokens 0..recent_tokens[b) through recent_table[b]
 *   out[b][q] = sum_{t in T} softmax_t(q . k_t / sqrt(128)) v_t
 *   lse[b][q] = log sum_{t in T} exp(q . k_t / sqrt(128))
 * with keys and values as the units stand for them, exactly (nothing is rounded to bf16 in
 * between). No tokens at all: out = 0, lse = -inf. Rows behind the last recent token are never
 * used, whatever they hold. A NaN among the tokens' keys or values gives NaN to the rows that
 * attend to it, and so may an infinity.
 * - q: q_type LOCKS_FP32 or LOCKS_BF16, contiguous [batch][num_q_heads][128], 16-byte aligned,
 *   each head's of magnitudes from 2^-60 to 2^60 or 0. fp32 queries enter the products as two
 *   fp16 parts, 22 bits below each head's largest (over recent tokens as two bf16 parts, 16 bits).
 *   The weights times the values' scales enter rounded to 11 bits, each off by 2^-11 of itself or
 *   by 2^-21 of what a token of the largest weight would have, whichever is more, however far apart
 *   the scales of tokens and groups are (over recent tokens as two bf16 parts, 16 bits). Sums and
 *   softmax statistics are fp32. Keys and values of magnitudes up to 2^50 are served.
 * - page_table int32 [batch][max_pages_per_seq], ids of packed pages; not read when
 *   max_pages_per_seq is 0.
 * - selected int32 [batch][num_kv_heads][k_cap] (logical pages, in any order; the same one
 *   twice counts twice) with n_selected, as locks_select_pages writes them, or NULL; seq_pages
 *   is not read then and may be NULL. k_cap at least 1.
 * - recent_table int32 [batch][max_recent_pages], ids of bf16 pages, recent_tokens int32 [batch]
 *   in [0, 16 * max_recent_pages]; both not read, nor k_cache and v_cache, when
 *   max_recent_pages is 0 (num_phys_pages may then be 0 too).
 * - All counts, tables and lists are read on the device, so a captured graph may be replayed
 *   after they change. A count out of range counts as 0, a page id out of range is read as
 *   page 0; each records LOCKS_ERR_BAD_INDEX.
 * - out bf16 bits [batch][num_q_heads][128], 16-byte aligned; lse fp32, may be NULL.
 * - batch at most 65536.
 * One kernel launch, or two for long lists. The result depends on the batch and the widths of
 * the tables through rounding alone (the order in which parts of the softmax are joined), and
 * repeats exactly for the same arguments.
 */
LOCKS_API int locks_packed_attention(const locks_dims_t* dims, const void* q, int32_t q_type, const uint8_t* packed,
                                     int32_t num_packed_pages, const int32_t* page_table, const int32_t* seq_pages,
                                     const int32_t* selected, const int32_t* n_selected, int32_t k_cap,
                                     const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* recent_table,
                                     int32_t max_recent_pages, const int32_t* recent_tokens, uint16_t* out,
                                     float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Arrays that hold something of every page of a pool: of all layers the keys, the values, the
 * packed pages, the four arrays of the summaries. Page p of array i is the page_bytes[i] bytes
 * from base[i] + p * page_bytes[i]; both the base and page_bytes are multiples of 8. */
typedef struct {
    int32_t num_planes;                    /* 0..LOCKS_MAX_PLANES */
    int32_t num_pages;                     /* of every array */
    void* base[LOCKS_MAX_PLANES];          /* device */
    int64_t page_bytes[LOCKS_MAX_PLANES];
} locks_planes_t;

/*
 * Copies page src_pages[i] over page dst_pages[i] in every array, for all i < n: n = *n_pairs
 * (read on the device, in [0, max_pairs]; others record LOCKS_ERR_BAD_INDEX and copy nothing),
 * or max_pairs where n_pairs is NULL. No page may be named twice in dst_pages, nor in both
 * lists. A negative id in either list skips the pair; one out of range does too and records
 * LOCKS_ERR_BAD_INDEX. planes is a HOST pointer, read during the call.
 * workspace: optional, 256 bytes (status only). One launch.
 */
LOCKS_API int locks_copy_pages(const locks_planes_t* planes, const int32_t* src_pages, const int32_t* dst_pages,
                               int32_t max_pairs, const int32_t* n_pairs, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Workspace bytes of locks_fork_sequences, locks_take_pages and locks_compact_pages for these dims
 * (256-byte aligned). The pool they work on, of num_phys_pages pages, may have up to 2^30. */
LOCKS_API int locks_pool_workspace_size(const locks_dims_t* dims, size_t* bytes);

/*
 * Rows continue rows, all at once: row b of the new table continues row p = parents[b] of the
 * old one (itself where p = b; a beam's step, samples of one prompt), or is empty where
 * parents[b] is -1. With n = seq_tokens[p]:
 *   page_table_out[b][j] = page_table[p][j], j < n / 16 (full pages, shared)
 *   page_table_out[b][n / 16], if n % 16: the page itself for one of p's children (p, or else
 *       the first), for each other one a free page of its own
 *   seq_tokens_out[b] = n, 0 where parents[b] is -1; further entries are not written
 *   copy_src[i], copy_dst[i], i < *n_copies: the pages whose first n % 16 rows the caller has
 *       to copy (locks_copy_pages), in ascending order of b
 *   refs_out: refs with the old rows' holds let go and the new rows' added, 1 for the pages taken
 * Free are the pages with refs <= 0 before the call, taken in ascending order for ascending b;
 * pages that lose their last holder become free after it. Where there are too few,
 * LOCKS_ERR_NO_PAGES is recorded and the last ones go without: their rows keep the full pages
 * alone, seq_tokens_out[b] = n / 16 * 16.
 * - page_table, page_table_out int32 [batch][max_pages_per_seq], seq_tokens, seq_tokens_out,
 *   parents, copy_src, copy_dst int32 [batch], n_copies int32 [1], refs, refs_out int32
 *   [num_phys_pages]. refs_out may be refs; else no output may overlap an input or another output.
 * - num_phys_pages is the size of the pool that the table names pages of.
 * - seq_tokens out of [0, 16 * max_pages_per_seq] count as 0, a parent out of [-1, batch) as -1,
 *   a page id out of range is handed on and not counted; each records LOCKS_ERR_BAD_INDEX.
 * - batch at most 65536. Two launches, or one for small pools.
 */
LOCKS_API int locks_fork_sequences(const locks_dims_t* dims, const int32_t* page_table, const int32_t* seq_tokens,
                                   const int32_t* parents, const int32_t* refs, int32_t* page_table_out,
                                   int32_t* seq_tokens_out, int32_t* refs_out, int32_t* copy_src, int32_t* copy_dst,
                                   int32_t* n_copies, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sequences grow: row b, of seq_tokens[b] tokens, gets pages for new_tokens[b]:
 *   page_table[b][j], ceil(seq_tokens[b] / 16) <= j < ceil(new_tokens[b] / 16): free pages,
 *       in ascending order for ascending b and j; other entries are left as they are
 *   seq_tokens_out[b] = new_tokens[b];  refs_out = refs, 1 for the pages taken
 * A row whose pages are not all there any more gets none (nor do later ones that need any):
 * seq_tokens_out[b] = seq_tokens[b], and LOCKS_ERR_NO_PAGES is recorded. new_tokens[b] below
 * seq_tokens[b], or either out of [0, 16 * max_pages_per_seq], leaves the row as it is and
 * records LOCKS_ERR_BAD_INDEX.
 * - seq_tokens_out may be seq_tokens and refs_out refs; else no output may overlap another array.
 * - n_free (int32 [1], may be NULL) receives the number of pages that are free afterwards.
 * - batch at most 65536. Two launches, or one for small pools.
 */
LOCKS_API int locks_take_pages(const locks_dims_t* dims, int32_t* page_table, const int32_t* seq_tokens,
                               const int32_t* new_tokens, const int32_t* refs, int32_t* seq_tokens_out,
                               int32_t* refs_out, int32_t* n_free, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Holders let pages go: refs_out = refs less one for every time a page is among
 * pages[r][0..counts[r]), r < rows. The rows may be those of a page table with the page counts of
 * the sequences that end (0 for the others), or what locks_evict_pages evicted.
 * A count out of [0, stride] records LOCKS_ERR_BAD_INDEX and the row is skipped; so is an id
 * out of range, and a page that nobody holds any more (it stays at 0).
 * - pages int32 [rows][stride]; refs, refs_out int32 [num_pages]; refs_out may be refs, else may
 *   not overlap it. workspace: optional, 256 bytes (status only). One launch, two where refs_out
 *   is not refs.
 */
LOCKS_API int locks_free_pages(const int32_t* refs, int32_t num_pages, const int32_t* pages, int32_t stride,
                               const int32_t* counts, int32_t rows, int32_t* refs_out, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * The pages in use move to the front of the pool. With u pages of refs > 0, the used pages from
 * id u on move, in ascending order, to the free pages below u:
 *   move_src[i] -> move_dst[i], i < *n_moves: both ascending; the caller copies the pages
 *       (locks_copy_pages; no page is in both lists)
 *   new_page[p] = the new id of page p (p itself where it does not move), p < num_phys_pages
 *   page_table_out[b][j] = new_page[page_table[b][j]], j < ceil(seq_tokens[b] / 16); other
 *       entries are not written. Further tables go by new_page.
 *   refs_out = refs at the new ids, 0 from u on
 * - move_src, move_dst int32 [move_cap], move_cap >= num_phys_pages / 2 and at least 1; n_moves
 *   int32 [1]. page_table_out may be page_table and refs_out refs; else no output may overlap
 *   another array.
 * - seq_tokens out of [0, 16 * max_pages_per_seq] record LOCKS_ERR_BAD_INDEX and the row is not
 *   written; an id out of range is handed on and records it too.
 * Three launches, or one or two for small pools.
 */
LOCKS_API int locks_compact_pages(const locks_dims_t* dims, const int32_t* page_table, const int32_t* seq_tokens,
                                  const int32_t* refs, int32_t* page_table_out, int32_t* refs_out, int32_t* move_src,
                                  int32_t* move_dst, int32_t move_cap, int32_t* n_moves, int32_t* new_page,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOCKS_POOL_H */
