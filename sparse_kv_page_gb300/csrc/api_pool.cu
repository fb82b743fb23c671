// api_pool.cu - the C ABI of include/locks_pool.h: argument validation, workspace layout and
// kernel launches of the packed cache and the page pool. No allocation and no host
// synchronisation.
#include <climits>
#include <cstring>
#include <initializer_list>

#include "pool_internal.h"

namespace {

constexpr int kMaxBatch = 65536;
constexpr int kMaxPoolPages = 1 << 30;    // pages are counted a few rounds past the pool's end in int32
constexpr size_t kStatusBytes = 256;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return LOCKS_OK;
    cudaGetLastError();
    return LOCKS_ERR_CUDA;
}

struct Buffer {
    const void* p;
    size_t bytes;
    const void* may_be = nullptr;      // an output: the input that it may be
};
Buffer ints(const void* p, int64_t n, const void* may_be = nullptr) {
    return {p, static_cast<size_t>(n) * sizeof(int32_t), may_be};
}
// No output overlaps an input (but the one that it may be) or another output.
bool apart(std::initializer_list<Buffer> in, std::initializer_list<Buffer> out) {
    const auto overlap = [](const Buffer& a, const Buffer& b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
    };
    for (const Buffer* o = out.begin(); o != out.end(); ++o) {
        for (const Buffer& i : in)
            if (overlap(*o, i) && !(o->p == i.p && o->may_be == i.p)) return false;
        for (const Buffer* other = out.begin(); other != o; ++other)
            if (overlap(*o, *other)) return false;
    }
    return true;
}
bool words(std::initializer_list<const void*> all) {
    for (const void* p : all)
        if (!aligned(p, 4)) return false;
    return true;
}

// dims of the packed attention: num_phys_pages, the bf16 pool's, may be 0 where no recent tokens
// are given.
int check_packed(const locks_dims_t* d) {
    if (!d) return LOCKS_ERR_INVALID_ARG;
    locks_dims_t x = *d;
    if (x.num_phys_pages == 0) x.num_phys_pages = 1;
    const int s = locks::check_dims(&x);
    return s == LOCKS_OK && x.batch > kMaxBatch ? LOCKS_ERR_UNSUPPORTED : s;
}

// What the calls that change tables have in common. Counts of tokens are int32, and a block
// takes 4096 entries of a row.
int check_table(const locks_dims_t* d) {
    const int s = locks::check_dims(d);
    if (s != LOCKS_OK) return s;
    if (d->batch > kMaxBatch || d->max_pages_per_seq > INT_MAX / LOCKS_PAGE_SIZE) return LOCKS_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->batch) * (d->max_pages_per_seq / 4096 + 1) > INT_MAX / 2) return LOCKS_ERR_UNSUPPORTED;
    if (d->num_phys_pages > kMaxPoolPages) return LOCKS_ERR_UNSUPPORTED;
    return LOCKS_OK;
}

locks::PoolArgs pool_args(const locks_dims_t* d, void* workspace) {
    locks::PoolArgs a;
    std::memset(&a, 0, sizeof(a));
    a.batch = d->batch;
    a.max_pages = d->max_pages_per_seq;
    a.num_pages = d->num_phys_pages;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const locks::PoolLayout w = locks::pool_layout(d->batch, d->num_phys_pages);
    a.needed = reinterpret_cast<int32_t*>(base + w.needed);
    a.block_counts = reinterpret_cast<int32_t*>(base + w.block_counts);
    a.scan = reinterpret_cast<int32_t*>(base + w.scan);
    a.shift = reinterpret_cast<int32_t*>(base + w.shift);
    a.children = a.shift;
    a.keeper = reinterpret_cast<int32_t*>(base + w.keeper);
    a.fresh = reinterpret_cast<int32_t*>(base + w.fresh);
    a.flags = base + w.flags;
    a.st = locks::device_status(workspace);
    return a;
}

int check_pages(const locks_dims_t* dims, const uint16_t* k_cache, const uint16_t* v_cache, const uint8_t* packed,
                int32_t num_packed_pages, const int32_t* src, const int32_t* dst, int32_t n, void* workspace,
                size_t workspace_bytes) {
    int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (n < 0 || num_packed_pages < 0) return LOCKS_ERR_INVALID_ARG;
    if (workspace && (s = locks::check_workspace(workspace, workspace_bytes, kStatusBytes)) != LOCKS_OK) return s;
    if (n == 0) return LOCKS_OK;
    if (!k_cache || !v_cache || !packed || !src) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(packed, 16) || !words({src, dst}))
        return LOCKS_ERR_INVALID_ARG;
    return LOCKS_OK;
}

}  // namespace

extern "C" {

int locks_pack_pages(const locks_dims_t* dims, const uint16_t* k_cache, const uint16_t* v_cache,
                     const int32_t* src_pages, const int32_t* dst_pages, int32_t n_pages, uint8_t* packed,
                     int32_t num_packed_pages, void* workspace, size_t workspace_bytes, void* stream) {
    const int s = check_pages(dims, k_cache, v_cache, packed, num_packed_pages, src_pages, dst_pages, n_pages, workspace,
                              workspace_bytes);
    if (s != LOCKS_OK || n_pages == 0) return s;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    const locks::PackArgs a = {k_cache,   v_cache,   nullptr,  nullptr, packed, src_pages,
                               dst_pages, n_pages,   dims->num_kv_heads, dims->num_phys_pages, num_packed_pages,
                               locks::device_status(workspace)};
    return cuda_status(locks::launch_pack(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_unpack_pages(const locks_dims_t* dims, const uint8_t* packed, int32_t num_packed_pages,
                       const int32_t* src_pages, const int32_t* dst_pages, int32_t n_pages, uint16_t* k_cache,
                       uint16_t* v_cache, void* workspace, size_t workspace_bytes, void* stream) {
    const int s = check_pages(dims, k_cache, v_cache, packed, num_packed_pages, src_pages, dst_pages, n_pages, workspace,
                              workspace_bytes);
    if (s != LOCKS_OK || n_pages == 0) return s;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    const locks::PackArgs a = {nullptr,   nullptr, k_cache, v_cache, const_cast<uint8_t*>(packed), src_pages,
                               dst_pages, n_pages, dims->num_kv_heads, num_packed_pages, dims->num_phys_pages,
                               locks::device_status(workspace)};
    return cuda_status(locks::launch_unpack(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_packed_workspace_size(const locks_dims_t* dims, size_t* bytes) {
    if (!bytes) return LOCKS_ERR_INVALID_ARG;
    const int s = check_packed(dims);
    if (s != LOCKS_OK) return s;
    *bytes = locks::packed_layout(dims->num_q_heads / dims->num_kv_heads).bytes;
    return LOCKS_OK;
}

int locks_packed_attention(const locks_dims_t* dims, const void* q, int32_t q_type, const uint8_t* packed,
                           int32_t num_packed_pages, const int32_t* page_table, const int32_t* seq_pages,
                           const int32_t* selected, const int32_t* n_selected, int32_t k_cap, const uint16_t* k_cache,
                           const uint16_t* v_cache, const int32_t* recent_table, int32_t max_recent_pages,
                           const int32_t* recent_tokens, uint16_t* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    int s = check_packed(dims);
    if (s != LOCKS_OK) return s;
    if (q_type != LOCKS_FP32 && q_type != LOCKS_BF16) return LOCKS_ERR_INVALID_ARG;
    if (num_packed_pages < 0 || max_recent_pages < 0 || (selected && k_cap < 1)) return LOCKS_ERR_INVALID_ARG;
    // steps of a row are int32
    if (max_recent_pages > INT_MAX / LOCKS_PAGE_SIZE / 2 || dims->max_pages_per_seq > INT_MAX / 4 || (selected && k_cap > INT_MAX / 4))
        return LOCKS_ERR_UNSUPPORTED;
    const locks::PackedLayout w = locks::packed_layout(dims->num_q_heads / dims->num_kv_heads);
    if ((s = locks::check_workspace(workspace, workspace_bytes, w.bytes)) != LOCKS_OK) return s;
    if (dims->batch == 0) return LOCKS_OK;
    if (!q || !out) return LOCKS_ERR_INVALID_ARG;
    if (selected ? !n_selected : !seq_pages) return LOCKS_ERR_INVALID_ARG;
    // pages are read wherever a list may have some; a bad id is read as page 0
    if ((selected || dims->max_pages_per_seq > 0) && (!packed || num_packed_pages < 1)) return LOCKS_ERR_INVALID_ARG;
    if (dims->max_pages_per_seq > 0 && !page_table) return LOCKS_ERR_INVALID_ARG;
    if (max_recent_pages > 0 && (!k_cache || !v_cache || !recent_table || !recent_tokens || dims->num_phys_pages < 1))
        return LOCKS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(packed, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !words({page_table, seq_pages, selected, n_selected, recent_table, recent_tokens, lse}))
        return LOCKS_ERR_INVALID_ARG;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    locks::PackedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.packed = packed;
    a.page_table = page_table;
    a.seq_pages = seq_pages;
    a.selected = selected;
    a.n_selected = n_selected;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.recent_table = recent_table;
    a.recent_tokens = recent_tokens;
    a.out = out;
    a.lse = lse;
    a.q_type = q_type;
    a.k_cap = k_cap;
    a.max_recent = max_recent_pages;
    a.batch = dims->batch;
    a.hq = dims->num_q_heads;
    a.hkv = dims->num_kv_heads;
    a.group = a.hq / a.hkv;
    a.max_pages = dims->max_pages_per_seq;
    a.num_packed = num_packed_pages;
    a.num_cache = dims->num_phys_pages;
    a.cuts = reinterpret_cast<locks::PackedCut*>(base + kStatusBytes);
    a.part_ml = reinterpret_cast<float2*>(base + w.ml);
    a.part_o = reinterpret_cast<float*>(base + w.o);
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_packed_attention(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_copy_pages(const locks_planes_t* planes, const int32_t* src_pages, const int32_t* dst_pages,
                     int32_t max_pairs, const int32_t* n_pairs, void* workspace, size_t workspace_bytes,
                     void* stream) {
    if (!planes) return LOCKS_ERR_INVALID_ARG;
    if (planes->num_planes < 0 || planes->num_planes > LOCKS_MAX_PLANES || planes->num_pages < 0 || max_pairs < 0)
        return LOCKS_ERR_INVALID_ARG;
    int s;
    if (workspace && (s = locks::check_workspace(workspace, workspace_bytes, kStatusBytes)) != LOCKS_OK) return s;
    locks::CopyArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int i = 0; i < planes->num_planes; ++i) {
        const int64_t bytes = planes->page_bytes[i];
        if (bytes < 0 || bytes % 8 != 0 || bytes > INT64_MAX / INT_MAX) return LOCKS_ERR_INVALID_ARG;
        if (bytes > 0 && !planes->base[i]) return LOCKS_ERR_INVALID_ARG;
        if (!aligned(planes->base[i], 8)) return LOCKS_ERR_INVALID_ARG;
        a.base[i] = static_cast<uint8_t*>(planes->base[i]);
        a.page_bytes[i] = bytes;
        a.num_planes += 1;
    }
    const bool nothing = max_pairs == 0 || a.num_planes == 0;
    if (nothing && !n_pairs) return LOCKS_OK;
    if (!nothing && (!src_pages || !dst_pages)) return LOCKS_ERR_INVALID_ARG;
    if (!words({src_pages, dst_pages, n_pairs})) return LOCKS_ERR_INVALID_ARG;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    a.src = src_pages;
    a.dst = dst_pages;
    a.n_pairs = n_pairs;
    a.max_pairs = max_pairs;
    a.num_pages = planes->num_pages;
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_copy_pages(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_pool_workspace_size(const locks_dims_t* dims, size_t* bytes) {
    if (!bytes) return LOCKS_ERR_INVALID_ARG;
    const int s = check_table(dims);
    if (s != LOCKS_OK) return s;
    *bytes = locks::pool_layout(dims->batch, dims->num_phys_pages).bytes;
    return LOCKS_OK;
}

int locks_fork_sequences(const locks_dims_t* dims, const int32_t* page_table, const int32_t* seq_tokens,
                         const int32_t* parents, const int32_t* refs, int32_t* page_table_out,
                         int32_t* seq_tokens_out, int32_t* refs_out, int32_t* copy_src, int32_t* copy_dst,
                         int32_t* n_copies, void* workspace, size_t workspace_bytes, void* stream) {
    int s = check_table(dims);
    if (s != LOCKS_OK) return s;
    if ((s = locks::check_workspace(workspace, workspace_bytes, locks::pool_layout(dims->batch, dims->num_phys_pages).bytes)) != LOCKS_OK)
        return s;
    if (!n_copies) return LOCKS_ERR_INVALID_ARG;
    const int64_t batch = dims->batch, cells = batch * dims->max_pages_per_seq, pages = dims->num_phys_pages;
    if (batch > 0 && (!seq_tokens || !parents || !seq_tokens_out || !copy_src || !copy_dst)) return LOCKS_ERR_INVALID_ARG;
    if (cells > 0 && (!page_table || !page_table_out)) return LOCKS_ERR_INVALID_ARG;
    if (pages > 0 && (!refs || !refs_out)) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(refs, 16) || !aligned(refs_out, 16) ||
        !words({page_table, seq_tokens, parents, page_table_out, seq_tokens_out, copy_src, copy_dst, n_copies}))
        return LOCKS_ERR_INVALID_ARG;
    if (!apart({ints(page_table, cells), ints(seq_tokens, batch), ints(parents, batch), ints(refs, pages)},
               {ints(page_table_out, cells), ints(seq_tokens_out, batch), ints(refs_out, pages, refs),
                ints(copy_src, batch), ints(copy_dst, batch), ints(n_copies, 1)}))
        return LOCKS_ERR_INVALID_ARG;
    if (locks::current_sms() <= 0) return LOCKS_ERR_CUDA;
    locks::PoolArgs a = pool_args(dims, workspace);
    a.page_table = page_table;
    a.page_table_out = page_table_out;
    a.seq_tokens = seq_tokens;
    a.parents = parents;
    a.seq_tokens_out = seq_tokens_out;
    a.refs = refs;
    a.refs_out = refs_out;
    a.list_src = copy_src;
    a.list_dst = copy_dst;
    a.n_list = n_copies;
    return cuda_status(locks::launch_fork(a, static_cast<cudaStream_t>(stream)));
}

int locks_take_pages(const locks_dims_t* dims, int32_t* page_table, const int32_t* seq_tokens,
                     const int32_t* new_tokens, const int32_t* refs, int32_t* seq_tokens_out, int32_t* refs_out,
                     int32_t* n_free, void* workspace, size_t workspace_bytes, void* stream) {
    int s = check_table(dims);
    if (s != LOCKS_OK) return s;
    if ((s = locks::check_workspace(workspace, workspace_bytes, locks::pool_layout(dims->batch, dims->num_phys_pages).bytes)) != LOCKS_OK)
        return s;
    const int64_t batch = dims->batch, cells = batch * dims->max_pages_per_seq, pages = dims->num_phys_pages;
    if (batch > 0 && (!seq_tokens || !new_tokens || !seq_tokens_out)) return LOCKS_ERR_INVALID_ARG;
    if (cells > 0 && !page_table) return LOCKS_ERR_INVALID_ARG;
    if (pages > 0 && (!refs || !refs_out)) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(refs, 16) || !aligned(refs_out, 16) ||
        !words({page_table, seq_tokens, new_tokens, seq_tokens_out, n_free}))
        return LOCKS_ERR_INVALID_ARG;
    if (!apart({ints(seq_tokens, batch), ints(new_tokens, batch), ints(refs, pages)},
               {ints(page_table, cells), ints(seq_tokens_out, batch, seq_tokens), ints(refs_out, pages, refs),
                ints(n_free, 1)}))
        return LOCKS_ERR_INVALID_ARG;
    if (locks::current_sms() <= 0) return LOCKS_ERR_CUDA;
    locks::PoolArgs a = pool_args(dims, workspace);
    a.page_table_out = page_table;
    a.seq_tokens = seq_tokens;
    a.new_tokens = new_tokens;
    a.seq_tokens_out = seq_tokens_out;
    a.refs = refs;
    a.refs_out = refs_out;
    a.n_free = n_free;
    return cuda_status(locks::launch_take(a, static_cast<cudaStream_t>(stream)));
}

int locks_free_pages(const int32_t* refs, int32_t num_pages, const int32_t* pages, int32_t stride,
                     const int32_t* counts, int32_t rows, int32_t* refs_out, void* workspace, size_t workspace_bytes,
                     void* stream) {
    int s;
    if (num_pages < 0 || stride < 0 || rows < 0) return LOCKS_ERR_INVALID_ARG;
    if (stride > INT_MAX / 2 || num_pages > kMaxPoolPages) return LOCKS_ERR_UNSUPPORTED;
    if (workspace && (s = locks::check_workspace(workspace, workspace_bytes, kStatusBytes)) != LOCKS_OK) return s;
    const int64_t cells = static_cast<int64_t>(rows) * stride;
    if (num_pages > 0 && (!refs || !refs_out)) return LOCKS_ERR_INVALID_ARG;
    if (rows > 0 && !counts) return LOCKS_ERR_INVALID_ARG;
    if (cells > 0 && !pages) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(refs, 16) || !aligned(refs_out, 16) || !words({pages, counts})) return LOCKS_ERR_INVALID_ARG;
    if (!apart({ints(refs, num_pages), ints(pages, cells), ints(counts, rows)}, {ints(refs_out, num_pages, refs)}))
        return LOCKS_ERR_INVALID_ARG;
    if (num_pages == 0 && rows == 0) return LOCKS_OK;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    locks::PoolArgs a;
    std::memset(&a, 0, sizeof(a));
    a.refs = refs;
    a.refs_out = refs_out;
    a.lists = pages;
    a.counts = counts;
    a.rows = rows;
    a.stride = stride;
    a.num_pages = num_pages;
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_free(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_compact_pages(const locks_dims_t* dims, const int32_t* page_table, const int32_t* seq_tokens,
                        const int32_t* refs, int32_t* page_table_out, int32_t* refs_out, int32_t* move_src,
                        int32_t* move_dst, int32_t move_cap, int32_t* n_moves, int32_t* new_page, void* workspace,
                        size_t workspace_bytes, void* stream) {
    int s = check_table(dims);
    if (s != LOCKS_OK) return s;
    if ((s = locks::check_workspace(workspace, workspace_bytes, locks::pool_layout(dims->batch, dims->num_phys_pages).bytes)) != LOCKS_OK)
        return s;
    const int64_t batch = dims->batch, cells = batch * dims->max_pages_per_seq, pages = dims->num_phys_pages;
    if (move_cap < 1 || move_cap < pages / 2) return LOCKS_ERR_INVALID_ARG;
    if (!n_moves || !move_src || !move_dst || (batch > 0 && !seq_tokens)) return LOCKS_ERR_INVALID_ARG;
    if (cells > 0 && (!page_table || !page_table_out)) return LOCKS_ERR_INVALID_ARG;
    if (pages > 0 && (!refs || !refs_out || !new_page)) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(refs, 16) || !aligned(refs_out, 16) ||
        !words({page_table, seq_tokens, page_table_out, move_src, move_dst, n_moves, new_page}))
        return LOCKS_ERR_INVALID_ARG;
    if (!apart({ints(page_table, cells), ints(seq_tokens, batch), ints(refs, pages)},
               {ints(page_table_out, cells, page_table), ints(refs_out, pages, refs), ints(move_src, move_cap),
                ints(move_dst, move_cap), ints(n_moves, 1), ints(new_page, pages)}))
        return LOCKS_ERR_INVALID_ARG;
    if (locks::current_sms() <= 0) return LOCKS_ERR_CUDA;
    locks::PoolArgs a = pool_args(dims, workspace);
    a.page_table = page_table;
    a.page_table_out = page_table_out;
    a.seq_tokens = seq_tokens;
    a.refs = refs;
    a.refs_out = refs_out;
    a.list_src = move_src;
    a.list_dst = move_dst;
    a.n_list = n_moves;
    a.new_page = new_page;
    return cuda_status(locks::launch_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
