// api_cache.cu - the C ABI of include/locks_cache.h: argument validation, workspace
// layout and kernel launches of the paged-cache operators. No allocation and no host
// synchronisation.
#include <climits>
#include <cmath>
#include <cstring>

#include "cache_internal.h"
#include "rope_turns.h"

namespace {

constexpr int kMaxBatch = 65536;          // tables of the prefix call; grids of the others take less
constexpr size_t kStatusBytes = 256;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return LOCKS_OK;
    cudaGetLastError();
    return LOCKS_ERR_CUDA;
}
int type_bytes(int32_t t) { return t == LOCKS_FP32 ? 4 : 2; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}
// Two buffers that are the same one or have nothing in common.
bool same_or_apart(const void* a, const void* b, size_t bytes) { return a == b || !overlap(a, bytes, b, bytes); }

struct MassLayout {
    size_t partials, total;
};
MassLayout mass_layout(const locks_dims_t* d) {
    MassLayout w;
    w.partials = kStatusBytes;
    w.total = w.partials + static_cast<size_t>(d->batch) * d->num_q_heads *
                               locks::mass_partials_row(d->max_pages_per_seq) * sizeof(float2);
    return w;
}

}  // namespace

extern "C" {

int locks_append_tokens(const locks_dims_t* dims, const locks_rope_t* rope, const void* q, const void* k,
                        const void* v, int32_t in_type, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                        int32_t num_tokens, const int32_t* positions, const int32_t* token_seq,
                        const int32_t* cache_index, const int32_t* page_table, const float* q_weight,
                        const float* k_weight, float eps, void* q_out, int32_t q_type, uint16_t* k_cache,
                        uint16_t* v_cache, void* workspace, size_t workspace_bytes, void* stream) {
    int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (num_tokens < 0) return LOCKS_ERR_INVALID_ARG;
    if (in_type < LOCKS_BF16 || in_type > LOCKS_FP32) return LOCKS_ERR_INVALID_ARG;
    if (q_type != LOCKS_FP32 && q_type != LOCKS_BF16) return LOCKS_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return LOCKS_ERR_INVALID_ARG;
    if (rope) {
        if (rope->rot_dim < 0 || rope->rot_dim > LOCKS_HEAD_DIM) return LOCKS_ERR_INVALID_ARG;
        if (rope->rot_dim % 16 != 0) return LOCKS_ERR_UNSUPPORTED;
        if (rope->num_axes < 1 || rope->num_axes > LOCKS_MAX_AXES) return LOCKS_ERR_INVALID_ARG;
        if (rope->interleaved != 0 && rope->interleaved != 1) return LOCKS_ERR_INVALID_ARG;
        if (!std::isfinite(rope->scale)) return LOCKS_ERR_INVALID_ARG;
        for (int i = 0; i < rope->rot_dim / 2; ++i)
            if (!std::isfinite(rope->inv_freq[i]) || std::fabs(rope->inv_freq[i]) > 4096.0 || rope->axis[i] < 0 ||
                rope->axis[i] >= rope->num_axes)
                return LOCKS_ERR_INVALID_ARG;
    }
    if (workspace && (s = locks::check_workspace(workspace, workspace_bytes, kStatusBytes)) != LOCKS_OK) return s;
    if (num_tokens == 0) return LOCKS_OK;
    if (!token_seq && num_tokens > dims->batch) return LOCKS_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr)) return LOCKS_ERR_INVALID_ARG;
    const bool turned = rope && rope->rot_dim > 0;
    if (!k || !v || !cache_index || !page_table || !k_cache || !v_cache || (turned && !positions))
        return LOCKS_ERR_INVALID_ARG;
    const int size = type_bytes(in_type);
    const int64_t strides[3] = {q ? q_stride : 0, k_stride, v_stride};
    for (int64_t st : strides)
        if (st < 0 || st > INT64_MAX / 16 / num_tokens || (st * size) % 16 != 0) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
        return LOCKS_ERR_INVALID_ARG;
    if (q) {
        const size_t out_bytes =
            static_cast<size_t>(num_tokens) * dims->num_q_heads * LOCKS_HEAD_DIM * type_bytes(q_type);
        const auto span = [&](int64_t stride, int heads) {
            return (static_cast<size_t>(num_tokens - 1) * stride + static_cast<size_t>(heads) * LOCKS_HEAD_DIM) * size;
        };
        if (overlap(q_out, out_bytes, q, span(q_stride, dims->num_q_heads)) ||
            overlap(q_out, out_bytes, k, span(k_stride, dims->num_kv_heads)) ||
            overlap(q_out, out_bytes, v, span(v_stride, dims->num_kv_heads)))
            return LOCKS_ERR_INVALID_ARG;
    }
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    locks::AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = strides[0];
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.token_seq = token_seq;
    a.cache_index = cache_index;
    a.page_table = page_table;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_tokens = num_tokens;
    a.batch = dims->batch;
    a.hq = dims->num_q_heads;
    a.hkv = dims->num_kv_heads;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.in_type = in_type;
    a.q_type = q_type;
    if (turned) {
        a.rot_dim = rope->rot_dim;
        a.interleaved = rope->interleaved;
        a.rope_scale = rope->scale;
        for (int i = 0; i < rope->rot_dim / 2; ++i) {
            a.turns[i] = locks::turn_fraction(rope->inv_freq[i]);
            a.axis[i] = static_cast<uint8_t>(rope->axis[i]);
        }
    }
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_append(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_prefix_workspace_size(const locks_dims_t* dims, int32_t num_groups, size_t* bytes) {
    if (!bytes) return LOCKS_ERR_INVALID_ARG;
    const int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (num_groups < 0) return LOCKS_ERR_INVALID_ARG;
    if (dims->batch > kMaxBatch || num_groups > kMaxBatch) return LOCKS_ERR_UNSUPPORTED;
    *bytes = locks::prefix_layout(dims->batch, dims->num_q_heads).bytes;
    return LOCKS_OK;
}

int locks_prefix_attention(const locks_dims_t* dims, const void* q, int32_t q_type, const uint16_t* k_cache,
                           const uint16_t* v_cache, const int32_t* prefix_table, const int32_t* prefix_tokens,
                           const int32_t* group_start, int32_t num_groups, int32_t max_prefix_pages,
                           const int32_t* page_table, const int32_t* seq_tokens, uint16_t* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
    int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (q_type != LOCKS_FP32 && q_type != LOCKS_BF16) return LOCKS_ERR_INVALID_ARG;
    if (num_groups < 0 || max_prefix_pages < 0) return LOCKS_ERR_INVALID_ARG;
    if (dims->batch > kMaxBatch || num_groups > kMaxBatch) return LOCKS_ERR_UNSUPPORTED;
    // token counts are int32
    if (max_prefix_pages > INT_MAX / LOCKS_PAGE_SIZE || dims->max_pages_per_seq > INT_MAX / LOCKS_PAGE_SIZE)
        return LOCKS_ERR_UNSUPPORTED;
    // cache rows are TMA coordinates (int32)
    if (static_cast<int64_t>(dims->num_phys_pages) * dims->num_kv_heads * LOCKS_PAGE_SIZE > INT_MAX)
        return LOCKS_ERR_UNSUPPORTED;
    const locks::PrefixLayout w = locks::prefix_layout(dims->batch, dims->num_q_heads);
    if ((s = locks::check_workspace(workspace, workspace_bytes, w.bytes)) != LOCKS_OK) return s;
    if (dims->batch == 0) return LOCKS_OK;
    if (!q || !k_cache || !v_cache || !seq_tokens || !out) return LOCKS_ERR_INVALID_ARG;
    if (dims->max_pages_per_seq > 0 && !page_table) return LOCKS_ERR_INVALID_ARG;
    if (num_groups > 0 && (!prefix_tokens || !group_start || (max_prefix_pages > 0 && !prefix_table)))
        return LOCKS_ERR_INVALID_ARG;
    if (dims->num_phys_pages <= 0) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return LOCKS_ERR_INVALID_ARG;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    locks::PrefixArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.q_type = q_type;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.prefix_table = prefix_table;
    a.prefix_tokens = prefix_tokens;
    a.group_start = group_start;
    a.page_table = page_table;
    a.seq_tokens = seq_tokens;
    a.out = out;
    a.lse = lse;
    a.num_groups = num_groups;
    a.max_prefix_pages = max_prefix_pages;
    a.batch = dims->batch;
    a.hq = dims->num_q_heads;
    a.hkv = dims->num_kv_heads;
    a.group = a.hq / a.hkv;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.total = reinterpret_cast<int64_t*>(base + kStatusBytes);
    a.seqs = reinterpret_cast<locks::PrefixSeq*>(base + w.seqs);
    a.part_ml = reinterpret_cast<float2*>(base + w.ml);
    a.part_o = reinterpret_cast<float*>(base + w.o);
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_prefix(a, sms, static_cast<cudaStream_t>(stream)));
}

int locks_mass_workspace_size(const locks_dims_t* dims, size_t* bytes) {
    if (!bytes) return LOCKS_ERR_INVALID_ARG;
    const int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    *bytes = mass_layout(dims).total;
    return LOCKS_OK;
}

int locks_accumulate_mass(const locks_dims_t* dims, const float* scores, const float* lse_partials,
                          const int32_t* seq_pages, const float* mass, float* mass_out, float decay, void* workspace,
                          size_t workspace_bytes, void* stream) {
    int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (!std::isfinite(decay)) return LOCKS_ERR_INVALID_ARG;
    if (dims->batch > 65535) return LOCKS_ERR_UNSUPPORTED;              // a grid dimension
    const MassLayout w = mass_layout(dims);
    if ((s = locks::check_workspace(workspace, workspace_bytes, w.total)) != LOCKS_OK) return s;
    if (dims->batch == 0 || dims->max_pages_per_seq == 0) return LOCKS_OK;
    if (!scores || !seq_pages || !mass || !mass_out) return LOCKS_ERR_INVALID_ARG;
    if (!aligned(scores, 4) || !aligned(mass, 4) || !aligned(mass_out, 4)) return LOCKS_ERR_INVALID_ARG;
    if (lse_partials && !aligned(lse_partials, 16)) return LOCKS_ERR_INVALID_ARG;
    if (!same_or_apart(mass, mass_out, static_cast<size_t>(dims->batch) * dims->max_pages_per_seq * sizeof(float)))
        return LOCKS_ERR_INVALID_ARG;
    const int sms = locks::current_sms();
    if (sms <= 0) return LOCKS_ERR_CUDA;
    locks::MassArgs a;
    a.scores = scores;
    a.seq_pages = seq_pages;
    a.mass = mass;
    a.mass_out = mass_out;
    a.decay = decay;
    a.batch = dims->batch;
    a.hq = dims->num_q_heads;
    a.max_pages = dims->max_pages_per_seq;
    a.st = locks::device_status(workspace);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float2* own = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + w.partials);
    a.partials = own;
    if (lse_partials) {
        a.row = 1;
        s = cuda_status(locks::launch_mass_reduce(reinterpret_cast<const float2*>(lse_partials),
                                                  locks::scorer_slots(dims, sms), a, own, st));
    } else {
        a.row = locks::mass_partials_row(dims->max_pages_per_seq);
        s = cuda_status(locks::launch_mass_partials(a, own, st));
    }
    if (s != LOCKS_OK) return s;
    return cuda_status(locks::launch_mass(a, st));
}

int locks_evict_pages(const locks_dims_t* dims, const float* mass, const int32_t* page_table,
                      const int32_t* seq_pages, int32_t keep_pages, int32_t sink_pages, int32_t recent_pages,
                      int32_t extra_pages, float* mass_out, int32_t* page_table_out, int32_t* seq_pages_out,
                      int32_t* evicted, int32_t evict_cap, int32_t* n_evicted, void* workspace,
                      size_t workspace_bytes, void* stream) {
    int s = locks::check_dims(dims);
    if (s != LOCKS_OK) return s;
    if (keep_pages < 0 || sink_pages < 0 || recent_pages < 0 || extra_pages < 0) return LOCKS_ERR_INVALID_ARG;
    if (static_cast<int64_t>(sink_pages) + recent_pages > keep_pages) return LOCKS_ERR_INVALID_ARG;
    if (evict_cap < 1 || evict_cap < static_cast<int64_t>(dims->max_pages_per_seq) - keep_pages)
        return LOCKS_ERR_INVALID_ARG;
    if (dims->max_pages_per_seq > locks::kMaxEvictPages || dims->batch > INT_MAX / 16) return LOCKS_ERR_UNSUPPORTED;
    if (workspace && (s = locks::check_workspace(workspace, workspace_bytes, kStatusBytes)) != LOCKS_OK) return s;
    if (dims->batch == 0) return LOCKS_OK;
    if (!seq_pages || !seq_pages_out || !n_evicted || !evicted) return LOCKS_ERR_INVALID_ARG;
    if (dims->max_pages_per_seq > 0 && (!mass || !page_table || !mass_out || !page_table_out))
        return LOCKS_ERR_INVALID_ARG;
    const size_t row = static_cast<size_t>(dims->batch) * dims->max_pages_per_seq * 4;
    if (!same_or_apart(mass, mass_out, row) || !same_or_apart(page_table, page_table_out, row) ||
        !same_or_apart(seq_pages, seq_pages_out, static_cast<size_t>(dims->batch) * 4))
        return LOCKS_ERR_INVALID_ARG;
    if (locks::current_sms() <= 0) return LOCKS_ERR_CUDA;
    locks::EvictArgs a;
    a.mass = mass;
    a.page_table = page_table;
    a.seq_pages = seq_pages;
    a.mass_out = mass_out;
    a.page_table_out = page_table_out;
    a.seq_pages_out = seq_pages_out;
    a.evicted = evicted;
    a.n_evicted = n_evicted;
    a.batch = dims->batch;
    a.max_pages = dims->max_pages_per_seq;
    a.keep = keep_pages;
    a.sink = sink_pages;
    a.recent = recent_pages;
    a.extra = extra_pages;
    a.evict_cap = evict_cap;
    a.st = locks::device_status(workspace);
    return cuda_status(locks::launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
