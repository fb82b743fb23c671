// marshal.cpp - argument checks of the Python bindings of locks_cache.h and locks_pool.h (module
// _marshal).
//
// A decode step's small calls take a few microseconds on the GPU; reading the type, size,
// layout and address of a dozen tensors through Python attributes took longer than that.
// Here each tensor is read once through torch's C++ handle, and the C entry point is called
// with the result. Nothing of the operators is computed here. Every function returns the
// entry point's status, or raises TypeError / ValueError for a tensor that does not fit.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/locks_pool.h"

namespace {

using Append = decltype(&locks_append_tokens);
using Prefix = decltype(&locks_prefix_attention);
using Mass = decltype(&locks_accumulate_mass);
using Evict = decltype(&locks_evict_pages);
Append g_append;
Prefix g_prefix;
Mass g_mass;
Evict g_evict;
decltype(&locks_pack_pages) g_pack;
decltype(&locks_unpack_pages) g_unpack;
decltype(&locks_packed_attention) g_attend;
decltype(&locks_copy_pages) g_copy;
decltype(&locks_fork_sequences) g_fork;
decltype(&locks_take_pages) g_take;
decltype(&locks_free_pages) g_free;
decltype(&locks_compact_pages) g_compact;

struct Refused {};                       // a Python error is set

enum Kind : unsigned { kI32 = 1, kF32 = 2, kBf16 = 4, kF16 = 8, kBytes = 16, kU8 = 32 };   // kBf16: int16 bits too

unsigned kind_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kInt: return kI32;
        case at::kFloat: return kF32;
        case at::kBFloat16: case at::kShort: return kBf16;
        case at::kHalf: return kF16;
        case at::kByte: return kU8;
        default: return 0;
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s is no tensor", name);
        throw Refused();
    }
    return THPVariable_Unpack(o);
}

struct Call {
    int device;                          // of the call's tensors
    mutable const char* off = nullptr;   // the first tensor that is not on it
    mutable int at = -1;                 // ... but there (-1: on the host)

    void on_device(const at::Tensor& t, const char* name) const {
        const int d = t.is_cuda() ? static_cast<int>(t.get_device()) : -1;
        if (!off && (d != device || d < 0)) off = name, at = d;
    }
    // After the other checks of all tensors.
    void settle() const {
        if (!off) return;
        if (at < 0) PyErr_Format(PyExc_ValueError, "%s is no CUDA tensor", off);
        else PyErr_Format(PyExc_ValueError, "%s is on device %d, the call is on device %d", off, at, device);
        throw Refused();
    }
    void typed(const at::Tensor& t, const char* name, unsigned kinds) const {
        if (kinds != kBytes && !(kind_of(t) & kinds)) {
            PyErr_Format(PyExc_TypeError, "%s has type %s", name, at::toString(t.scalar_type()));
            throw Refused();
        }
    }
    // The address of a contiguous tensor of `size` elements (None: null, where it may be).
    void* at_(PyObject* o, const char* name, unsigned kinds, int64_t size, bool may_be_none = false) const {
        if (may_be_none && o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name);
        typed(t, name, kinds);
        if (kinds != kBytes && t.numel() != size) {
            PyErr_Format(PyExc_ValueError, "%s has %lld elements, not %lld", name, static_cast<long long>(t.numel()),
                         static_cast<long long>(size));
            throw Refused();
        }
        if (!t.is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "LOCKS buffers must be contiguous");
            throw Refused();
        }
        on_device(t, name);
        return t.data_ptr();
    }
    template <typename T>
    T* get(PyObject* o, const char* name, unsigned kinds, int64_t size, bool may_be_none = false) const {
        return static_cast<T*>(at_(o, name, kinds, size, may_be_none));
    }
    // The address of a contiguous list of at least `size` entries.
    int32_t* list(PyObject* o, const char* name, int64_t size, bool may_be_none = false) const {
        if (may_be_none && o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name);
        if (t.numel() < size) {
            PyErr_Format(PyExc_ValueError, "%s has %lld elements, fewer than %lld", name, static_cast<long long>(t.numel()),
                         static_cast<long long>(size));
            throw Refused();
        }
        return get<int32_t>(o, name, kI32, t.numel());
    }
    // The address of packed pages [pages][kv heads][LOCKS_PACKED_BYTES], and how many there are.
    uint8_t* units(PyObject* o, int64_t heads, int32_t* pages) const {
        const at::Tensor& t = tensor(o, "packed");
        typed(t, "packed", kU8);
        if (t.dim() != 3 || t.size(0) > INT32_MAX || t.size(1) != heads || t.size(2) != LOCKS_PACKED_BYTES) {
            PyErr_Format(PyExc_ValueError, "packed is not [pages][%lld][%d]", static_cast<long long>(heads),
                         LOCKS_PACKED_BYTES);
            throw Refused();
        }
        *pages = static_cast<int32_t>(t.size(0));
        return get<uint8_t>(o, "packed", kU8, t.numel());
    }
    // [tokens][heads][128] rows; only the token axis may be strided.
    void* rows(PyObject* o, const char* name, at::ScalarType type, int64_t tokens, int64_t heads, int64_t* step) const {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != type) {
            PyErr_Format(PyExc_TypeError, "%s has type %s, k has %s", name, at::toString(t.scalar_type()),
                         at::toString(type));
            throw Refused();
        }
        if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != 128) {
            PyErr_Format(PyExc_ValueError, "%s is not [%lld][%lld][128]", name, static_cast<long long>(tokens),
                         static_cast<long long>(heads));
            throw Refused();
        }
        if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != 128)) {
            PyErr_Format(PyExc_ValueError, "%s: the heads of a token must lie beside each other", name);
            throw Refused();
        }
        on_device(t, name);
        *step = tokens > 1 ? t.stride(0) : 0;
        return t.data_ptr();
    }
    void* workspace(PyObject* o, size_t* bytes) const {
        *bytes = 0;
        if (o == Py_None) return nullptr;
        void* p = at_(o, "workspace", kBytes, 0);
        *bytes = THPVariable_Unpack(o).nbytes();
        return p;
    }
};

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
int32_t int32_of(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s is out of range", name);
        throw Refused();
    }
    return static_cast<int32_t>(v);
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return static_cast<float>(v);
}
template <typename T>
T* address(PyObject* o) {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(integer(o)));
}
// q's type for the C ABI.
int32_t query_type(PyObject* o) {
    return o != Py_None && THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() != at::kFloat ? LOCKS_BF16
                                                                                                    : LOCKS_FP32;
}
// The entry point's status. Other Python threads run meanwhile: a launch may wait for room in the
// stream's queue, and what drains it (a host callback) may need the interpreter.
template <typename F>
int released(F entry) {
    PyThreadState* const state = PyEval_SaveThread();
    const int status = entry();
    PyEval_RestoreThread(state);
    return status;
}
// fp32, or the bf16 bits that int16 holds too.
constexpr unsigned kQuery = kF32 | kBf16;

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(addresses of the four entry points)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        g_append = reinterpret_cast<Append>(integer(a[0]));
        g_prefix = reinterpret_cast<Prefix>(integer(a[1]));
        g_mass = reinterpret_cast<Mass>(integer(a[2]));
        g_evict = reinterpret_cast<Evict>(integer(a[3]));
        return 0;
    });
}

// append(device, stream, dims, rope, q, k, v, positions, cache_index, page_table, q_out, k_cache, v_cache,
//        token_seq, q_weight, k_weight, eps, workspace)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 18, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const locks_rope_t* rope = address<const locks_rope_t>(a[3]);
        const at::Tensor& kt = tensor(a[5], "k");
        const at::ScalarType type = kt.scalar_type();
        const unsigned kind = kind_of(kt);
        if (!(kind & (kBf16 | kF16 | kF32))) c.typed(kt, "k", kBf16 | kF16 | kF32);
        const int64_t t = kt.dim() > 0 ? kt.size(0) : 0;
        if (t > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "too many tokens for one call");
            throw Refused();
        }
        int64_t qs = 0, ks = 0, vs = 0;
        const void* k = c.rows(a[5], "k", type, t, d->num_kv_heads, &ks);
        const void* v = c.rows(a[6], "v", type, t, d->num_kv_heads, &vs);
        const void* q = a[4] == Py_None ? nullptr : c.rows(a[4], "q", type, t, d->num_q_heads, &qs);
        const int64_t cache = static_cast<int64_t>(d->num_phys_pages) * d->num_kv_heads * 2048;
        const int32_t* positions = nullptr;
        if (rope && a[7] != Py_None) {
            const at::Tensor& p = tensor(a[7], "positions");
            const bool rows = p.dim() == 2 && p.size(0) == rope->num_axes && p.size(1) == t;
            if (!rows && !(p.dim() == 1 && rope->num_axes == 1 && p.size(0) == t)) {
                PyErr_Format(PyExc_ValueError, "positions is not [%d][%lld]", static_cast<int>(rope->num_axes),
                             static_cast<long long>(t));
                throw Refused();
            }
            positions = c.get<int32_t>(a[7], "positions", kI32, t * rope->num_axes);
        }
        const int32_t* index = c.get<int32_t>(a[8], "cache_index", kI32, t);
        const int32_t* table =
            c.get<int32_t>(a[9], "page_table", kI32, static_cast<int64_t>(d->batch) * d->max_pages_per_seq);
        void* q_out = c.at_(a[10], "q_out", kQuery, t * d->num_q_heads * 128, true);
        uint16_t* kc = c.get<uint16_t>(a[11], "k_cache", kBf16, cache);
        uint16_t* vc = c.get<uint16_t>(a[12], "v_cache", kBf16, cache);
        const int32_t* seq = c.get<int32_t>(a[13], "token_seq", kI32, t, true);
        const float* qw = c.get<float>(a[14], "q_weight", kF32, 128, true);
        const float* kw = c.get<float>(a[15], "k_weight", kF32, 128, true);
        size_t bytes;
        void* ws = c.workspace(a[17], &bytes);
        const float eps = real(a[16]);
        const int32_t in_type = kind == kF32 ? LOCKS_FP32 : kind == kF16 ? LOCKS_FP16 : LOCKS_BF16;
        const int32_t q_type = query_type(a[10]);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] {
            return g_append(d, rope, q, k, v, in_type, qs, ks, vs, static_cast<int32_t>(t), positions, seq, index, table,
                            qw, kw, eps, q_out, q_type, kc, vc, ws, bytes, stream);
        });
    });
}

// prefix(device, stream, dims, q, k_cache, v_cache, prefix_table, prefix_tokens, group_start, page_table, seq_tokens,
//        out, workspace, lse)
PyObject* prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, cells = b * d->num_q_heads * 128;
        const int64_t cache = static_cast<int64_t>(d->num_phys_pages) * d->num_kv_heads * 2048;
        const void* q = c.at_(a[3], "q", kQuery, cells);
        const uint16_t* kc = c.get<uint16_t>(a[4], "k_cache", kBf16, cache);
        const uint16_t* vc = c.get<uint16_t>(a[5], "v_cache", kBf16, cache);
        int64_t groups = 0, pages = 0;
        const int32_t *table = nullptr, *tokens = nullptr, *start = nullptr;
        if (a[6] != Py_None) {
            const at::Tensor& pt = tensor(a[6], "prefix_table");
            if (pt.dim() != 2 || pt.size(0) > INT32_MAX || pt.size(1) > INT32_MAX) {
                PyErr_SetString(PyExc_ValueError, "prefix_table is not [groups][pages]");
                throw Refused();
            }
            groups = pt.size(0);
            pages = pt.size(1);
            if (groups > 0) {
                table = c.get<int32_t>(a[6], "prefix_table", kI32, groups * pages);
                tokens = c.get<int32_t>(a[7], "prefix_tokens", kI32, groups);
                start = c.get<int32_t>(a[8], "group_start", kI32, groups + 1);
            }
        }
        const int32_t* own = c.get<int32_t>(a[9], "page_table", kI32, b * d->max_pages_per_seq, true);
        const int32_t* seq = c.get<int32_t>(a[10], "seq_tokens", kI32, b);
        uint16_t* out = c.get<uint16_t>(a[11], "out", kBf16, cells);
        size_t bytes;
        void* ws = c.workspace(a[12], &bytes);
        float* lse = c.get<float>(a[13], "lse", kF32, b * d->num_q_heads, true);
        const int32_t q_type = query_type(a[3]);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] {
            return g_prefix(d, q, q_type, kc, vc, table, tokens, start, static_cast<int32_t>(groups),
                            static_cast<int32_t>(pages), own, seq, out, lse, ws, bytes, stream);
        });
    });
}

// mass(device, stream, dims, scores, seq_pages, mass, mass_out, workspace, decay, lse_partials, partials' size)
PyObject* mass(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, p = d->max_pages_per_seq;
        const float* scores = c.get<float>(a[3], "scores", kF32, b * d->num_q_heads * p);
        const int32_t* seq = c.get<int32_t>(a[4], "seq_pages", kI32, b);
        const float* old = c.get<float>(a[5], "mass", kF32, b * p);
        float* out = c.get<float>(a[6], "mass_out", kF32, b * p);
        size_t bytes;
        void* ws = c.workspace(a[7], &bytes);
        const float* partials = c.get<float>(a[9], "lse_partials", kF32, integer(a[10]), true);
        const float decay = real(a[8]);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] { return g_mass(d, scores, partials, seq, old, out, decay, ws, bytes, stream); });
    });
}

// evict(device, stream, dims, mass, page_table, seq_pages, keep, mass_out, page_table_out, seq_pages_out, evicted,
//       n_evicted, sink, recent, extra, workspace)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, cells = b * d->max_pages_per_seq;
        const float* m = c.get<float>(a[3], "mass", kF32, cells);
        const int32_t* table = c.get<int32_t>(a[4], "page_table", kI32, cells);
        const int32_t* seq = c.get<int32_t>(a[5], "seq_pages", kI32, b);
        float* mo = c.get<float>(a[7], "mass_out", kF32, cells);
        int32_t* to = c.get<int32_t>(a[8], "page_table_out", kI32, cells);
        int32_t* so = c.get<int32_t>(a[9], "seq_pages_out", kI32, b);
        const at::Tensor& e = tensor(a[10], "evicted");
        const int64_t cap = e.dim() == 2 ? e.size(1) : -1;
        if (cap < 0 || cap > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "evicted is not [batch][pages]");
            throw Refused();
        }
        int32_t* ev = c.get<int32_t>(a[10], "evicted", kI32, b * cap);
        int32_t* ne = c.get<int32_t>(a[11], "n_evicted", kI32, b);
        size_t bytes;
        void* ws = c.workspace(a[15], &bytes);
        const int32_t keep = int32_of(a[6], "keep_pages"), sink = int32_of(a[12], "sink_pages");
        const int32_t recent = int32_of(a[13], "recent_pages"), extra = int32_of(a[14], "extra_pages");
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] {
            return g_evict(d, m, table, seq, keep, sink, recent, extra, mo, to, so, ev, static_cast<int32_t>(cap), ne, ws,
                           bytes, stream);
        });
    });
}

// bind_pool(addresses of the eight entry points of locks_pool.h)
PyObject* bind_pool(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        g_pack = reinterpret_cast<decltype(g_pack)>(integer(a[0]));
        g_unpack = reinterpret_cast<decltype(g_unpack)>(integer(a[1]));
        g_attend = reinterpret_cast<decltype(g_attend)>(integer(a[2]));
        g_copy = reinterpret_cast<decltype(g_copy)>(integer(a[3]));
        g_fork = reinterpret_cast<decltype(g_fork)>(integer(a[4]));
        g_take = reinterpret_cast<decltype(g_take)>(integer(a[5]));
        g_free = reinterpret_cast<decltype(g_free)>(integer(a[6]));
        g_compact = reinterpret_cast<decltype(g_compact)>(integer(a[7]));
        return 0;
    });
}

// What packing and unpacking read: (device, stream, dims, k_cache, v_cache, src, dst, pages, packed, workspace)
template <typename F>
PyObject* pages_of(PyObject* const* a, Py_ssize_t n, F entry) {
    return guarded(n, 10, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t cache = static_cast<int64_t>(d->num_phys_pages) * d->num_kv_heads * 2048;
        uint16_t* k = c.get<uint16_t>(a[3], "k_cache", kBf16, cache);
        uint16_t* v = c.get<uint16_t>(a[4], "v_cache", kBf16, cache);
        const int32_t pages = int32_of(a[7], "n_pages");
        const int32_t* src = c.list(a[5], "src_pages", pages);
        const int32_t* dst = c.list(a[6], "dst_pages", pages, true);
        int32_t num = 0;
        uint8_t* packed = c.units(a[8], d->num_kv_heads, &num);
        size_t bytes;
        void* ws = c.workspace(a[9], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] { return entry(d, k, v, src, dst, pages, packed, num, ws, bytes, stream); });
    });
}
PyObject* pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return pages_of(a, n, [](auto d, auto k, auto v, auto src, auto dst, auto pages, auto packed, auto num, auto ws,
                             auto bytes, auto stream) {
        return g_pack(d, k, v, src, dst, pages, packed, num, ws, bytes, stream);
    });
}
PyObject* unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return pages_of(a, n, [](auto d, auto k, auto v, auto src, auto dst, auto pages, auto packed, auto num, auto ws,
                             auto bytes, auto stream) {
        return g_unpack(d, packed, num, src, dst, pages, k, v, ws, bytes, stream);
    });
}

// attend(device, stream, dims, q, packed, page_table, seq_pages, selected, n_selected, k_cache, v_cache,
//        recent_table, recent_tokens, out, lse, workspace)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, cells = b * d->num_q_heads * 128;
        const void* q = c.at_(a[3], "q", kQuery, cells);
        int32_t num = 0;
        const uint8_t* packed = a[4] == Py_None ? nullptr : c.units(a[4], d->num_kv_heads, &num);
        const int32_t* table = c.get<int32_t>(a[5], "page_table", kI32, b * d->max_pages_per_seq, true);
        const int32_t* seq = c.get<int32_t>(a[6], "seq_pages", kI32, b, true);
        const int32_t *selected = nullptr, *n_selected = nullptr;
        int64_t cap = 0;
        if (a[7] != Py_None) {
            const at::Tensor& t = tensor(a[7], "selected");
            if (t.dim() != 3 || t.size(0) != b || t.size(1) != d->num_kv_heads || t.size(2) > INT32_MAX) {
                PyErr_Format(PyExc_ValueError, "selected is not [%lld][%d][pages]", static_cast<long long>(b),
                             static_cast<int>(d->num_kv_heads));
                throw Refused();
            }
            cap = t.size(2);
            selected = c.get<int32_t>(a[7], "selected", kI32, t.numel());
            n_selected = c.get<int32_t>(a[8], "n_selected", kI32, b * d->num_kv_heads);
        }
        const uint16_t *kc = nullptr, *vc = nullptr;
        const int32_t *recent = nullptr, *tokens = nullptr;
        int64_t pages = 0;
        if (a[11] != Py_None) {
            const at::Tensor& t = tensor(a[11], "recent_table");
            if (t.dim() != 2 || t.size(0) != b || t.size(1) > INT32_MAX) {
                PyErr_Format(PyExc_ValueError, "recent_table is not [%lld][pages]", static_cast<long long>(b));
                throw Refused();
            }
            pages = t.size(1);
            if (pages > 0) {
                const int64_t cache = static_cast<int64_t>(d->num_phys_pages) * d->num_kv_heads * 2048;
                recent = c.get<int32_t>(a[11], "recent_table", kI32, b * pages);
                tokens = c.get<int32_t>(a[12], "recent_tokens", kI32, b);
                kc = c.get<uint16_t>(a[9], "k_cache", kBf16, cache);
                vc = c.get<uint16_t>(a[10], "v_cache", kBf16, cache);
            }
        }
        uint16_t* out = c.get<uint16_t>(a[13], "out", kBf16, cells);
        float* lse = c.get<float>(a[14], "lse", kF32, b * d->num_q_heads, true);
        size_t bytes;
        void* ws = c.workspace(a[15], &bytes);
        const int32_t q_type = query_type(a[3]);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] {
            return g_attend(d, q, q_type, packed, num, table, seq, selected, n_selected, static_cast<int32_t>(cap), kc,
                            vc, recent, static_cast<int32_t>(pages), tokens, out, lse, ws, bytes, stream);
        });
    });
}

// copy(device, stream, planes, src, dst, n_pairs, workspace)
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_planes_t* planes = address<const locks_planes_t>(a[2]);
        const int64_t pairs = tensor(a[3], "src_pages").numel();
        if (pairs > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "too many pairs for one call");
            throw Refused();
        }
        const int32_t* src = c.get<int32_t>(a[3], "src_pages", kI32, pairs);
        const int32_t* dst = c.get<int32_t>(a[4], "dst_pages", kI32, pairs);
        const int32_t* count = c.get<int32_t>(a[5], "n_pairs", kI32, 1, true);
        size_t bytes;
        void* ws = c.workspace(a[6], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] { return g_copy(planes, src, dst, static_cast<int32_t>(pairs), count, ws, bytes, stream); });
    });
}

// fork(device, stream, dims, page_table, seq_tokens, parents, refs, page_table_out, seq_tokens_out, refs_out, copy_src,
//      copy_dst, n_copies, workspace)
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, cells = b * d->max_pages_per_seq, pages = d->num_phys_pages;
        const int32_t* table = c.get<int32_t>(a[3], "page_table", kI32, cells);
        const int32_t* tokens = c.get<int32_t>(a[4], "seq_tokens", kI32, b);
        const int32_t* parents = c.get<int32_t>(a[5], "parents", kI32, b);
        const int32_t* refs = c.get<int32_t>(a[6], "refs", kI32, pages);
        int32_t* to = c.get<int32_t>(a[7], "page_table_out", kI32, cells);
        int32_t* so = c.get<int32_t>(a[8], "seq_tokens_out", kI32, b);
        int32_t* ro = c.get<int32_t>(a[9], "refs_out", kI32, pages);
        int32_t* src = c.get<int32_t>(a[10], "copy_src", kI32, b);
        int32_t* dst = c.get<int32_t>(a[11], "copy_dst", kI32, b);
        int32_t* count = c.get<int32_t>(a[12], "n_copies", kI32, 1);
        size_t bytes;
        void* ws = c.workspace(a[13], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        return released(
            [&] { return g_fork(d, table, tokens, parents, refs, to, so, ro, src, dst, count, ws, bytes, stream); });
    });
}

// take(device, stream, dims, page_table, seq_tokens, new_tokens, refs, seq_tokens_out, refs_out, n_free, workspace)
PyObject* take(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, pages = d->num_phys_pages;
        int32_t* table = c.get<int32_t>(a[3], "page_table", kI32, b * d->max_pages_per_seq);
        const int32_t* tokens = c.get<int32_t>(a[4], "seq_tokens", kI32, b);
        const int32_t* now = c.get<int32_t>(a[5], "new_tokens", kI32, b);
        const int32_t* refs = c.get<int32_t>(a[6], "refs", kI32, pages);
        int32_t* so = c.get<int32_t>(a[7], "seq_tokens_out", kI32, b);
        int32_t* ro = c.get<int32_t>(a[8], "refs_out", kI32, pages);
        int32_t* left = c.get<int32_t>(a[9], "n_free", kI32, 1, true);
        size_t bytes;
        void* ws = c.workspace(a[10], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] { return g_take(d, table, tokens, now, refs, so, ro, left, ws, bytes, stream); });
    });
}

// free(device, stream, refs, pages, counts, refs_out, workspace)
PyObject* free_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Call c{int32_of(a[0], "device")};
        const int64_t num = tensor(a[2], "refs").numel();
        const at::Tensor& t = tensor(a[3], "pages");
        if (t.dim() != 2 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || num > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "pages is not [rows][pages]");
            throw Refused();
        }
        const int32_t rows = static_cast<int32_t>(t.size(0)), stride = static_cast<int32_t>(t.size(1));
        const int32_t* refs = c.get<int32_t>(a[2], "refs", kI32, num);
        const int32_t* pages = c.get<int32_t>(a[3], "pages", kI32, t.numel());
        const int32_t* counts = c.get<int32_t>(a[4], "counts", kI32, rows);
        int32_t* out = c.get<int32_t>(a[5], "refs_out", kI32, num);
        size_t bytes;
        void* ws = c.workspace(a[6], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        return released([&] {
            return g_free(refs, static_cast<int32_t>(num), pages, stride, counts, rows, out, ws, bytes, stream);
        });
    });
}

// compact(device, stream, dims, page_table, seq_tokens, refs, page_table_out, refs_out, move_src, move_dst, n_moves,
//         new_page, workspace)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Call c{int32_of(a[0], "device")};
        const locks_dims_t* d = address<const locks_dims_t>(a[2]);
        const int64_t b = d->batch, cells = b * d->max_pages_per_seq, pages = d->num_phys_pages;
        const int32_t* table = c.get<int32_t>(a[3], "page_table", kI32, cells);
        const int32_t* tokens = c.get<int32_t>(a[4], "seq_tokens", kI32, b);
        const int32_t* refs = c.get<int32_t>(a[5], "refs", kI32, pages);
        int32_t* to = c.get<int32_t>(a[6], "page_table_out", kI32, cells);
        int32_t* ro = c.get<int32_t>(a[7], "refs_out", kI32, pages);
        const int64_t cap = tensor(a[8], "move_src").numel();
        int32_t* src = c.get<int32_t>(a[8], "move_src", kI32, cap);
        int32_t* dst = c.get<int32_t>(a[9], "move_dst", kI32, cap);
        int32_t* count = c.get<int32_t>(a[10], "n_moves", kI32, 1);
        int32_t* now = c.get<int32_t>(a[11], "new_page", kI32, pages);
        size_t bytes;
        void* ws = c.workspace(a[12], &bytes);
        void* stream = address<void>(a[1]);
        c.settle();
        const int32_t most = cap > INT32_MAX ? INT32_MAX : static_cast<int32_t>(cap);
        return released([&] {
            return g_compact(d, table, tokens, refs, to, ro, src, dst, most, count, now, ws, bytes, stream);
        });
    });
}

template <typename F>
PyMethodDef method(const char* name, F f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method("bind", bind),   method("append", append), method("prefix", prefix),
                           method("mass", mass),   method("evict", evict),   method("bind_pool", bind_pool),
                           method("pack", pack),   method("unpack", unpack), method("attend", attend),
                           method("copy", copy),   method("fork", fork),     method("take", take),
                           method("free", free_pages), method("compact", compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
