"""Host-side argument checks of the paged-cache operators (include/locks_cache.h): every
refusal is returned before any CUDA call, and the stand-in device addresses are never
read. Also the binding's own checks, and pins of the float64 forms the GPU tests use."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from tests import cache_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                                       # stand-in device address
OK, INV, UNSUP, SMALL = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    from sparse_kv_page_gb300 import build as b
    b.build()
    import sparse_kv_page_gb300 as L
    L.cache.load_library()
    return L


@pytest.fixture(scope="module")
def so(L):
    return L.load_library()


def test_exports_every_declared_symbol(L):
    with open(os.path.join(ROOT, "include", "locks_cache.h")) as f:
        names = set(re.findall(r"LOCKS_API\s+int\s+(locks_\w+)\s*\(", f.read()))
    assert names == {"locks_append_tokens", "locks_prefix_workspace_size", "locks_prefix_attention",
                     "locks_mass_workspace_size", "locks_accumulate_mass", "locks_evict_pages"}
    lib = ctypes.CDLL(L.library_path())
    for n in names:
        assert hasattr(lib, n), n
        assert n in L.__all__


def rope(L, **kw):
    r = L.make_rope(128, [1.0 / (i + 1) for i in range(64)])
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INV), (dict(n=0), OK), (dict(n=0, k=None, cache_index=None), OK), (dict(in_type=3), INV),
    (dict(in_type=-1), INV), (dict(q_type=1), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(cache_index=None), INV),
    (dict(page_table=None), INV), (dict(k_cache=None), INV), (dict(v_cache=None), INV), (dict(q=None), INV),
    (dict(q_out=None), INV), (dict(positions=None), INV), (dict(token_seq=None, n=5), INV),
    (dict(q_stride=-128), INV), (dict(k_stride=1 << 62), INV), (dict(v_stride=4), INV), (dict(q=A + 8), INV),
    (dict(k=A + 2), INV), (dict(q_out=A + 4), INV), (dict(k_cache=A + 8), INV), (dict(q_weight=A + 4), INV),
    (dict(q_out=A), INV), (dict(q_out=2 * A - 16), INV), (dict(ws=A + 16, nws=512), INV), (dict(ws=A, nws=128), SMALL)])
def test_append_refusals(L, so, change, status):
    a = dict(n=3, in_type=0, q_type=2, eps=1e-6, q=A, k=2 * A, v=3 * A, cache_index=A, page_table=A, k_cache=5 * A,
             v_cache=6 * A, q_out=4 * A, positions=A, token_seq=A, q_stride=8 * 128, k_stride=256, v_stride=256,
             q_weight=None, ws=None, nws=0)
    a.update(change)
    d = L.make_dims(4, 8, 2, 16, 64)
    got = so.locks_append_tokens(ctypes.byref(d), ctypes.byref(rope(L)), a["q"], a["k"], a["v"], a["in_type"],
                                 a["q_stride"], a["k_stride"], a["v_stride"], a["n"], a["positions"], a["token_seq"],
                                 a["cache_index"], a["page_table"], a["q_weight"], None, a["eps"], a["q_out"],
                                 a["q_type"], a["k_cache"], a["v_cache"], a["ws"], a["nws"], None)
    assert got == status


@pytest.mark.parametrize("change,status", [
    (dict(rot_dim=-16), INV), (dict(rot_dim=144), INV), (dict(rot_dim=24), UNSUP), (dict(num_axes=0), INV),
    (dict(num_axes=5), INV), (dict(interleaved=2), INV), (dict(scale=float("inf")), INV)])
def test_append_refuses_bad_rotations(L, so, change, status):
    d = L.make_dims(4, 8, 2, 16, 64)

    def call(r, n=0):
        return so.locks_append_tokens(ctypes.byref(d), ctypes.byref(r), A, A, A, 0, 1024, 256, 256, n, A, A, A, A, None,
                                      None, 1e-6, 4 * A, 2, A, A, None, 0, None)

    assert call(rope(L, **change)) == status
    for name, value in (("inv_freq", float("nan")), ("inv_freq", 5000.0), ("axis", 1), ("axis", -1)):
        r = rope(L)
        getattr(r, name)[63] = value
        assert call(r) == INV
        r.rot_dim = 112                           # the pair is not rotated: its entry is not looked at
        assert call(r) == OK


@pytest.mark.parametrize("change,status", [
    (dict(q_type=1), INV), (dict(groups=-1), INV), (dict(pages=-1), INV), (dict(groups=65537), UNSUP),
    (dict(pages=1 << 28), UNSUP), (dict(ws=None, nws=0), SMALL), (dict(nws=1000), SMALL), (dict(ws=A + 64), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(seq=None), INV), (dict(out=None), INV),
    (dict(table=None), INV), (dict(ptable=None), INV), (dict(ptok=None), INV), (dict(start=None), INV),
    (dict(q=A + 8), INV), (dict(k=A + 8), INV), (dict(out=A + 8), INV)])
def test_prefix_refusals(L, so, change, status):
    d = L.make_dims(4, 8, 2, 16, 64)
    a = dict(q=A, q_type=2, k=A, v=A, ptable=A, ptok=A, start=A, groups=2, pages=8, table=A, seq=A, out=A, ws=A,
             nws=L.locks_prefix_workspace_size(d, 2))
    a.update(change)
    assert so.locks_prefix_attention(ctypes.byref(d), a["q"], a["q_type"], a["k"], a["v"], a["ptable"], a["ptok"],
                                     a["start"], a["groups"], a["pages"], a["table"], a["seq"], a["out"], None,
                                     a["ws"], a["nws"], None) == status


def test_prefix_sizes(L, so):
    n = ctypes.c_size_t(0)
    assert so.locks_prefix_workspace_size(None, 1, ctypes.byref(n)) == INV
    d = L.make_dims(4, 8, 2, 16, 64)
    assert so.locks_prefix_workspace_size(ctypes.byref(d), 1, None) == INV
    assert so.locks_prefix_workspace_size(ctypes.byref(d), -1, ctypes.byref(n)) == INV
    big = L.make_dims(65537, 8, 2, 16, 64)
    assert so.locks_prefix_workspace_size(ctypes.byref(big), 1, ctypes.byref(n)) == UNSUP
    rows = L.make_dims(4, 8, 8, 16, 1 << 24)      # 2^31 cache rows: more than a TMA coordinate holds
    ws = L.locks_prefix_workspace_size(rows, 1)
    assert so.locks_prefix_attention(ctypes.byref(rows), A, 2, A, A, A, A, A, 1, 8, A, A, A, None, A, ws, None) == UNSUP
    empty = L.make_dims(0, 8, 2, 16, 64)
    ws = L.locks_prefix_workspace_size(empty, 0)
    assert so.locks_prefix_attention(ctypes.byref(empty), None, 2, None, None, None, None, None, 0, 0, None, None, None,
                                     None, A, ws, None) == OK
    none = L.make_dims(2, 8, 2, 0, 0)             # no pool to read from
    ws = L.locks_prefix_workspace_size(none, 0)
    assert so.locks_prefix_attention(ctypes.byref(none), A, 2, A, A, None, None, None, 0, 0, None, A, A, None, A, ws,
                                     None) == INV


@pytest.mark.parametrize("change,status", [
    (dict(decay=float("nan")), INV), (dict(decay=float("inf")), INV), (dict(scores=None), INV), (dict(seq=None), INV),
    (dict(mass=None), INV), (dict(out=None), INV), (dict(scores=A + 2), INV), (dict(out=3 * A + 4), INV),
    (dict(out=3 * A - 256), INV), (dict(partials=A + 8), INV), (dict(ws=None, nws=0), SMALL), (dict(nws=256), SMALL),
    (dict(ws=A + 16), INV), (dict(partials=A, ws=None, nws=0), SMALL)])
def test_mass_refusals(L, so, change, status):
    d = L.make_dims(2, 8, 2, 100, 64)
    a = dict(scores=A, partials=None, seq=A, mass=3 * A, out=4 * A, decay=1.0, ws=A, nws=L.locks_mass_workspace_size(d))
    a.update(change)

    def call(d):
        return so.locks_accumulate_mass(ctypes.byref(d), a["scores"], a["partials"], a["seq"], a["mass"], a["out"],
                                        a["decay"], a["ws"], a["nws"], None)

    assert call(d) == status
    if change == dict(scores=None):
        assert call(L.make_dims(0, 8, 2, 100, 64)) == OK and call(L.make_dims(2, 8, 2, 0, 64)) == OK
        assert call(L.make_dims(65536, 8, 2, 0, 64)) == UNSUP
        n = ctypes.c_size_t(0)
        assert so.locks_mass_workspace_size(None, ctypes.byref(n)) == INV
        assert so.locks_mass_workspace_size(ctypes.byref(d), None) == INV


@pytest.mark.parametrize("change,status", [
    (dict(keep=-1), INV), (dict(sink=-1), INV), (dict(recent=-1), INV), (dict(extra=-1), INV),
    (dict(sink=50, recent=11), INV), (dict(cap=39), INV), (dict(keep=100, cap=0), INV), (dict(mass=None), INV),
    (dict(table=None), INV), (dict(seq=None), INV), (dict(mass_out=None), INV), (dict(table_out=None), INV),
    (dict(seq_out=None), INV), (dict(evicted=None), INV), (dict(n_evicted=None), INV), (dict(mass_out=2 * A + 4), INV),
    (dict(table_out=3 * A - 4), INV), (dict(seq_out=4 * A + 4), INV), (dict(ws=A + 1, nws=256), INV),
    (dict(ws=A, nws=255), SMALL)])
def test_evict_refusals(L, so, change, status):
    a = dict(mass=2 * A, table=3 * A, seq=4 * A, keep=60, sink=1, recent=4, extra=2, mass_out=5 * A, table_out=6 * A,
             seq_out=7 * A, evicted=8 * A, cap=40, n_evicted=9 * A, ws=None, nws=0)
    a.update(change)

    def call(d):
        return so.locks_evict_pages(ctypes.byref(d), a["mass"], a["table"], a["seq"], a["keep"], a["sink"], a["recent"],
                                    a["extra"], a["mass_out"], a["table_out"], a["seq_out"], a["evicted"], a["cap"],
                                    a["n_evicted"], a["ws"], a["nws"], None)

    assert call(L.make_dims(2, 8, 2, 100, 64)) == status
    if change == dict(mass=None):
        assert call(L.make_dims(0, 8, 2, 100, 64)) == OK
        a["cap"] = 1 << 20
        assert call(L.make_dims(2, 8, 2, 393217, 64)) == UNSUP


def test_binding_checks_types_shapes_and_layouts(L):
    d = L.make_dims(2, 4, 2, 8, 16)
    k = torch.zeros(2, 2, 128)
    cache = torch.zeros(16, 2, 16, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 8, dtype=torch.int32)

    def append(k=k, v=k, cache_index=i32, page_table=table, k_cache=cache, **kw):
        L.locks_append_tokens(d, None, None, k, v, None, cache_index, page_table, None, k_cache, cache, **kw)

    for kw, err in ((dict(k=k.double()), TypeError), (dict(v=k.half()), TypeError), (dict(v=k[:1]), ValueError),
                    (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(cache_index=i32.long()), TypeError), (dict(page_table=table[:, :4]), ValueError),
                    (dict(page_table=table.t().contiguous().t()), ValueError), (dict(k_cache=cache.float()), TypeError),
                    (dict(k_cache=cache[:8]), ValueError), ({}, ValueError)):        # last: not CUDA tensors
        with pytest.raises(err):
            append(**kw)
    for args in ((128, [1.0] * 63), (0, [1.0]), (132, [1.0] * 66)):
        with pytest.raises(ValueError):
            L.make_rope(*args)
    with pytest.raises(ValueError):
        L.make_rope(16, [1.0] * 8, axis=[0] * 7)
    r = L.make_rope(32, [0.5] * 16, interleaved=True, axis=[0] * 8 + [2] * 8, scale=0.5)
    assert (r.rot_dim, r.interleaved, r.num_axes, r.scale, r.axis[15], r.inv_freq[15]) == (32, 1, 3, 0.5, 2, 0.5)
    with pytest.raises(ValueError):               # shapes against dims
        L.locks_evict_pages(d, torch.zeros(2, 9), table, i32, 4, torch.zeros(2, 8), table, i32, table, i32)
    with pytest.raises(TypeError):
        L.locks_accumulate_mass(d, torch.zeros(2, 4, 8).half(), i32, torch.zeros(2, 8), torch.zeros(2, 8),
                                torch.zeros(512, dtype=torch.uint8))


# ------------------------------------------------------- the float64 forms themselves

def test_reference_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 128))
    for inter in (False, True):
        angle = rng.uniform(-9, 9, 48)
        y = ref.rotate(x, angle, inter, 1.0)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[:, 96:], x[:, 96:])
        assert np.allclose(ref.rotate(y, -angle, inter, 1.0), x)
        # scores depend on the difference of the angles alone
        z = rng.standard_normal((3, 128))
        d = ref.rotate(x, angle + 1, inter, 1.0) * ref.rotate(z, angle + 1.5, inter, 1.0)
        e = ref.rotate(x, angle * 0, inter, 1.0) * ref.rotate(z, angle * 0 + 0.5, inter, 1.0)
        assert np.allclose(d.sum(-1), e.sum(-1))
    e0 = np.zeros(128)
    e0[0] = 1
    assert ref.rotate(e0, np.full(64, np.pi / 2), False, 1.0)[64] == 1.0
    assert ref.rotate(e0, np.full(64, np.pi / 2), True, 1.0)[1] == 1.0


def test_reference_attention_mass_and_eviction():
    v = np.arange(256.0).reshape(2, 128)
    out, lse, w, size = ref.attend(np.zeros((1, 128)), np.ones((2, 128)), v)
    assert np.allclose(out, v.mean(0)) and np.allclose(lse, np.log(2)) and np.allclose(w, v.mean(0)) and size[0] == 0
    out, lse, _, _ = ref.attend(np.zeros((1, 128)), np.zeros((0, 128)), np.zeros((0, 128)))
    assert np.all(out == 0) and np.isneginf(lse[0])
    s = np.log(np.array([[[1.0, 3.0, 5.0], [2.0, 2.0, np.nan]]]))
    assert np.allclose(ref.mass(s, [2], np.full((1, 3), 4.0), 0.5)[0], [2 + (0.25 + 0.5) / 2, 2 + (0.75 + 0.5) / 2])
    assert np.allclose(ref.mass(s, [3], np.zeros((1, 3)), 1.0)[0].sum(), 1)
    m, t = np.array([3.0, 1.0, 1.0, 9.0, 0.5, 7.0], np.float32), np.arange(10, 16)
    kept, mass, gone = ref.evict(m, t, 5, 3, 0, 0, 1)
    assert kept.tolist() == [10, 12, 13, 15] and gone.tolist() == [11, 14] and mass.tolist() == [3, 1, 9, 7]
    kept, _, gone = ref.evict(m, t, 5, 3, 1, 1, 0)      # the last page is held: the tie falls whole
    assert kept.tolist() == [10, 13, 14] and gone.tolist() == [11, 12]
    assert ref.evict(m, t, 2, 3, 0, 0, 0)[2].size == 0
