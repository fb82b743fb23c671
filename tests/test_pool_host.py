"""Host-side argument checks of the packed cache and the page pool (include/locks_pool.h): every
refusal is returned before any CUDA call, and the stand-in device addresses are never read. Also
the binding's own checks, and pins of the forms the GPU tests compare with."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from tests import pool_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                                       # stand-in device address
OK, INV, UNSUP, SMALL = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    from sparse_kv_page_gb300 import build as b
    b.build()
    import sparse_kv_page_gb300 as L
    L.pool.load_library()
    return L


@pytest.fixture(scope="module")
def so(L):
    return L.load_library()


def test_exports_every_declared_symbol(L):
    with open(os.path.join(ROOT, "include", "locks_pool.h")) as f:
        src = f.read()
    names = set(re.findall(r"LOCKS_API\s+int\s+(locks_\w+)\s*\(", src))
    assert names == {"locks_pack_pages", "locks_unpack_pages", "locks_packed_workspace_size", "locks_packed_attention",
                     "locks_copy_pages", "locks_pool_workspace_size", "locks_fork_sequences", "locks_take_pages",
                     "locks_free_pages", "locks_compact_pages"}
    lib = ctypes.CDLL(L.library_path())
    for n in names:
        assert hasattr(lib, n), n
        assert n in L.__all__
    assert f"LOCKS_PACKED_BYTES {L.LOCKS_PACKED_BYTES}\n" in src
    assert f"LOCKS_MAX_PLANES {L.pool.LOCKS_MAX_PLANES}\n" in src
    assert "free pages" in L.locks_status_string(-7)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INV), (dict(num=-1), INV), (dict(n=0), OK), (dict(n=0, k=None, packed=None, src=None), OK),
    (dict(k=None), INV), (dict(v=None), INV), (dict(packed=None), INV), (dict(src=None), INV), (dict(k=A + 8), INV),
    (dict(v=A + 2), INV), (dict(packed=A + 8), INV), (dict(src=A + 2), INV), (dict(dst=A + 1), INV),
    (dict(ws=A + 1, nws=256), INV), (dict(ws=A, nws=255), SMALL), (dict(n=0, ws=A, nws=255), SMALL)])
def test_pack_and_unpack_refusals(L, so, change, status):
    a = dict(k=A, v=A, src=A, dst=None, n=3, packed=A, num=9, ws=None, nws=0)
    a.update(change)
    d = ctypes.byref(L.make_dims(1, 8, 2, 4, 16))
    assert so.locks_pack_pages(d, a["k"], a["v"], a["src"], a["dst"], a["n"], a["packed"], a["num"], a["ws"], a["nws"],
                               None) == status
    assert so.locks_unpack_pages(d, a["packed"], a["num"], a["src"], a["dst"], a["n"], a["k"], a["v"], a["ws"], a["nws"],
                                 None) == status
    bad = ctypes.byref(L.make_dims(1, 6, 3, 4, 16))
    assert so.locks_pack_pages(bad, A, A, A, None, 0, A, 9, None, 0, None) == UNSUP


@pytest.mark.parametrize("change,status", [
    (dict(q_type=1), INV), (dict(num=-1), INV), (dict(recents=-1), INV), (dict(k_cap=0), INV), (dict(q=None), INV),
    (dict(out=None), INV), (dict(n_sel=None), INV), (dict(sel=None, seq=None), INV), (dict(packed=None), INV),
    (dict(num=0), INV), (dict(table=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(rtable=None), INV),
    (dict(rtok=None), INV), (dict(q=A + 8), INV), (dict(packed=A + 8), INV), (dict(k=A + 8), INV), (dict(out=A + 2), INV),
    (dict(lse=A + 2), INV), (dict(sel=A + 1), INV), (dict(rtok=A + 3), INV), (dict(recents=1 << 27), UNSUP),
    (dict(k_cap=1 << 30), UNSUP), (dict(ws=None, nws=0), SMALL), (dict(nws=1000), SMALL), (dict(ws=A + 64), INV)])
def test_attention_refusals(L, so, change, status):
    d = L.make_dims(4, 8, 2, 16, 64)
    a = dict(q=A, q_type=2, packed=A, num=9, table=A, seq=None, sel=A, n_sel=A, k_cap=4, k=A, v=A, rtable=A, recents=2,
             rtok=A, out=A, lse=None, ws=A, nws=L.locks_packed_workspace_size(d))
    a.update(change)

    def call(d, **kw):
        b = dict(a, **kw)
        return so.locks_packed_attention(ctypes.byref(d), b["q"], b["q_type"], b["packed"], b["num"], b["table"], b["seq"],
                                         b["sel"], b["n_sel"], b["k_cap"], b["k"], b["v"], b["rtable"], b["recents"],
                                         b["rtok"], b["out"], b["lse"], b["ws"], b["nws"], None)

    assert call(d) == status
    if change == dict(q_type=1):
        none = dict(q_type=2, q=None, out=None, packed=None, table=None, sel=None, k=None, v=None, rtable=None, rtok=None)
        assert call(L.make_dims(0, 8, 2, 16, 64), **none) == OK
        assert call(L.make_dims(65537, 8, 2, 16, 64), q_type=2) == UNSUP
        # a bf16 pool without pages: only where nothing recent is given
        assert call(L.make_dims(4, 8, 2, 16, 0), q_type=2) == INV
        n = ctypes.c_size_t(0)
        assert so.locks_packed_workspace_size(ctypes.byref(L.make_dims(4, 8, 2, 16, 0)), ctypes.byref(n)) == OK
        assert n.value == a["nws"]
        assert so.locks_packed_workspace_size(None, ctypes.byref(n)) == INV
        assert so.locks_packed_workspace_size(ctypes.byref(d), None) == INV
        assert so.locks_packed_workspace_size(ctypes.byref(L.make_dims(65537, 8, 2, 16, 64)), ctypes.byref(n)) == UNSUP


def planes(L, **kw):
    p = L.locks_planes_t(2, 10)
    for i, (base, size) in enumerate(((A, 4096), (2 * A, 8))):
        p.base[i], p.page_bytes[i] = base, size
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(p, k)[v[0]] = v[1]
        else:
            setattr(p, k, v)
    return p


@pytest.mark.parametrize("change,args,status", [
    (dict(num_planes=-1), {}, INV), (dict(num_planes=129), {}, INV), (dict(num_pages=-1), {}, INV),
    (dict(page_bytes=(1, -8)), {}, INV), (dict(page_bytes=(1, 12)), {}, INV), (dict(page_bytes=(0, 1 << 62)), {}, INV),
    (dict(base=(1, None)), {}, INV), (dict(base=(0, A + 4)), {}, INV), ({}, dict(n=-1), INV), ({}, dict(n=0), OK),
    (dict(num_planes=0), {}, OK), ({}, dict(src=None), INV), ({}, dict(dst=None), INV), ({}, dict(src=A + 1), INV),
    ({}, dict(count=A + 2), INV), ({}, dict(ws=A + 1, nws=256), INV), ({}, dict(ws=A, nws=8), SMALL)])
def test_copy_refusals(L, so, change, args, status):
    a = dict(src=A, dst=A, n=3, count=None, ws=None, nws=0)
    a.update(args)
    p = planes(L, **change)
    assert so.locks_copy_pages(ctypes.byref(p), a["src"], a["dst"], a["n"], a["count"], a["ws"], a["nws"], None) == status
    assert so.locks_copy_pages(None, A, A, 0, None, None, 0, None) == INV


def pool_call(L, so, entry, d, change):
    """The entry with distinct arrays, far apart, but for `change`."""
    n = ctypes.c_size_t(0)
    assert so.locks_pool_workspace_size(ctypes.byref(d), ctypes.byref(n)) in (OK, UNSUP, INV)
    order = {"fork": ("table", "tokens", "parents", "refs", "table_out", "tokens_out", "refs_out", "src", "dst", "count"),
             "take": ("table", "tokens", "now", "refs", "tokens_out", "refs_out", "count"),
             "compact": ("table", "tokens", "refs", "table_out", "refs_out", "src", "dst", "cap", "count", "new")}[entry]
    a = {name: (2 + i) * A for i, name in enumerate(order)}
    a.update(cap=32, ws=64 * A, nws=n.value)
    a.update(change)
    fn = {"fork": so.locks_fork_sequences, "take": so.locks_take_pages, "compact": so.locks_compact_pages}[entry]
    return fn(ctypes.byref(d), *(a[k] for k in order), a["ws"], a["nws"], None)


COMMON = [(dict(ws=None, nws=0), SMALL), (dict(nws=300), SMALL), (dict(ws=A + 1), INV), (dict(table=None), INV),
          (dict(tokens=None), INV), (dict(refs=None), INV), (dict(refs_out=None), INV), (dict(refs=A + 4), INV),
          (dict(refs_out=A + 8), INV), (dict(tokens=A + 2), INV)]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(parents=None), INV), (dict(table_out=None), INV), (dict(tokens_out=None), INV), (dict(src=None), INV),
    (dict(dst=None), INV), (dict(count=None), INV), (dict(table_out=2 * A), INV), (dict(table_out=2 * A - 4), INV),
    (dict(tokens_out=3 * A), INV), (dict(refs_out=5 * A + 16), INV), (dict(src=10 * A - 4), INV), (dict(count=4 * A), INV),
    (dict(dst=2 * A + 4 * 39), INV)])
def test_fork_refusals(L, so, change, status):
    d = L.make_dims(4, 1, 1, 10, 64)
    assert pool_call(L, so, "fork", d, change) == status
    assert pool_call(L, so, "fork", L.make_dims(65537, 1, 1, 10, 64), {}) == UNSUP
    assert pool_call(L, so, "fork", L.make_dims(4, 1, 1, 1 << 28, 64), {}) == UNSUP
    assert pool_call(L, so, "fork", L.make_dims(4, 1, 1, 10, (1 << 30) + 1), {}) == UNSUP


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(now=None), INV), (dict(tokens_out=None), INV), (dict(tokens_out=3 * A + 4), INV), (dict(refs_out=5 * A + 16), INV),
    (dict(tokens_out=2 * A + 8), INV), (dict(count=5 * A), INV), (dict(count=A + 2), INV), (dict(table=5 * A), INV)])
def test_take_refusals(L, so, change, status):
    assert pool_call(L, so, "take", L.make_dims(4, 1, 1, 10, 64), change) == status
    assert pool_call(L, so, "take", L.make_dims(65537, 1, 1, 10, 64), {}) == UNSUP


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(table_out=None), INV), (dict(src=None), INV), (dict(dst=None), INV), (dict(count=None), INV),
    (dict(new=None), INV), (dict(cap=31), INV), (dict(cap=0), INV), (dict(table_out=2 * A + 4), INV),
    (dict(refs_out=4 * A + 16), INV), (dict(new=7 * A + 64), INV), (dict(dst=7 * A), INV)])
def test_compact_refusals(L, so, change, status):
    assert pool_call(L, so, "compact", L.make_dims(4, 1, 1, 10, 64), change) == status
    assert pool_call(L, so, "compact", L.make_dims(65537, 1, 1, 10, 64), {}) == UNSUP


@pytest.mark.parametrize("change,status", [
    (dict(pages=-1), INV), (dict(stride=-1), INV), (dict(rows=-1), INV), (dict(refs=None), INV), (dict(out=None), INV),
    (dict(lists=None), INV), (dict(counts=None), INV), (dict(refs=A + 4), INV), (dict(out=A + 8), INV),
    (dict(lists=A + 2), INV), (dict(out=2 * A + 16), INV), (dict(out=3 * A), INV), (dict(stride=(1 << 30) + 1), UNSUP),
    (dict(pages=(1 << 30) + 1), UNSUP), (dict(ws=A, nws=255), SMALL), (dict(ws=A + 1, nws=256), INV),
    (dict(pages=0, rows=0, refs=None, out=None, lists=None, counts=None), OK)])
def test_free_refusals(L, so, change, status):
    a = dict(refs=2 * A, pages=64, lists=3 * A, stride=8, counts=4 * A, rows=4, out=5 * A, ws=None, nws=0)
    a.update(change)
    assert so.locks_free_pages(a["refs"], a["pages"], a["lists"], a["stride"], a["counts"], a["rows"], a["out"], a["ws"],
                               a["nws"], None) == status


def test_binding_checks_types_shapes_and_layouts(L):
    d = L.make_dims(2, 4, 2, 8, 16)
    cache = torch.zeros(16, 2, 16, 128, dtype=torch.bfloat16)
    packed = torch.zeros(5, 2, 2432, dtype=torch.uint8)
    ids = torch.zeros(3, dtype=torch.int32)
    for change, err in ((dict(k=cache.float()), TypeError), (dict(v=cache[:8]), ValueError), (dict(src=ids.long()), TypeError),
                        (dict(n=4), ValueError), (dict(dst=ids[:2]), ValueError), (dict(packed=packed.float()), TypeError),
                        (dict(packed=packed[:, :1]), ValueError), (dict(packed=packed[:, :, :2400]), ValueError),
                        (dict(packed=packed.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                        (dict(src=torch.zeros(6, dtype=torch.int32)[::2]), ValueError), ({}, ValueError)):
        a = dict(k=cache, v=cache, src=ids, dst=None, n=3, packed=packed)
        a.update(change)
        with pytest.raises(err):
            L.locks_pack_pages(d, a["k"], a["v"], a["src"], a["dst"], a["n"], a["packed"])
        with pytest.raises(err):
            L.locks_unpack_pages(d, a["packed"], a["src"], a["dst"], a["n"], a["k"], a["v"])
    table, seq, q = torch.zeros(2, 8, dtype=torch.int32), ids[:2], torch.zeros(2, 4, 128)
    ws = torch.zeros(256, dtype=torch.uint8)
    sel = torch.zeros(2, 2, 3, dtype=torch.int32)
    for change, err in ((dict(q=q.half()), TypeError), (dict(q=q[:1]), ValueError), (dict(out=q), TypeError),
                        (dict(selected=sel[:, :1]), ValueError), (dict(selected=sel), TypeError),
                        (dict(selected=sel, n_selected=ids), ValueError), (dict(page_table=table[:, :3]), ValueError),
                        (dict(recent_table=table[:1]), ValueError), (dict(recent_table=table), TypeError),
                        (dict(recent_table=table, recent_tokens=seq, k_cache=cache), TypeError), ({}, ValueError)):
        a = dict(q=q, page_table=table, out=q.bfloat16())
        a.update(change)
        with pytest.raises(err):
            L.locks_packed_attention(d, a.pop("q"), packed, a.pop("page_table"), seq, a.pop("out"), ws, **a)
    for arrays in ([cache], [torch.zeros(3, 2)], [torch.zeros(())], [torch.zeros(4, 4)[:, ::2]], [cache] * 129):
        with pytest.raises(ValueError):           # the first: no CUDA tensors
            L.make_planes(arrays)
    with pytest.raises(ValueError, match="CUDA"):
        L.locks_copy_pages(L.make_planes([]), ids, ids)
    with pytest.raises(ValueError):
        L.locks_copy_pages(L.make_planes([]), ids, ids[:2])
    one, eight = torch.zeros(1, dtype=torch.int32), torch.zeros(16, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.locks_fork_sequences(d, table, seq, ids, eight, table, seq, eight, seq, seq, one, ws)
    with pytest.raises(TypeError):
        L.locks_take_pages(d, table, seq, seq.long(), eight, seq, eight, ws)
    with pytest.raises(ValueError):
        L.locks_free_pages(eight, ids, ids, eight)
    with pytest.raises(ValueError):
        L.locks_compact_pages(d, table, seq, eight[:9], table, eight, ids, ids, one, eight, ws)


# ----------------------------------------------------------------- the forms themselves

def test_codes_places_cover_the_unit_once():
    seen = set()
    for values in (0, 1):
        for t in range(16):
            for d in range(128):
                byte, bit = ref.place(t, d, values)
                assert 1024 * values <= byte < 1024 * (values + 1) and bit in (0, 4)
                seen.add((byte, bit))
    assert len(seen) == 2 * 16 * 128


def test_codes_are_within_half_a_step():
    x = ref.cache_ref.bf16(np.random.default_rng(0).normal(size=(50, 128)))
    for group in (32, 64):
        code, scale, zero = ref.codes_of(x, group)
        assert code.min() == 0 and code.max() == 15
        assert (np.abs(zero + scale * code - x) <= scale * (0.5 + 15 * 2.0 ** -8)).all()


def test_page_calls_keep_the_counts_of_holders():
    """Fork, take and compact of the loops: every page's count is the number of rows that hold it."""
    rng = np.random.default_rng(2)
    tokens = rng.integers(0, 60, 6)
    table, refs = np.full((6, 8), -1), np.zeros(80, np.int64)
    tokens_now, refs, left, short = ref.take(table, np.zeros(6, int), tokens, refs)
    assert not short and left == 80 - sum(ref.pages_of(n) for n in tokens)

    def held(table, tokens):
        n = np.zeros(80, np.int64)
        for b in range(6):
            np.add.at(n, table[b, :ref.pages_of(tokens[b])], 1)
        return n

    assert np.array_equal(held(table, tokens_now), refs)
    out, out_tokens = np.full((6, 8), -1), np.zeros(6, int)
    refs, src, dst, short = ref.fork(table, tokens_now, [0, 0, 3, 3, -1, 0], refs, out, out_tokens)
    assert not short and np.array_equal(held(out, out_tokens), refs) and not set(src) & set(dst)
    packed = np.full((6, 8), -1)
    refs, src, dst, new = ref.compact(out, out_tokens, refs, packed)
    assert np.array_equal(held(packed, out_tokens), refs) and not refs[(refs > 0).sum():].any()
