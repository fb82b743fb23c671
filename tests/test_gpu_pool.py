"""GPU tests of the page pool's calls against the loops in pool_ref. Everything is whole numbers,
so results are compared exactly; entries that a call does not write keep what was in them."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
OLD = -77                                            # in entries that a call may leave alone


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


def host(t):
    return t.cpu().numpy()


def dims_of(batch, width, pool):
    return L.make_dims(batch, 1, 1, width, pool)


def filled(*shape):
    return torch.full(shape, OLD, dtype=torch.int32, device=DEV)


def world(tokens, width, pool, seed, shared=0, held=0):
    """A pool in which row b holds ceil(tokens[b] / 16) pages, of which the first `shared` full ones are
    those of row 0, and `held` more pages are somebody else's."""
    rng = np.random.default_rng(seed)
    order = list(rng.permutation(pool))
    table = np.full((len(tokens), width), OLD, np.int64)
    refs = np.zeros(pool, np.int64)
    for b, n in enumerate(tokens):
        for j in range(ref.pages_of(n)):
            common = b > 0 and j < shared and j < n // 16 and j < tokens[0] // 16
            table[b, j] = table[0, j] if common else order.pop()
            refs[table[b, j]] += 1
    for _ in range(held):
        refs[order.pop()] += rng.integers(1, 4)
    return table, refs


def call_fork(table, tokens, parents, refs, status=0, in_place=False):
    B, P = table.shape
    d, ws = dims_of(B, P, len(refs)), None
    ws = L.alloc_pool_workspace(d, DEV)
    to, so, src, dst, n = filled(B, P), filled(B), filled(B), filled(B), filled(1)
    r = dev(refs)
    ro = r if in_place else filled(len(refs))
    L.locks_fork_sequences(d, dev(table), dev(tokens), dev(parents), r, to, so, ro, src, dst, n, ws)
    assert L.locks_get_device_status(ws) == status
    return [host(x) for x in (to, so, ro, src, dst, n)]


def check_fork(table, tokens, parents, refs, in_place=False):
    B, P = table.shape
    want_t, want_s = np.full((B, P), OLD), np.full(B, OLD)
    new, src, dst, short = ref.fork(table, tokens, parents, refs, want_t, want_s)
    got = call_fork(table, tokens, parents, refs, -7 if short else 0, in_place)
    pad = [OLD] * (B - len(src))
    for g, w in zip(got, (want_t, want_s, new, src + pad, dst + pad, [len(src)])):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_parents_of_every_kind(in_place):
    tokens = [37, 64, 0, 5, 100, 16]
    table, refs = world(tokens, 7, 60, 1, shared=2, held=5)
    for parents in ([0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [0] * 6, [3] * 6, [-1] * 6, [1, 1, 1, 0, 0, 4],
                    [-1, 0, 0, -1, 4, 4], [2, 2, 5, 5, 0, 0]):
        check_fork(table, tokens, parents, refs, in_place)


@pytest.mark.parametrize("batch,pool", [(1, 3), (33, 400), (300, 9000), (1025, 20000), (5000, 40000)])
def test_fork_sizes(batch, pool):
    rng = np.random.default_rng(batch)
    tokens = rng.integers(0, 90, batch)
    table, refs = world(tokens, 6, pool, batch, shared=3, held=pool // 10)
    check_fork(table, tokens, rng.integers(-1, batch, batch), refs)
    check_fork(table, tokens, rng.integers(0, max(1, batch // 8), batch), refs)


def test_fork_long_rows():
    tokens = [70001, 16 * 4400, 3, 0]
    table, refs = world(tokens, 4400, 150001, 5, shared=4000, held=1000)
    check_fork(table, tokens, [0, 0, 0, 1], refs)
    check_fork(table, tokens, [1, 0, -1, 2], refs)


def test_fork_without_enough_pages():
    tokens = [37, 20, 48, 9]
    table, refs = world(tokens, 4, 12, 7)
    for held in range(4):                            # free pages left: 3, 2, 1, 0
        full = refs.copy()
        full[np.flatnonzero(refs == 0)[:held]] = 1
        check_fork(table, tokens, [0, 0, 0, 1], full)
        check_fork(table, tokens, [0, 1, 1, 1], full)


def test_fork_bad_input():
    tokens = np.array([37, 20, 48, 9])
    table, refs = world(tokens, 4, 30, 8)
    kept, kept_t = tokens.copy(), table.copy()
    for value in (-1, 65, 2 ** 31 - 1):              # counts as no tokens
        wrong, zero = kept.copy(), kept.copy()
        wrong[1], zero[1] = value, 0
        got, want = call_fork(table, wrong, [1, 1, 2, 0], refs, -6), call_fork(table, zero, [1, 1, 2, 0], refs)
        assert all(np.array_equal(x, y) for x, y in zip(got, want))
    for value in (-2, 4, 2 ** 31 - 1):               # counts as none
        got, want = call_fork(table, kept, [0, value, 2, 3], refs, -6), call_fork(table, kept, [0, -1, 2, 3], refs)
        assert all(np.array_equal(x, y) for x, y in zip(got, want))
    for value in (-5, 30):                           # handed on, not counted
        table = kept_t.copy()
        table[2, 1] = value
        got = call_fork(table, kept, [2, 2, -1, -1], refs, -6)
        assert got[0][0, 1] == got[0][1, 1] == value


def call_take(table, tokens, now, refs, status=0, in_place=False, count=True):
    B, P = table.shape
    d = dims_of(B, P, len(refs))
    ws = L.alloc_pool_workspace(d, DEV)
    t, s, r, n = dev(table), dev(tokens), dev(refs), filled(1)
    so, ro = (s, r) if in_place else (filled(B), filled(len(refs)))
    L.locks_take_pages(d, t, s, dev(now), r, so, ro, ws, n_free=n if count else None)
    assert L.locks_get_device_status(ws) == status
    return host(t), host(so), host(ro), host(n)


def check_take(table, tokens, now, refs, in_place=False):
    want_t = table.copy()
    so, ro, left, short = ref.take(want_t, np.asarray(tokens), np.asarray(now), refs)
    got = call_take(table, tokens, now, refs, -7 if short else 0, in_place)
    for g, w in zip(got, (want_t, so, ro, [left])):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("in_place", [False, True])
def test_take_growth_of_every_kind(in_place):
    tokens = [0, 0, 15, 16, 17, 100]
    now = [0, 1, 16, 17, 33, 160]
    table, refs = world(tokens, 12, 64, 1, held=20)
    check_take(table, tokens, now, refs, in_place)
    check_take(table, tokens, tokens, refs, in_place)
    check_take(table, tokens, [16 * 12] * 6, refs, in_place)      # more than there is


@pytest.mark.parametrize("batch,pool", [(1, 1), (1, 5), (70, 129), (300, 8191), (3000, 70000), (5000, 140001)])
def test_take_sizes(batch, pool):
    rng = np.random.default_rng(pool)
    tokens = rng.integers(0, 16 * max(1, min(6, pool // 2 // batch)), batch)
    table, refs = world(tokens, 24, pool, batch, held=pool // 8)
    for step in (1, 30, 200):
        check_take(table, tokens, np.minimum(tokens + rng.integers(0, step + 1, batch), 24 * 16), refs)


def test_take_a_whole_large_pool():
    pool = 300007
    refs = np.zeros(pool, np.int64)
    refs[::3] = 1
    table = np.full((2, 150000), OLD)
    check_take(table, [0, 0], [16 * 150000 - 3, 16 * 50000], refs)
    check_take(table, [0, 0], [16 * 150000 - 3, 16 * 50006], refs)      # one page too many for the second


def test_take_bad_input():
    tokens, now = [20, 30, 40], [50, 60, 70]
    table, refs = world(tokens, 6, 40, 3)
    for b, t, n in ((1, -1, 60), (1, 97, 97), (1, 30, 97), (1, 30, 29), (1, 30, -1), (0, 2 ** 31 - 1, 50)):
        wt, wn = list(tokens), list(now)
        wt[b], wn[b] = t, n
        st, sn = list(tokens), list(now)
        sn[b] = st[b]                                # as if it did not grow
        got, want = call_take(table, wt, wn, refs, -6), call_take(table, st, sn, refs)
        want[1][b] = t                               # its count is handed on
        assert all(np.array_equal(x, y) for x, y in zip(got, want))


def call_free(refs, lists, counts, status=0, in_place=False):
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    r = dev(refs)
    ro = r if in_place else filled(len(refs))
    L.locks_free_pages(r, dev(lists).view(len(counts), -1), dev(counts), ro, workspace=ws)
    assert L.locks_get_device_status(ws) == status
    return host(ro)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,stride,pool", [(1, 1, 1), (3, 7, 20), (70, 33, 4000), (5, 5000, 30001), (20000, 3, 100000)])
def test_free(rows, stride, pool, in_place):
    rng = np.random.default_rng(rows)
    lists, counts = rng.integers(0, pool, (rows, stride)), rng.integers(0, stride + 1, rows)
    want = rng.integers(0, 3, pool)
    refs = want.copy()
    for r, n in enumerate(counts):
        np.add.at(refs, lists[r, :n], 1)
    lists[np.arange(stride) >= counts[:, None]] = -9             # not read
    assert np.array_equal(call_free(refs, lists, counts, 0, in_place), want)


def test_free_bad_input():
    refs = [2, 1, 0, 5]
    assert np.array_equal(call_free(refs, [[0, 4, 1], [3, -1, 0]], [3, 2], -6), [1, 0, 0, 4])
    assert np.array_equal(call_free(refs, [[0, 1, 3], [3, 3, 0]], [4, 2], -6), [2, 1, 0, 3])
    assert np.array_equal(call_free(refs, [[0, 1, 3], [3, 3, 0]], [-1, 1], -6), [2, 1, 0, 4])
    assert np.array_equal(call_free(refs, [[2, 1, 1], [1, 0, 0]], [3, 3], -6), [0, 0, 0, 5])     # freed too often
    assert np.array_equal(call_free(refs, [[], []], [0, 0]), refs)


def call_compact(table, tokens, refs, status=0, in_place=False):
    B, P = table.shape
    pool = len(refs)
    d = dims_of(B, P, pool)
    ws = L.alloc_pool_workspace(d, DEV)
    t, r, cap = dev(table), dev(refs), max(1, pool // 2)
    to, ro = (t, r) if in_place else (filled(B, P), filled(pool))
    src, dst, n, new = filled(cap), filled(cap), filled(1), filled(pool)
    L.locks_compact_pages(d, t, dev(tokens), r, to, ro, src, dst, n, new, ws)
    assert L.locks_get_device_status(ws) == status
    return [host(x) for x in (to, ro, src, dst, n, new)]


def check_compact(table, tokens, refs, in_place=False):
    want_t = table.copy() if in_place else np.full(table.shape, OLD)
    after, src, dst, new = ref.compact(table, tokens, refs, want_t)
    got = call_compact(table, tokens, refs, 0, in_place)
    pad = [OLD] * (max(1, len(refs) // 2) - len(src))
    for g, w in zip(got, (want_t, after, src + pad, dst + pad, [len(src)], new)):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,pool,held", [(1, 1, 0), (1, 2, 1), (4, 40, 3), (20, 130, 9), (60, 8193, 50),
                                             (200, 40001, 3000), (50, 200003, 100000)])
def test_compact(batch, pool, held, in_place):
    rng = np.random.default_rng(pool)
    tokens = rng.integers(0, 16 * max(1, min(40, (pool - held) // batch)) + 1, batch) if pool > 2 else [0]
    table, refs = world(tokens, 41, pool, batch, shared=2, held=held)
    check_compact(table, tokens, refs, in_place)


def test_compact_full_empty_and_settled_pools():
    for refs in (np.ones(300), np.zeros(300), np.r_[np.ones(128), np.zeros(200)], np.r_[np.zeros(200), np.ones(200)],
                 np.r_[np.zeros(64), np.ones(1)]):
        check_compact(np.zeros((0, 3), np.int64), [], refs.astype(np.int64))


def test_compact_bad_input():
    tokens = [20, 30]
    table, refs = world(tokens, 3, 20, 4)
    want = call_compact(table, [20, 0], refs)
    for n in (-1, 49):
        got = call_compact(table, [20, n], refs, -6)
        assert all(np.array_equal(x, y) for x, y in zip(got, want))
    table[1, 0] = 20
    assert call_compact(table, tokens, refs, -6)[0][1, 0] == 20


# ------------------------------------------------------------------ copies

def arrays(pages, seed, hkv=2):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def some(*shape, dtype=torch.uint8):
        return torch.randint(0, 100, (pages,) + shape, generator=g, device=DEV).to(dtype)

    # K, V, packed pages, the four of the summaries of one kv head (their scales are 8 bytes), odd sizes
    return [some(hkv, 16, 128, dtype=torch.bfloat16), some(hkv, 16, 128, dtype=torch.int16), some(hkv, 2432), some(1, 128),
            some(1, 512), some(1, 4, dtype=torch.int16), some(3, dtype=torch.float64), some(16408), some(40000)]


@pytest.mark.parametrize("pages,n", [(2, 1), (9, 4), (300, 120)])
def test_copy_pages(pages, n):
    xs = arrays(pages, n)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n], order[n:2 * n]
    want = [host(x.view(torch.uint8) if x.dim() == 1 else x.view(pages, -1).view(torch.uint8)).copy() for x in xs]
    for w in want:
        w[dst] = w[src]
    L.locks_copy_pages(L.make_planes(xs), dev(src), dev(dst))
    for x, w in zip(xs, want):
        assert np.array_equal(host(x.view(pages, -1).view(torch.uint8)), w)


def test_copy_counts_padding_and_bad_ids():
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    x = torch.arange(10, device=DEV).view(10, 1)
    planes = L.make_planes([x])

    def after(src, dst, n=None, status=0):
        x.copy_(torch.arange(10, device=DEV).view(10, 1))
        ws.zero_()
        L.locks_copy_pages(planes, dev(src), dev(dst), None if n is None else dev([n]), workspace=ws)
        assert L.locks_get_device_status(ws) == status
        return {i: int(v) for i, v in enumerate(x[:, 0]) if int(v) != i}

    assert after([1, 2, 3], [4, 5, 6]) == {4: 1, 5: 2, 6: 3}
    assert after([1, 2, 3], [4, 5, 6], 2) == {4: 1, 5: 2}
    assert after([1, 2, 3], [4, 5, 6], 0) == {}
    assert after([1, -1, 3], [4, 5, -4]) == {4: 1}
    for n in (-1, 4, 2 ** 31 - 1):
        assert after([1, 2, 3], [4, 5, 6], n, status=-6) == {}
    assert after([1, 10, 3], [4, 5, 6], status=-6) == {4: 1, 6: 3}
    assert after([1, 2, 3], [4, 2 ** 31 - 1, 6], status=-6) == {4: 1, 6: 3}
    L.locks_copy_pages(L.make_planes([]), dev([1]), dev([2]))
    L.locks_copy_pages(planes, dev([]), dev([]))


def test_copy_past_2_31_bytes():
    x = torch.empty((150000, 4096), dtype=torch.int32, device=DEV)
    x[5], x[149999] = 7, 9
    y = torch.empty((150000, 1), dtype=torch.float64, device=DEV)
    y[5], y[149999] = 0.5, 1.5
    L.locks_copy_pages(L.make_planes([x, y]), dev([149999, 5]), dev([1, 149998]))
    assert (x[1] == 9).all() and (x[149998] == 7).all() and float(y[1]) == 1.5 and float(y[149998]) == 0.5


def test_calls_follow_a_captured_graph():
    """Take, fork and copy captured once and replayed on other counts and parents."""
    B, P, pool = 4, 6, 40
    tokens = np.array([37, 20, 0, 9])
    table, refs = world(tokens, P, pool, 3)
    d = dims_of(B, P, pool)
    ws = L.alloc_pool_workspace(d, DEV)
    t, s, now, par, r = dev(table), dev(tokens), dev(tokens), dev([0, 1, 2, 3]), dev(refs)
    mid, to, so, ro, src, dst, n, s2 = (filled(pool), filled(B, P), filled(B), filled(pool), filled(B), filled(B), filled(1),
                                        filled(B))
    x = torch.zeros((pool, 4), dtype=torch.int32, device=DEV)
    planes = L.make_planes([x])

    def calls():
        L.locks_take_pages(d, t, s, now, r, s2, mid, ws)
        L.locks_fork_sequences(d, t, s2, par, mid, to, so, ro, src, dst, n, ws)
        L.locks_copy_pages(planes, src, dst, n)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    for grown, parents in (([40, 50, 3, 9], [0, 0, 2, 2]), ([37, 20, 96, 9], [3, 2, 1, 0]), ([80, 20, 5, 10], [1, 1, 1, 1])):
        t.copy_(dev(table))
        now.copy_(dev(grown))
        par.copy_(dev(parents))
        for o in (to, so, src, dst):
            o.fill_(OLD)
        x.copy_(torch.arange(pool, device=DEV, dtype=torch.int32).view(pool, 1).expand(pool, 4))
        graph.replay()
        wt = table.copy()
        ws_, wr, _, short = ref.take(wt, tokens, np.array(grown), refs)
        want_t, want_s = np.full((B, P), OLD), np.full(B, OLD)
        new, fs, fd, lacking = ref.fork(wt, ws_, parents, wr, want_t, want_s)
        assert not short and not lacking
        assert np.array_equal(host(to), want_t) and np.array_equal(host(so), want_s) and np.array_equal(host(ro), new)
        moved = np.arange(pool)
        moved[fd] = fs
        assert np.array_equal(host(x)[:, 0], moved) and np.array_equal(host(x)[:, 3], moved)
    assert L.locks_get_device_status(ws) == 0
