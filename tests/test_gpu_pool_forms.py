"""GPU tests of the page pool's calls on either side of the borders between one block and several launches:
pools of 8192 and 16384 pages, batches of 1024, tables of 64 pieces of 128 entries; exactly as in
test_gpu_pool."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import DEV
from tests.test_gpu_pool import OLD, check_compact, check_fork, check_take, dev, dims_of, filled, host, world

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pool", [(1, 1, 1), (64, 9, 8192), (64, 9, 8193), (65, 9, 8192), (32, 256, 8192), (32, 257, 8191),
                                              (1, 7000, 8190), (3, 2600, 8192)])
def test_fork_on_both_sides(batch, width, pool, in_place):
    rng = np.random.default_rng(pool + batch)
    most = min(width, max(1, pool // 2 // batch))
    tokens = rng.integers(0, 16 * most + 1, batch)
    table, refs = world(tokens, width, pool, batch, shared=most // 2, held=pool // 9)
    for parents in (rng.integers(-1, batch, batch), np.arange(batch), np.full(batch, batch // 2), np.arange(batch) // 4 * 4):
        check_fork(table, tokens, parents, refs, in_place)


def test_fork_without_enough_pages_in_one_block_and_in_two_launches():
    for batch, pool in ((60, 700), (70, 700), (60, 8300)):
        rng = np.random.default_rng(batch)
        tokens = rng.integers(1, 16 * 8, batch)
        table, refs = world(tokens, 8, pool, batch)
        spare = np.flatnonzero(refs == 0)
        refs[spare[7:]] = 1
        refs[spare[:3]] = -2                         # free as well
        check_fork(table, tokens, np.zeros(batch, np.int64) + 5, refs)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,pool", [(1, 16384), (200, 16384), (200, 16385), (1024, 9000), (1025, 9000), (1000, 12289)])
def test_take_on_both_sides(batch, pool, in_place):
    rng = np.random.default_rng(pool + batch)
    tokens = rng.integers(0, 16 * max(1, min(6, pool // 4 // batch)), batch)
    table, refs = world(tokens, 24, pool, batch, held=pool // 8)
    refs[rng.permutation(np.flatnonzero(refs == 0))[:5]] = -3
    for step in (1, 30, 24 * 16):                    # the last: more than there is, for the larger batches
        check_take(table, tokens, np.minimum(tokens + rng.integers(0, step + 1, batch), 24 * 16), refs, in_place)


def test_take_every_page_of_a_pool_of_one_block():
    refs = np.zeros(16384, np.int64)
    check_take(np.full((2, 16000), OLD), [0, 0], [16 * 16000, 16 * 384], refs)
    check_take(np.full((2, 16000), OLD), [0, 0], [16 * 16000, 16 * 385], refs)
    check_take(np.full((3, 16000), OLD), [0, 0, 0], [16 * 16000, 16 * 385, 0], refs)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pool,held", [(64, 9, 8192, 3000), (64, 9, 8193, 3000), (65, 9, 3000, 500), (30, 300, 4096, 100),
                                                   (1, 8000, 8192, 1), (16, 128, 8191, 4000), (4, 9, 4097, 4000)])
def test_compact_on_both_sides(batch, width, pool, held, in_place):
    rng = np.random.default_rng(pool + batch)
    tokens = rng.integers(0, 16 * min(width, max(1, (pool - held) // 2 // batch)) + 1, batch)
    table, refs = world(tokens, width, pool, batch, shared=2, held=held)
    check_compact(table, tokens, refs, in_place)


def test_compact_full_empty_and_settled_pools_of_one_block():
    n = 8192
    half = np.r_[np.ones(n // 2), np.zeros(n // 2)]
    for refs in (np.ones(n), np.zeros(n), half, half[::-1], np.r_[np.zeros(n - 1), 1], np.r_[1, np.zeros(n - 1)], np.arange(n) % 2):
        check_compact(np.zeros((0, 3), np.int64), [], refs.astype(np.int64))


@pytest.mark.parametrize("pool", [40, 9000])
def test_bad_input_in_either_form(pool):
    """What a form does with counts and ids out of range is the same for a small pool and a large one."""
    tokens = [20, 30, 40]
    table, refs = world(tokens, 6, 40, 3)
    refs = np.r_[refs, np.ones(pool - 40, np.int64)]
    d = dims_of(3, 6, pool)

    def compact(t, n):
        ws = L.alloc_pool_workspace(d, DEV)
        to, ro, cap = filled(3, 6), filled(pool), pool // 2
        src, dst, m, new = filled(cap), filled(cap), filled(1), filled(pool)
        L.locks_compact_pages(d, dev(t), dev(n), dev(refs), to, ro, src, dst, m, new, ws)
        return L.locks_get_device_status(ws), host(to)

    want = compact(table, tokens)
    assert want[0] == 0
    for value in (-1, 97):
        status, got = compact(table, [20, value, 40])
        assert status == -6 and (got[1] == OLD).all() and np.array_equal(got[[0, 2]], want[1][[0, 2]])
    wrong = table.copy()
    wrong[1, 0] = pool
    status, got = compact(wrong, tokens)
    assert status == -6 and got[1, 0] == pool and np.array_equal(got[1, 1:], want[1][1, 1:])
