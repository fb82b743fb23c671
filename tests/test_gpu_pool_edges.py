"""GPU tests of the page pool's calls at the ends of their ranges: tables, needs and lists whose counts
pass 31 bits, and calls with nothing to do."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV
from tests.test_gpu_pool import OLD, dev, dims_of, filled, host

pytestmark = pytest.mark.gpu


def need_memory(num_bytes):
    if torch.cuda.mem_get_info()[0] < num_bytes + 2 ** 30:
        pytest.skip("not enough device memory")


def test_compact_a_table_of_more_threads_than_31_bits():
    """65536 rows of 33 pieces are 2^31 threads and more; only the last row holds pages."""
    batch, width, pool = 65536, 33 * 4096, 64
    need_memory(4 * batch * width)
    table = torch.empty((batch, width), dtype=torch.int32, device=DEV)
    tokens = np.zeros(batch, np.int64)
    tokens[-1] = 40
    table[-1, :4] = dev([50, 3, 63, OLD])
    refs = np.zeros(pool, np.int64)
    refs[[50, 3, 63]] = [1, 2, 3]
    d = dims_of(batch, width, pool)
    src, dst, n, new, ro = filled(32), filled(32), filled(1), filled(pool), filled(pool)
    ws = L.alloc_pool_workspace(d, DEV)
    L.locks_compact_pages(d, table, dev(tokens), dev(refs), table, ro, src, dst, n, new, ws)
    assert L.locks_get_device_status(ws) == 0
    assert host(n).tolist() == [3] and host(src).tolist()[:4] == [3, 50, 63, OLD] and host(dst).tolist()[:4] == [0, 1, 2, OLD]
    assert host(table[-1, :4]).tolist() == [1, 0, 2, OLD]
    assert host(ro).tolist() == [2, 1, 3] + [0] * (pool - 3)


def test_take_needs_of_more_than_31_bits():
    """17 rows want 2^27 - 1 pages each: nobody gets any, and nobody's count changes."""
    batch, width, pool = 17, 2 ** 27 - 1, 5000
    need_memory(4 * batch * width)
    table = torch.empty((batch, width), dtype=torch.int32, device=DEV)
    table[:, :8] = OLD
    d = dims_of(batch, width, pool)
    refs, tokens, n = dev(np.zeros(pool)), dev([0] * 16 + [20]), filled(1)
    more = np.full(batch, 16 * width)
    for now, free in ((more, pool), (np.r_[33, more[1:]], pool - 3)):
        out, ro = filled(batch), filled(pool)
        ws = L.alloc_pool_workspace(d, DEV)
        L.locks_take_pages(d, table, tokens, dev(now), refs, out, ro, ws, n_free=n)
        assert L.locks_get_device_status(ws) == -7
        first = 33 if free < pool else 0
        assert host(out).tolist() == [first] + [0] * 15 + [20] and host(n).tolist() == [free]
        assert host(ro).sum() == pool - free
    want = np.full((batch, 8), OLD)
    want[0, :3] = [0, 1, 2]
    assert np.array_equal(host(table[:, :8]), want)


def test_calls_with_nothing_to_do():
    none, some = filled(0), filled(8)
    ws = L.alloc_pool_workspace(dims_of(1, 1, 1), DEV)
    lib, p = L.pool.load_library(), lambda t: t.data_ptr()
    lists, counts = dev([[-1, 3]]), dev([0])
    # a pool without pages, whose counts go elsewhere
    assert lib.locks_free_pages(p(some), 0, p(lists), 2, p(counts), 1, p(some) + 16, p(ws), 256, 0) == 0
    torch.cuda.synchronize()
    assert L.locks_get_device_status(ws) == 0 and host(some).tolist() == [OLD] * 8
    # pages of no bytes
    planes = L.make_planes([torch.empty((5, 0), dtype=torch.uint8, device=DEV)])
    L.locks_copy_pages(planes, dev([0]), dev([1]), None, ws)
    L.locks_free_pages(none, dev(np.zeros((0, 3))), none, none, ws)
    assert L.locks_get_device_status(ws) == 0


def test_fork_records_a_bad_id_of_a_row_with_one_child():
    table, refs = np.array([[0, 99], [2, 3]]), np.array([1, 0, 1, 1])
    d = dims_of(2, 2, 4)
    ws, to, so, ro, src, dst, n = (L.alloc_pool_workspace(d, DEV), filled(2, 2), filled(2), filled(4), filled(2), filled(2),
                                   filled(1))
    L.locks_fork_sequences(d, dev(table), dev([32, 32]), dev([0, 1]), dev(refs), to, so, ro, src, dst, n, ws)
    assert L.locks_get_device_status(ws) == -6
    assert np.array_equal(host(to), table) and np.array_equal(host(ro), refs) and host(n).tolist() == [0]


@pytest.mark.parametrize("pool", [70, 9000])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_clears_counts_below_zero(pool, in_place):
    refs = np.full(pool, -2, np.int64)
    refs[[5, pool - 1]] = [3, 4]
    d, cap = dims_of(0, 1, pool), pool // 2
    r, src, dst, n, new = dev(refs), filled(cap), filled(cap), filled(1), filled(pool)
    ro = r if in_place else filled(pool)
    ws = L.alloc_pool_workspace(d, DEV)
    L.locks_compact_pages(d, filled(0, 1), filled(0), r, filled(0, 1), ro, src, dst, n, new, ws)
    assert L.locks_get_device_status(ws) == 0
    assert host(n).tolist() == [2] and host(src).tolist()[:2] == [5, pool - 1] and host(dst).tolist()[:2] == [0, 1]
    assert host(ro).tolist() == [3, 4] + [0] * (pool - 2)


def test_attention_over_large_zeros_and_tiny_scales():
    """The first 64 dims of all values are 2^40 and the others below 2^-86: weights grow with the scales,
    and their products with the zeros are numbers still. (Scales below 2^-49 count as fp16 numbers of
    2^-54: a value's error is at most 15 * 2^-25 * 2^-54, and 2^10 tokens of them less than 2^-60.)"""
    from tests.test_gpu_packed import make_case, run, tokens_of, f64
    from tests import pool_ref as ref
    c = make_case([40], [0], 8, 2, seed=31)
    fields = c["packed"][..., 2304:].contiguous().view(torch.bfloat16).view(*c["packed"].shape[:2], 16, 4)
    fields[..., 0], fields[..., 1], fields[..., 2], fields[..., 3] = 0.0, 2.0 ** -90, 2.0 ** 40, 2.0 ** -87
    c["packed"][..., 2304:] = fields.view(*c["packed"].shape[:2], 64).view(torch.uint8)
    run(c)
    assert L.locks_get_device_status(c["ws"]) == 0
    got, units, table = f64(c["out"]), c["packed"].cpu().numpy(), c["table"].cpu().numpy()
    assert (np.abs(got[0, :, :64] - 2.0 ** 40) <= 2.0 ** 32).all()
    for h in range(2):
        want, want_lse, _, size = ref.attend(f64(c["q"])[0, 4 * h:4 * h + 4], *tokens_of(c, 0, h, units, table))
        assert (np.abs(got[0, 4 * h:4 * h + 4, 64:] - want[:, 64:]) <= 2.0 ** -60).all()
        assert (np.abs(f64(c["lse"])[0, 4 * h:4 * h + 4] - want_lse) <= 2.0 ** -15 * size + 2.0 ** -16).all()
