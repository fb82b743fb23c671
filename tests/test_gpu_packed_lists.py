"""GPU tests of attention over packed pages by lists, where the tables are so wide that the call goes by
the line of all rows' steps (a row of 20000 entries takes a cluster of eight CTAs 140 us by the fit, the
line 41 for four): lengths by kv head, heads and sequences with nothing in between."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.test_gpu_packed import DEV, check, make_case

pytestmark = pytest.mark.gpu

WIDE = 20000


def wide(c, cap):
    """The same lists in rows of `cap` entries, ids that nobody may read behind them."""
    old = c["sel"]
    c["sel"] = torch.full(old.shape[:2] + (cap,), -7, dtype=torch.int32, device=DEV)
    c["sel"][..., :old.shape[2]] = old
    return c


def lists_of(pages, hkv, seed, most, empty):
    """Random lists, a share of them empty."""
    rng = np.random.default_rng(seed)
    out = []
    for n in pages:
        row = []
        for _ in range(hkv):
            k = 0 if n == 0 or rng.random() < empty else rng.integers(1, most + 1)
            row.append([int(x) for x in rng.integers(0, max(n, 1), k)])
        out.append(row)
    return out


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (16, 2), (5, 1), (32, 2), (9, 1)])
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_lists_on_the_line(hq, hkv, q_type):
    pages = [50, 7, 333, 0, 40]
    lists = lists_of(pages, hkv, hq, 300, 0.2)
    lists[4][0] = []                                 # the last sequence's first head
    lists[4][-1] = [0, 39] * 70 if hkv > 1 else []
    check(wide(make_case(pages, [3, 0, 29, 0, 0], hq, hkv, seed=hq, q_type=q_type, selected=lists), WIDE))
    check(wide(make_case(pages, [0, 0, 40, 17, 1], hq, hkv, seed=hq + 1, q_type=q_type, selected=lists), WIDE))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 2), (32, 2)])
def test_many_sequences_with_lists(hq, hkv):
    """More sequences than a CTA has threads, most heads empty, whole runs of sequences too."""
    n = 1100
    pages = [(b * 7) % 5 if b % 90 < 50 else 0 for b in range(n)]
    recent = [b % 19 if b % 12 == 0 and b % 90 < 60 else 0 for b in range(n)]
    check(wide(make_case(pages, recent, hq, hkv, seed=4, width=5, selected=lists_of(pages, hkv, 9, 6, 0.6)), 3000))


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("n", [64, 1500])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 2)])
def test_two_sequences_at_the_ends_of_a_batch(hq, hkv, n, lists):
    """Slots between that nobody uses."""
    pages = [0] * n
    pages[0], pages[-1] = 60, 41
    c = make_case(pages, [0] * (n - 1) + [9], hq, hkv, seed=5, width=64,
                  selected=[[list(range(p)) for _ in range(hkv)] for p in pages] if lists else None)
    check(wide(c, 3000) if lists else c)


def test_a_full_batch_of_short_selections():
    """96 sequences of 8 kv heads, up to 128 chosen pages each: rows that lie in two CTAs each."""
    rng = np.random.default_rng(1)
    n, hkv = 96, 8
    pages = [int(x) for x in rng.integers(1, 60, n)]
    lists = [[[int(x) for x in rng.integers(0, p, rng.integers(0, 9))] for _ in range(hkv)] for p in pages]
    lists[7] = [[int(x) for x in rng.integers(0, pages[7], 128)] for _ in range(hkv)]
    lists[50][3] = [int(x) for x in rng.integers(0, pages[50], 128)]
    check(make_case(pages, [b % 21 for b in range(n)], 32, hkv, seed=6, selected=lists))


@pytest.mark.parametrize("lists", [False, True])
def test_unused_slots_are_not_gone_through_one_by_one(lists):
    """4096 slots, the first and the last in use: 0.05 and 0.08 ms a call, against 0.014 ms for those two
    alone; 8 ms and more where a CTA looks at every row between them."""
    n, hkv, pages = 4096, 8, [101, 64]       # steps 0 .. 808 and 808 .. 1320 of 83 CTAs: one has both ends
    packed = torch.zeros((sum(pages), hkv, L.LOCKS_PACKED_BYTES), dtype=torch.uint8, device=DEV)
    table = torch.zeros((n, 512), dtype=torch.int32, device=DEV)
    counts = torch.zeros(n, dtype=torch.int32, device=DEV)
    for b, first, k in ((0, 0, pages[0]), (n - 1, pages[0], pages[1])):
        table[b, :k] = torch.arange(first, first + k, device=DEV)
        counts[b] = k
    dims = L.make_dims(n, 4 * hkv, hkv, 512, 1)
    ws = L.alloc_packed_workspace(dims, DEV)
    q, out = torch.ones((n, 4 * hkv, 128), device=DEV), torch.ones((n, 4 * hkv, 128), dtype=torch.bfloat16, device=DEV)
    kw = {}
    if lists:
        kw = dict(selected=torch.arange(512, dtype=torch.int32, device=DEV).expand(n, hkv, 512).contiguous(),
                  n_selected=counts[:, None].expand(n, hkv).contiguous())
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(7):
        if i == 2:
            start.record()
        L.locks_packed_attention(dims, q, packed, table, counts, out, ws, **kw)
    end.record()
    torch.cuda.synchronize()
    assert L.locks_get_device_status(ws) == 0 and float(out.abs().max()) == 0
    assert start.elapsed_time(end) / 5 < 1
