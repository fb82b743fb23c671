"""GPU tests of page calls that have nothing to do and a count to refuse: what the device reads is checked
all the same."""

import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def fresh_ws():
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("num", [0, 5])
@pytest.mark.parametrize("in_place", [True, False])
def test_free_counts_of_lists_without_entries(num, in_place):
    lists = torch.zeros((3, 0), dtype=torch.int32, device=DEV)
    for counts, status in (([0, 0, 0], 0), ([0, 2, 0], -6), ([0, 0, -1], -6), ([1, 0, 0], -6)):
        refs, ws = i32(list(range(num))), fresh_ws()
        out = refs if in_place else torch.full_like(refs, 9)
        L.locks_free_pages(refs, lists, i32(counts), out, workspace=ws)
        assert L.locks_get_device_status(ws) == status
        assert out.tolist() == list(range(num))


def planes_of(kind):
    if kind == "none":
        return L.make_planes([])
    return L.make_planes([torch.zeros((4, 0 if kind == "no bytes" else 16), dtype=torch.uint8, device=DEV)])


@pytest.mark.parametrize("kind,pairs", [("some", 0), ("no bytes", 2), ("no bytes", 0), ("none", 2), ("none", 0)])
def test_copy_counts_where_nothing_is_copied(kind, pairs):
    ids = torch.arange(pairs, dtype=torch.int32, device=DEV)
    for n, status in ((0, 0), (pairs, 0), (pairs + 1, -6), (-1, -6), (2 ** 31 - 1, -6)):
        ws = fresh_ws()
        L.locks_copy_pages(planes_of(kind), ids, ids, n_pairs=i32([n]), workspace=ws)
        assert L.locks_get_device_status(ws) == status
