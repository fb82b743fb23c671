"""The cache operators' binding: what it does around the C entry points."""
import ctypes

import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

ENTRIES = ("locks_append_tokens", "locks_prefix_attention", "locks_accumulate_mass", "locks_evict_pages")


@pytest.fixture
def entries():
    """Puts another function in place of the four entry points."""
    lib = L.cache.load_library()
    from sparse_kv_page_gb300 import _marshal

    def bind(address):
        _marshal.bind(*([address] * 4))

    yield bind
    _marshal.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ENTRIES))


def test_other_threads_run_during_a_call(entries):
    """The interpreter's lock is free while an entry point runs. In its place: the interpreter's own
    question whether this thread holds the lock, whose answer (1 or 0) comes back as the status."""
    d = L.make_dims(1, 2, 1, 4, 4)
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = torch.zeros((4, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((1, 1, 128), device=DEV)
    table, one, rows = torch.zeros((1, 4), **i32), torch.zeros(1, **i32), torch.zeros((1, 4), device=DEV)
    q = torch.zeros((1, 2, 128), device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    entries(ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value)
    L.locks_append_tokens(d, None, None, kv, kv, None, one, table, None, cache, cache)
    L.locks_prefix_attention(d, q, cache, cache, None, None, None, table, one, q.bfloat16(), ws)
    L.locks_accumulate_mass(d, torch.zeros((1, 2, 4), device=DEV), one, rows, rows, ws)
    L.locks_evict_pages(d, rows, table, one, 4, rows, table, one, torch.zeros((1, 1), **i32), one)
