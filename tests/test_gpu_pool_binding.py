"""The binding of the packed cache and the page pool: what it does around the C entry points."""
import ctypes

import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

ENTRIES = ("locks_pack_pages", "locks_unpack_pages", "locks_packed_attention", "locks_copy_pages", "locks_fork_sequences",
           "locks_take_pages", "locks_free_pages", "locks_compact_pages")


@pytest.fixture
def entries():
    """Puts another function in place of the eight entry points."""
    lib = L.pool.load_library()
    from sparse_kv_page_gb300 import _marshal

    yield lambda address: _marshal.bind_pool(*([address] * 8))
    _marshal.bind_pool(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ENTRIES))


def zeros(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def arguments():
    d = L.make_dims(1, 2, 1, 4, 4)
    cache = torch.zeros((4, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
    packed = torch.zeros((4, 1, L.LOCKS_PACKED_BYTES), dtype=torch.uint8, device=DEV)
    return d, cache, packed, L.alloc_pool_workspace(d, DEV)


def test_other_threads_run_during_a_call(entries):
    """The interpreter's lock is free while an entry point runs. In its place: the interpreter's own
    question whether this thread holds the lock, whose answer (1 or 0) comes back as the status."""
    d, cache, packed, ws = arguments()
    table, one, four, q = zeros(1, 4), zeros(1), zeros(4), torch.zeros((1, 2, 128), device=DEV)
    entries(ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value)
    L.locks_pack_pages(d, cache, cache, one, None, 1, packed)
    L.locks_unpack_pages(d, packed, one, None, 1, cache, cache)
    L.locks_packed_attention(d, q, packed, table, one, q.bfloat16(), ws)
    L.locks_copy_pages(L.make_planes([cache]), one, one)
    L.locks_fork_sequences(d, table, one, one, four, table, one, four, one, one, one, ws)
    L.locks_take_pages(d, table, one, one, four, one, four, ws)
    L.locks_free_pages(four, table, one, four)
    L.locks_compact_pages(d, table, one, four, table, four, four, four, one, four, ws)


def test_calls_go_to_the_stream_they_are_given():
    """A call on another stream than the current one does not wait for the current one's work, and its own
    order is kept: the counts pass from call to call."""
    d, cache, packed, ws = arguments()
    side = torch.cuda.Stream()
    table, tokens, refs, n = zeros(1, 4), zeros(1), zeros(4), zeros(1)
    want = torch.tensor([40], dtype=torch.int32, device=DEV)
    three = torch.tensor([3], dtype=torch.int32, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    L.locks_take_pages(d, table, tokens, want, refs, tokens, refs, ws, n_free=n, stream=side)
    L.locks_free_pages(refs, table, three, refs, stream=side)
    with torch.cuda.stream(side):                     # the current one, by default
        L.locks_take_pages(d, table, torch.zeros_like(tokens), want, refs, tokens, refs, ws, n_free=n)
    side.synchronize()
    assert table.tolist() == [[0, 1, 2, 0]] and tokens.tolist() == [40] and refs.tolist() == [1, 1, 1, 0] and n.tolist() == [1]
    assert L.locks_get_device_status(ws) == 0


def test_two_graphs_with_a_workspace_each_replayed_at_once():
    """Captured page calls and attention hold no state but their arguments: two graphs of the same calls on
    tensors of their own, replayed on two streams in turn, give what one after the other gives."""
    def program(seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        pool, batch, hkv = 50, 3, 2
        d, s = L.make_dims(batch, 8, hkv, 8, pool), torch.cuda.Stream()
        t = dict(table=zeros(batch, 8), tokens=zeros(batch), refs=zeros(pool), n=zeros(1), ws=L.alloc_pool_workspace(d, DEV),
                 aws=L.alloc_packed_workspace(d, DEV), out=torch.zeros((batch, 8, 128), dtype=torch.bfloat16, device=DEV),
                 want=torch.tensor([16 * seed, 100, 128], dtype=torch.int32, device=DEV), pages=zeros(batch),
                 q=torch.randn((batch, 8, 128), generator=g, device=DEV))
        k, v = (torch.randn((pool, hkv, 16, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
        packed = t["packed"] = torch.zeros((pool, hkv, L.LOCKS_PACKED_BYTES), dtype=torch.uint8, device=DEV)
        L.locks_pack_pages(d, k, v, torch.arange(pool, dtype=torch.int32, device=DEV), None, pool, packed)

        def step():
            L.locks_take_pages(d, t["table"], t["tokens"], t["want"], t["refs"], t["tokens"], t["refs"], t["ws"], n_free=t["n"])
            t["pages"].copy_(t["tokens"] // 16)
            L.locks_packed_attention(d, t["q"], packed, t["table"], t["pages"], t["out"], t["aws"])
            L.locks_free_pages(t["refs"], t["table"], (t["tokens"] + 15) // 16, t["refs"])
            t["tokens"].zero_()

        step()
        torch.cuda.synchronize()
        want = [t[x].clone() for x in ("table", "tokens", "refs", "n", "out")]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        return t, want, graph, s

    runs = [program(1), program(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, _, graph, s in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for t, want, _, _ in runs:
        assert all(torch.equal(t[x], y) for x, y in zip(("table", "tokens", "refs", "n", "out"), want))
        assert L.locks_get_device_status(t["ws"]) == 0 and L.locks_get_device_status(t["aws"]) == 0
