"""The tiled shared-prefix attention where its pieces are short: a piece of one or two tiles is
weighed while the softmax groups still join the sums of the one before, so each piece's
maxima have to outlive the next one's. Tolerances are test_gpu_cache's; repeated calls
have to agree to the bit."""
import numpy as np
import pytest
import torch

from tests import test_gpu_cache as T
from tests.test_gpu_cache_prefix_forms import scratch_untouched, wide

pytestmark = pytest.mark.gpu


CASES = [
    # groups, own tokens, hq, hkv
    ([], [(i * 37) % 257 for i in range(150)], 32, 2),           # sixteen queries a kv head: 1 and 2 tiles
    ([], [1 + i % 128 for i in range(300)], 16, 1),              # one tile each
    ([(1, 129)] * 120, [(i * 5) % 128 for i in range(130)], 8, 1),          # groups of one sequence
    ([(40, 120)] * 12, [0] * 480, 32, 8),                        # wide pieces of one tile
    ([(40, 250), (1, 64), (33, 128)] * 5, [(i * 3) % 200 for i in range(370)], 16, 2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_short_pieces(case, q_type):
    groups, own, hq, hkv = CASES[case]
    c = wide(T.prefix_case(groups, own, hq, hkv, seed=160 + case, q_type=q_type, scale=2.0))
    T.check_prefix(c)
    assert not scratch_untouched(c)
    first, first_lse = c["out"].clone(), c["lse"].clone()
    for _ in range(40):
        c["out"].fill_(float("nan"))
        T.run_prefix(c)
        assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])


@pytest.fixture
def wait_limit():
    yield T.L.locks_set_wait_limit_ns
    T.L.locks_set_wait_limit_ns(0)


TIMEOUT = -5


@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_giving_up_leaves_nothing_in_flight(q_type, wait_limit):
    """With a limit that waits for loads run past, a call either ends as ever or records that it gave
    up. In both cases nothing of it may land in the shared memory of the calls behind it."""
    c = wide(T.prefix_case([(40, 3000), (3, 20000)], [(i * 131) % 1500 for i in range(50)], 32, 8, seed=170, q_type=q_type))
    d = T.prefix_case([(2, 333)], [45, 3], 32, 8, seed=171, q_type=q_type)
    T.check_prefix(c)
    T.check_prefix(d)
    want = [x[n].clone() for x in (c, d) for n in ("out", "lse")]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=T.DEV)
    for limit in (1, 1, 500, 2000, 5000):
        for behind in (c, d):                     # other kernels, and the same
            c["ws"][:256] = 0
            d["out"].fill_(float("nan"))
            flush.fill_(1)                        # the loads come from memory
            wait_limit(limit)
            T.run_prefix(c)
            wait_limit(0)
            status = T.L.locks_get_device_status(c["ws"])
            assert status in (0, TIMEOUT)
            if status == 0:
                assert torch.equal(c["out"], want[0]) and torch.equal(c["lse"], want[1])
            wait_limit(limit)
            T.run_prefix(c)
            wait_limit(0)
            T.run_prefix(behind)
            i = 0 if behind is c else 2
            assert torch.equal(behind["out"], want[i]) and torch.equal(behind["lse"], want[i + 1])
    c["ws"][:256] = 0
    T.check_prefix(c)


@pytest.mark.parametrize("own", [False, True])
def test_longest_lists(own):
    """2^31 - 16 tokens, seven pages over and over: the attention over those seven, whose sum is as
    many times as large. Each CTA adds up to 2^24 / 152 tiles, eight products and two sums a
    tile: that many last bits (2^-23) of sums of p |v| and of p."""
    pages = (1 << 27) - 1                         # 7 * 19173961
    tokens = 16 * pages
    g = T.gen(5)
    k = torch.randn((7, 1, 16, 128), generator=g, device=T.DEV).bfloat16()
    v = torch.randn((7, 1, 16, 128), generator=g, device=T.DEV).bfloat16()
    q = torch.randn((1, 2, 128), generator=g, device=T.DEV)
    table = (torch.arange(pages, dtype=torch.int32, device=T.DEV) % 7).view(1, pages)
    dims = T.L.make_dims(1, 2, 1, pages if own else 0, 7)
    count = torch.tensor([tokens], dtype=torch.int32, device=T.DEV)
    none = torch.zeros(1, dtype=torch.int32, device=T.DEV)
    out, lse = torch.empty((1, 2, 128), device=T.DEV).bfloat16(), torch.empty((1, 2), device=T.DEV)
    ws = T.L.alloc_prefix_workspace(dims, 1, T.DEV)
    if own:
        T.L.locks_prefix_attention(dims, q, k, v, None, None, None, table, count, out, ws, lse=lse)
    else:
        bounds = torch.tensor([0, 1], dtype=torch.int32, device=T.DEV)
        T.L.locks_prefix_attention(dims, q, k, v, table, count, bounds, None, none, out, ws, lse=lse)
    assert T.L.locks_get_device_status(ws) == 0
    want, want_lse, w, size = T.ref.attend(T.f64(q[0]), T.f64(k).reshape(-1, 128), T.f64(v).reshape(-1, 128))
    last_bits = 2.0 ** -23 * (2 ** 24 / 152 + 1)
    e = 2.0 ** -15 * size
    tol = (2 * e[:, None] + T.UB + 10 * last_bits) * w + T.UB * np.abs(want)
    assert np.all(np.abs(T.f64(out)[0] - want) <= tol)
    assert np.all(np.abs(T.f64(lse)[0] - np.log(pages // 7) - want_lse) <= e + 4 * last_bits)


def test_a_limit_that_every_load_passes_runs_out(wait_limit):
    """A nanosecond: some wait of ten calls finds its load on the way and gives up."""
    c = wide(T.prefix_case([(40, 3000), (3, 20000)], [7] * 50, 32, 8, seed=172))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=T.DEV)
    c["ws"][:256] = 0
    for _ in range(10):
        flush.fill_(1)
        wait_limit(1)
        T.run_prefix(c)
        wait_limit(0)
    assert T.L.locks_get_device_status(c["ws"]) == TIMEOUT
    c["ws"][:256] = 0
    T.check_prefix(c)
