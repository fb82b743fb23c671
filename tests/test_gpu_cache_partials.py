"""Page mass from the scorer's partials, whatever the buffer held before: locks_score_pages
writes the slots of the CTAs that a sequence's pages went to and leaves the rest of its row
alone. Tolerances are test_gpu_cache's."""
import pytest
import torch

from tests import test_gpu_cache as T

pytestmark = pytest.mark.gpu

L = T.L


def scored(B, hq, hkv, P, seq, fill, low=False, partials=None):
    """Random summaries, their scores, and partials written over `fill` pairs or the given buffer."""
    g = T.gen(hq + P + B)
    dims = L.make_dims(B, hq, hkv, P, B * P)
    summ = L.Summaries.empty(B * P, hkv, T.DEV)
    summ.coef.random_(-127, 128, generator=g)
    q = torch.randn((B, hq, 128), generator=g, device=T.DEV)
    if low:                                       # scores around -200
        summ.mu.random_(-127, -90, generator=g)
        summ.scales[..., 0] = torch.tensor(0.2, dtype=torch.float16).view(torch.int16)
        q = 1 + 0.05 * q
    else:
        summ.mu.random_(-127, 128, generator=g)
        summ.scales[..., 0] = torch.tensor(0.01, dtype=torch.float16).view(torch.int16)
    table = torch.randperm(B * P, generator=g, device=T.DEV).view(B, P).int()
    scores = torch.zeros((B, hq, P), device=T.DEV)
    size = L.locks.lse_partials_shape(dims)[0]
    partials = torch.tensor(fill, device=T.DEV).repeat(size // 2) if partials is None else partials[:size]
    L.locks_score_pages(dims, q, summ, table, seq, scores, lse_partials=partials)
    if low:
        assert float(scores[0, :, :int(seq[0])].max()) < -150
    return dims, scores, partials


FILLS = [(float("nan"), float("nan")), (3e38, 5.0), (0.0, 0.0), (float("inf"), 1.0), (-3.0, 7.0)]


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("B,hq,hkv,P", [(1, 32, 8, 1600),    # 200 items: 52 of 152 CTAs have none
                                        (1, 32, 2, 31), (3, 32, 8, 700), (5, 4, 1, 64), (7, 20, 4, 333),
                                        (64, 8, 8, 40)])
def test_partials_over_anything(B, hq, hkv, P, fill):
    seq = torch.tensor([P - (17 * b) % P for b in range(B)], dtype=torch.int32, device=T.DEV)
    if B > 2:
        seq[1] = 0
    old = torch.rand((B, P), generator=T.gen(P), device=T.DEV)
    for low in (False, True):
        dims, scores, partials = scored(B, hq, hkv, P, seq, fill, low)
        a = T.check_mass(scores, seq, old, 0.75, partials=partials, dims=dims)
        b = T.check_mass(scores, seq, old, 0.75, dims=dims)
        assert (a - b).abs().max() <= 1e-6


def test_partials_of_an_earlier_call_with_other_sizes():
    """One buffer for two calls: what the larger one left is no part of the smaller one's."""
    seq = torch.tensor([2000, 1500, 700], dtype=torch.int32, device=T.DEV)
    big = scored(3, 32, 8, 2000, seq, (0.0, 0.0))[2]
    seq = torch.tensor([300], dtype=torch.int32, device=T.DEV)
    small, scores, reused = scored(1, 32, 8, 300, seq, None, low=True, partials=big)
    T.check_mass(scores, seq, torch.zeros((1, 300), device=T.DEV), 1.0, partials=reused, dims=small)
