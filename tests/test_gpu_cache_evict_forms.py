"""Eviction on a GB300 with every number of CTAs a sequence that a call may take."""
import pytest
import torch

from tests import test_gpu_cache as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,P", [(1, 1536), (1, 1537), (24, 2048), (25, 2048), (8, 2049), (9, 2049), (40, 4096),
                                 (40, 4097), (96, 1601), (97, 1601), (100, 5000), (3, 16384), (3, 16385), (5, 16385)])
def test_evict_every_form(B, P):
    keep = P * 3 // 4
    for i, ties in enumerate((0.3, 0.95)):
        mass, table = T.evict_case(B, P, seed=B + P + i, ties=ties)
        seq = torch.tensor([P - 3 - (7 * b) % (P // 2) for b in range(B)], dtype=torch.int32, device=T.DEV)
        T.check_evict(mass, table, seq, keep, 2, 5, 3)
        T.check_evict(mass, table, seq, keep, 0, 0, 0, in_place=True)


def test_evict_forms_agree():
    """A sequence's result does not depend on the batch it is in."""
    mass, table = T.evict_case(97, 2500, seed=4)
    seq = torch.full((97,), 2500, dtype=torch.int32, device=T.DEV)
    want = None
    for B in (1, 9, 40, 97):
        m, t, n = mass[:B].clone(), table[:B].clone(), seq[:B].clone()
        dims = T.L.make_dims(B, 1, 1, 2500, 1 << 20)
        ev = torch.full((B, 2500), -1, dtype=torch.int32, device=T.DEV)
        cnt = torch.empty(B, dtype=torch.int32, device=T.DEV)
        T.L.locks_evict_pages(dims, m, t, n, 1000, m, t, n, ev, cnt, sink_pages=1, recent_pages=4)
        got = [x[:1].clone() for x in (m, t, n, ev, cnt)]
        assert want is None or all(torch.equal(x, y) for x, y in zip(want, got))
        want = got
