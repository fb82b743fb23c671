"""Workspace sizes of the cache operators at the largest tables (host)."""
import pytest


@pytest.fixture(scope="module")
def L():
    from sparse_kv_page_gb300 import build as b
    b.build()
    import sparse_kv_page_gb300 as L
    return L


@pytest.mark.parametrize("pages", [0, 1, 8191, 8192, 8193, 1 << 20, (1 << 31) - 8192, (1 << 31) - 8191, (1 << 31) - 1])
@pytest.mark.parametrize("batch,hq", [(1, 1), (3, 32)])
def test_mass_workspace_holds_a_pair_per_head_and_slice(L, pages, batch, hq):
    """256 bytes and a pair of fp32 per (sequence, query head, 8192 pages), for any int32 of pages."""
    slices = -(-pages // 8192)
    assert L.locks_mass_workspace_size(L.make_dims(batch, hq, 2 if hq > 16 else 1, pages, 64)) == 256 + batch * hq * slices * 8
