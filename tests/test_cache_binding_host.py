"""Shapes that the cache operators' binding refuses or takes, on host tensors: those are refused in
the end, but only after everything else has been looked at."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from sparse_kv_page_gb300 import build as b
    b.build()
    import sparse_kv_page_gb300 as L
    L.cache.load_library()
    return L


def append(L, positions, axes):
    d = L.make_dims(6, 4, 2, 8, 16)
    kv = torch.zeros(6, 2, 128)
    cache = torch.zeros(16, 2, 16, 128, dtype=torch.bfloat16)
    rope = L.make_rope(32, [0.5] * 16, num_axes=axes)
    L.locks_append_tokens(d, rope, None, kv, kv, positions, torch.zeros(6, dtype=torch.int32),
                          torch.zeros(6, 8, dtype=torch.int32), None, cache, cache)


@pytest.mark.parametrize("shape,axes", [((6, 3), 3), ((18,), 3), ((1, 18), 3), ((3, 3, 2), 3), ((6, 1), 1), ((1, 1, 6), 1),
                                        ((2, 6), 3), ((2, 6), 1), ((5,), 1), ((), 1)])
def test_positions_of_another_layout_are_refused(L, shape, axes):
    """As many elements or not: rows are axes, columns tokens."""
    with pytest.raises(ValueError, match="positions is not"):
        append(L, torch.zeros(shape, dtype=torch.int32), axes)


@pytest.mark.parametrize("shape,axes", [((3, 6), 3), ((1, 6), 1), ((6,), 1)])
def test_positions_by_axis_are_taken(L, shape, axes):
    with pytest.raises(ValueError, match="CUDA"):
        append(L, torch.zeros(shape, dtype=torch.int32), axes)
    with pytest.raises(TypeError, match="positions has type"):
        append(L, torch.zeros(shape, dtype=torch.int64), axes)
    with pytest.raises(ValueError, match="contiguous"):
        append(L, torch.zeros(shape + (2,), dtype=torch.int32)[..., 0], axes)
