"""The tiled shared-prefix attention where its pieces are short: a piece of one or two tiles is
weighed while the softmax groups still join the sums of the one before, so each piece's
maxima have to outlive the next one's. Tolerances are test_gpu_cache's; repeated calls
have to agree to the bit."""
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
