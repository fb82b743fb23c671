"""What the shared-prefix attention's softmax weights keep of their 24 bits, in every form of it.

Tolerance: scores are off by at most e = 2^-15 max_t sum |q k| / sqrt(128), a weight by 2 e
(test_gpu_cache). A weight meets the values as a bf16 high and low part: the high part leaves
at most 2^-8 of it, of which the low part's rounding leaves 2^-8: 2^-16. Every token that is
added to a sum may cost a last bit of it, 2^-23. 2^-20 covers exp2. All of that is relative
to sum p |v|; then the output's own rounding, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from tests import test_gpu_cache as T
from tests.test_gpu_cache_prefix_forms import scratch_untouched, wide

pytestmark = pytest.mark.gpu


def check(c):
    T.run_prefix(c)
    out, lse, w, size = T.prefix_ref(c)
    tokens = max(c["own"]) + max([n for _, n in c["groups"]] + [0])
    tol = (2 * 2.0 ** -15 * size[..., None] + 2.0 ** -16 + 2.0 ** -20 + tokens * 2.0 ** -23) * w + T.UB * np.abs(out)
    far = np.abs(T.f64(c["out"]) - out) > tol
    assert not far.any(), (int(far.sum()), far.size, np.abs(T.f64(c["out"]) - out).max())


CASES = {  # groups, own tokens, hq, hkv, tables made wide
    "clusters": ([(2, 333)], [45, 4], 32, 8, ()),
    "clusters of eight warps": ([(1, 4000)], [45], 32, 8, ()),
    "clusters, sixteen queries": ([(2, 700)], [46, 3], 32, 2, ()),
    "lists": ([(10, 100), (20, 64)], [i * 7 for i in range(40)], 32, 8, ()),
    "lists, sixteen queries": ([(40, 100)], [i * 8 for i in range(48)], 32, 2, ()),
    "tiles, own by pages": ([(30, 3000), (4, 64)], [i * 6 for i in range(38)], 32, 8, ("prefix_table",)),
    "tiles": ([(30, 1000), (4, 64)], [i * 26 for i in range(38)], 32, 8, ("prefix_table", "page_table")),
    "tiles, sixteen queries": ([(3, 1000), (2, 130)], [i * 51 for i in range(7)], 32, 2, ("prefix_table", "page_table")),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_weights_close_to_each_other(name, q_type):
    """Tokens of values +1 and -1 whose weights differ by less than a bf16 step: the output is the
    difference of the weights."""
    groups, own, hq, hkv, tables = CASES[name]
    c = T.prefix_case(groups, own, hq, hkv, seed=3, q_type=q_type)
    c["q"].zero_()
    c["q"][:, :, 0] = 2.0 ** -9 * 128 ** 0.5 * (1 + torch.arange(hq, device=T.DEV) % 5)
    c["k"].zero_()
    c["k"][:, :, ::2, 0] = 1.0                    # every other token
    c["v"][:, :, ::2], c["v"][:, :, 1::2] = 1.0, -1.0
    c = wide(c, tables) if tables else c
    check(c)
    assert scratch_untouched(c) == (not tables)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_weights_of_any_size(name, q_type):
    groups, own, hq, hkv, tables = CASES[name]
    for scale in (0.05, 0.6):
        c = T.prefix_case(groups, own, hq, hkv, seed=4, q_type=q_type, scale=scale)
        check(wide(c, tables) if tables else c)
