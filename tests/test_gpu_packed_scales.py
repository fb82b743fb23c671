"""GPU tests of attention over packed pages whose values' scales are far apart: a token's output is as
exact as its own scale allows, whatever scales lie beside it. The bounds are those of
tests/test_gpu_packed.py: a weight times a scale is off by 2^-11 of itself (half a step of fp16), or by
2^-21 of the scale times the largest weight. (The latter needs no term of its own: a warp's share has up to
2^11 tokens here, so it is below 2^-10 of the output's sizes, and the scores' part, 2 e, is 2^-9 and more.)"""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import bf16_out
from tests.test_gpu_packed import DEV, f64, make_case, run, tokens_of

pytestmark = pytest.mark.gpu

LAYOUTS = [(8, 2), (16, 2), (32, 2)]                 # 4, 8 and 16 queries a kv head


def check(c):
    run(c)
    assert L.locks_get_device_status(c["ws"]) == 0
    got, lse, q = bf16_out(c["out"].view(torch.int16)), f64(c["lse"]), f64(c["q"])
    units, table, g = c["packed"].cpu().numpy(), c["table"].cpu().numpy(), c["hq"] // c["hkv"]
    for b in range(c["B"]):
        for h in range(c["hkv"]):
            rows = slice(h * g, h * g + g)
            parts = tokens_of(c, b, h, units, table)
            want, want_lse, weight, size = ref.attend(q[b, rows], *parts)
            n = len(parts[0]) / 16 + 2
            e = 2.0 ** -15 * size
            tol = weight * (2 * e + 2.0 ** -11 + 2.0 ** -19 + n * 2.0 ** -23)[:, None] + 2.0 ** -8 * np.abs(want)
            off = np.abs(got[b, rows] - want)
            assert (off <= tol + 1e-30).all(), (b, h, (off / (tol + 1e-30)).max(), np.argwhere(off > tol + 1e-30)[:4])
            assert (np.abs(lse[b, rows] - want_lse) <= e + 2.0 ** -22 * np.abs(want_lse) + 2.0 ** -18 + n * 2.0 ** -23
                    ).all(), (b, h)


def value_fields(c):
    """Scales and zeros of the values, [pages][heads][16 tokens][2][2 groups], as a copy; put(x) stores one."""
    phys, hkv = c["packed"].shape[:2]
    x = c["packed"][..., 2304:].contiguous().view(torch.bfloat16).view(phys, hkv, 16, 2, 2).clone()

    def put(x):
        c["packed"][..., 2304:] = x.bfloat16().reshape(phys, hkv, -1).contiguous().view(torch.uint8)
    return x.float(), put


def key_fields(c):
    phys, hkv = c["packed"].shape[:2]
    x = c["packed"][..., 2048:2304].contiguous().view(torch.bfloat16).view(phys, hkv, 16, 2, 4).clone()

    def put(x):
        c["packed"][..., 2048:2304] = x.bfloat16().reshape(phys, hkv, -1).contiguous().view(torch.uint8)
    return x.float(), put


@pytest.mark.parametrize("hq,hkv", LAYOUTS)
@pytest.mark.parametrize("small", [2.0 ** -14, 2.0 ** -24, 2.0 ** -30, 2.0 ** -45])
@pytest.mark.parametrize("pages,recent", [(30, 0), (2500, 19)])
def test_a_group_far_smaller_than_the_other(hq, hkv, small, pages, recent):
    c = make_case([pages, 3], [recent, 0], hq, hkv, seed=31)
    x, put = value_fields(c)
    x[..., 1] *= small                               # scales and zeros of dims 64..127
    put(x)
    c["v"][..., 64:] = (c["v"][..., 64:].float() * small).bfloat16()
    check(c)


@pytest.mark.parametrize("hq,hkv", LAYOUTS)
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 17, 29])
def test_a_large_token_of_no_weight(hq, hkv, q_type, at):
    """One token's scale is 2^40 times the others', its softmax weight about 2^-60."""
    c = make_case([30], [5], hq, hkv, seed=32, q_type=q_type)
    c["q"][..., :32] = c["q"][..., :32].abs() + 1    # their sum is at least 32
    page = int(c["table"][0, at])
    x, put = key_fields(c)
    x[page, :, 3, :, :] = 0
    x[page, :, 3, 1, 0] = -12.0                      # a key of -12 in dims 0..31: scores below -33
    put(x)
    x, put = value_fields(c)
    x[page, :, 3] *= 2.0 ** 40
    put(x)
    parts = tokens_of(c, 0, 0, c["packed"].cpu().numpy(), c["table"].cpu().numpy())
    score = f64(c["q"])[0, 0] @ parts[0].T / np.sqrt(128.0)
    assert score[16 * at + 3] < score.max() - 33
    check(c)


@pytest.mark.parametrize("hq,hkv", LAYOUTS)
@pytest.mark.parametrize("growing", [False, True])
def test_scales_that_go_over_many_orders(hq, hkv, growing):
    """From 2^40 to 2^-40 along the row, or the other way, while scores grow so that the last pages count."""
    n = 900
    c = make_case([n], [0], hq, hkv, seed=33, steep=2.0)
    ramp = torch.zeros(c["packed"].shape[0], device=DEV)
    ramp[c["table"][0].long()] = torch.linspace(0, 3, n, device=DEV)
    x, put = key_fields(c)
    put(x * ramp[:, None, None, None, None])
    down = torch.zeros(c["packed"].shape[0], device=DEV)
    down[c["table"][0].long()] = torch.linspace(-40, 40, n, device=DEV) * (1 if growing else -1)
    x, put = value_fields(c)
    put(x * 2.0 ** down[:, None, None, None, None])
    check(c)


@pytest.mark.parametrize("hq,hkv", LAYOUTS)
@pytest.mark.parametrize("pages", [20, 2500])
def test_scales_below_zero(hq, hkv, pages):
    """The unit's definition takes any scale: a group counted down from its greatest value."""
    c = make_case([pages], [7], hq, hkv, seed=34)
    for fields in (key_fields, value_fields):
        x, put = fields(c)
        scale, zero = x[..., 0, :].clone(), x[..., 1, :].clone()
        x[..., 0, :], x[..., 1, :] = -scale, zero + 15 * scale
        if fields is value_fields:
            x[:, :, ::3] *= 2.0 ** 12                # past fp16 with the sum's slack
        put(x)
    check(c)


@pytest.mark.parametrize("hq,hkv,pages", [(4, 1, 30000), (8, 1, 30000), (16, 1, 30000), (16, 1, 4000)])
def test_long_rows_of_small_groups(hq, hkv, pages):
    """A group's scales and zeros times 2^-30 are its output times 2^-30, also where a long row's output is far
    smaller than its values. (Both outputs are off by 2^-8 of themselves for their rounding, by 2^-10 at most
    for everything ahead of it.)"""
    c = make_case([pages], [0], hq, hkv, seed=35, steep=0.2)
    run(c)
    first = f64(c["out"])
    x, put = value_fields(c)
    x[..., 1] *= 2.0 ** -30
    put(x)
    run(c)
    second = f64(c["out"])
    for dims, size in ((slice(0, 64), 1.0), (slice(64, 128), 2.0 ** 30)):
        a, b = first[..., dims], size * second[..., dims]
        assert np.linalg.norm(a - b) <= (2.0 ** -7 + 2.0 ** -9) * np.linalg.norm(a)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** -30])
def test_scales_below_zero_behind_flat_groups(hq, hkv, size):
    """Four pages of five have scales 0, so that warps meet one below 0 before any above."""
    n = 9000
    c = make_case([n], [0], hq, hkv, seed=36)
    x, put = value_fields(c)
    x *= size
    x[..., 1, :] += 15 * x[..., 0, :]
    x[..., 0, :] *= -1
    flat = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    flat[c["table"][0].long()[4::5]] = False
    x[flat, :, :, 0] = 0
    put(x)
    check(c)
