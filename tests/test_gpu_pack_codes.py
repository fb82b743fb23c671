"""GPU tests of packing's codes where a quotient or a neighbour may go wrong: groups that are not
finite beside groups that are, every mantissa of a scale, and the rounding of unpacked values."""

import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

UNIT = L.LOCKS_PACKED_BYTES


def pack(k, v):
    """Units of all pages of k and v (float64 arrays of bf16 values [pages][16][128])."""
    k, v = (torch.from_numpy(x).to(DEV).bfloat16()[:, None].contiguous() for x in (k, v))
    n = k.shape[0]
    packed = torch.full((n, 1, UNIT), 0xA5, dtype=torch.uint8, device=DEV)
    L.locks_pack_pages(L.make_dims(1, 1, 1, 1, n), k, v, torch.arange(n, dtype=torch.int32, device=DEV), None, n, packed)
    return packed


def unpack(packed):
    n = packed.shape[0]
    k, v = (torch.zeros((n, 1, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    L.locks_unpack_pages(L.make_dims(1, 1, 1, 1, n), packed, torch.arange(n, dtype=torch.int32, device=DEV), None, n, k, v)
    return [x[:, 0].double().cpu().numpy() for x in (k, v)]


BAD = {"nan": ([0], [np.nan]), "inf": ([3], [np.inf]), "minus_inf": ([7], [-np.inf]),
       "both_infs": ([1, 2], [np.inf, -np.inf]), "range": ([4, 9], [3e38, -3e38]), "all": (range(32), [np.nan] * 32)}


@pytest.mark.parametrize("kind", list(BAD))
def test_groups_that_are_not_finite_leave_the_others_alone(kind):
    """Page 16 g + t has one bad group, g of token t; the last ones have several."""
    g = torch.Generator()
    g.manual_seed(7)
    n = 16 * 4 + 6
    k, v = (torch.randn((n, 16, 128), generator=g).bfloat16().double().numpy() for _ in range(2))
    bad = [np.zeros((n, 16, groups), bool) for groups in (4, 2)]
    for page in range(64):
        for b, groups in zip(bad, (4, 2)):
            b[page, page % 16, page // 16 % groups] = True
    rng = np.random.default_rng(3)
    for b in bad:
        b[64:] = rng.random(b[64:].shape) < 0.3
    at, values = BAD[kind]
    clean = []
    for x, b in zip((k, v), bad):
        size = 128 // b.shape[-1]
        clean.append(np.where(np.repeat(b, size, -1), 0.0, x))
        for page, token, group in zip(*np.nonzero(b)):
            x[page, token, [size * group + d for d in at]] = values
    packed = pack(k, v)
    units = packed[:, 0].cpu().numpy()
    for x, b, got, out in zip(clean, bad, ref.fields(units), unpack(packed)):
        size = 128 // b.shape[-1]
        good = ~np.repeat(b, size, -1)
        for a, w in zip(got, ref.codes_of(x, size)):
            assert np.array_equal(a[good], w[good])
        assert np.isfinite(out[good]).all() and not np.isfinite(out[~good]).any()


@pytest.mark.parametrize("exponent", [-85, -20, 0, 31, 100])
def test_codes_of_every_scale(exponent):
    """For each of the 128 mantissas a scale can have: all bf16 values of a group of that scale, of which
    many have quotients on a border between two codes, or next to one."""
    tokens = []
    for m in range(128):
        scale = Fraction(128 + m, 128)
        # the greatest value is 15 scales (12 bits) cut to 8, the least what is missing: the range is 15 scales
        whole = 15 * scale
        high = Fraction(int(whole * 8), 8)
        low = high - whole
        values = np.arange(0x3e80, 0x4200, dtype=np.uint16)         # 0.25 .. 32
        x = ref.f32_of(values).astype(np.float64)
        x = x[x < float(high)]
        x = np.concatenate([x, -x[x < float(-low)]])
        for i in range(0, len(x), 30):
            row = np.full(32, float(high))
            row[1] = float(low)
            row[2:2 + len(x[i:i + 30])] = x[i:i + 30]
            tokens.append(row)
    tokens = np.array(tokens)
    assert np.array_equal(ref.cache_ref.bf16(tokens), tokens)
    n = -(-len(tokens) // 32)
    k = np.resize(tokens, (n * 64, 32)).reshape(n, 16, 128) * 2.0 ** exponent
    v = np.resize(tokens.repeat(2, 0), (n * 32, 64)).reshape(n, 16, 128) * 2.0 ** exponent
    units = pack(k, v)[:, 0].cpu().numpy()
    for x, size, (code, scale, zero) in zip((k, v), (32, 64), ref.fields(units)):
        c, s, z = ref.codes_of(x, size)
        assert len(np.unique(s)) == 128
        assert np.array_equal(s, scale) and np.array_equal(z, zero)
        wrong = c != code
        assert not wrong.any(), (int(wrong.sum()), x[wrong][:4], s[wrong][:4], z[wrong][:4], code[wrong][:4], c[wrong][:4])


def bf16_of(x: Fraction) -> float:
    """The bf16 value nearest to x (a number of its range), ties to the even one."""
    if x == 0:
        return 0.0
    size = abs(x)
    e = size.numerator.bit_length() - size.denominator.bit_length()
    e -= size < Fraction(2) ** e
    step = Fraction(2) ** (max(e, -126) - 7)
    return float(round(x / step) * step)             # round() takes ties to even


def test_unpacked_values_are_rounded_once():
    """Products on a tie between two bf16 values, and zeros on either side that are too small for fp32 to
    see beside them."""
    scales = [Fraction(128 + m, 128) for m in (0, 1, 2, 5, 33, 64, 85, 101, 127)]
    zeros = [sign * Fraction(128 + m, 128) * Fraction(2) ** e for sign in (1, -1) for m in (0, 77)
             for e in (-40, -30, -24, -17, -16, -15, -13, -12, -11, -9, -8, -3, 0, 7, 14, 15, 16, 17, 20, 30)] + [Fraction(0)]
    pairs = list(itertools.product(scales, zeros))
    n = -(-len(pairs) // 32)
    code = np.arange(128) % 16
    units = np.zeros((n, UNIT), np.uint8)
    want = np.zeros((2, n, 16, 128))
    groups = []
    for i in range(n * 16):                          # token i of all: pair 2i of its dims 0..63, pair 2i + 1 of the others
        groups.append([pairs[(2 * i + j) % len(pairs)] for j in range(2)])
    for values in (0, 1):
        byte, bit = ref.PLACES[values]
        for t in range(16):
            for d in range(128):
                units[:, byte[t, d]] |= np.uint8(int(code[d]) << int(bit[t, d]))
        per = (4, 2)[values]
        fields = np.zeros((n, 16, 2, per), np.float32)
        for i, pair in enumerate(groups):
            for g in range(per):
                fields[i // 16, i % 16, :, g] = [float(x) for x in pair[g * 2 // per]]
            for d in range(128):
                s, z = pair[d // 64]
                want[values, i // 16, i % 16, d] = bf16_of(z + s * int(code[d]))
        bits = (fields.view(np.uint32) >> 16).astype(np.uint16)
        at = (2048, 2304)[values]
        units[:, at:at + 64 * per] = bits.reshape(n, -1).view(np.uint8)
    got = unpack(torch.from_numpy(units).to(DEV)[:, None].contiguous())
    for x, w in zip(got, want):
        wrong = x != w
        assert not wrong.any(), (int(wrong.sum()), x[wrong][:6], w[wrong][:6])
