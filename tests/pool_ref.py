"""The packed cache and the page pool written out from their definitions in
include/locks_pool.h: codes and values in float64, the page calls as loops over sequences.
Nothing here is shared with the library."""

from __future__ import annotations

import numpy as np

from tests import cache_ref

PAGE, D, UNIT = 16, 128, 2432


def f32_of(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def place(t, d, values):
    """Byte (within the unit) and lowest bit of a code."""
    w = d // 16
    if values:
        lane, bit = 4 * (d % 8) + t % 8 // 2, 16 * (t % 2) + 4 * (d // 8 % 2) + 8 * (t // 8)
    else:
        lane, bit = 4 * (t % 8) + d % 8 // 2, 16 * (d % 2) + 4 * (d // 8 % 2) + 8 * (t // 8)
    return 1024 * values + 512 * (w // 4) + 16 * lane + 4 * (w % 4) + bit // 8, bit % 8


T_, D_ = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
PLACES = [place(T_, D_, 0), place(T_, D_, 1)]


def fields(units):
    """uint8 [..., 2432] -> (codes, scales, zeros) of keys and of values, per element [..., 16, 128]."""
    out = []
    for values, at, groups in ((0, 2048, 4), (1, 2304, 2)):
        byte, bit = PLACES[values]
        code = (units[..., byte] >> bit) & 15
        sz = np.ascontiguousarray(units[..., at:at + 64 * groups]).view(np.uint16)
        sz = f32_of(sz).astype(np.float64).reshape(units.shape[:-1] + (PAGE, 2, groups))
        scale, zero = (np.repeat(sz[..., i, :], D // groups, axis=-1) for i in (0, 1))
        out.append((code, scale, zero))
    return out


def unpack(units):
    """Keys and values as the units stand for them, float64."""
    return tuple(zero + scale * code for code, scale, zero in fields(units))


def sizes(units):
    """|zero| + |scale code| of keys and values: what the errors of sums are counted from."""
    return tuple(np.abs(zero) + np.abs(scale * code) for code, scale, zero in fields(units))


def codes_of(x, group):
    """x float64 (bf16 values) [..., 128] -> codes, scales, zeros per element."""
    g = x.reshape(x.shape[:-1] + (D // group, group))
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    scale = cache_ref.bf16((hi - lo) / 15)
    scale = np.where(scale < 2.0 ** -126, 0.0, scale)
    code = np.rint(np.divide(g - lo, scale, out=np.zeros_like(g), where=scale > 0))
    wide = (lambda y: np.broadcast_to(y, g.shape).reshape(x.shape))
    return wide(code).astype(np.int64), wide(scale), wide(lo)


def attend(q, k, v, ks, vs):
    """q [rows, 128], keys and values [tokens, 128], their sizes -> out, lse, sum p |v|, max |q||k|."""
    rows = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros((rows, D)), np.full(rows, -np.inf), np.zeros((rows, D)), np.zeros(rows)
    s = q @ k.T / np.sqrt(128.0)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    return p @ v / l, (m + np.log(l))[:, 0], p @ vs / l, (np.abs(q) @ ks.T).max(1) / np.sqrt(128.0)


# ------------------------------------------------------------- page calls

def pages_of(tokens):
    return -(-int(tokens) // PAGE)


def fork(table, tokens, parents, refs, table_out, tokens_out):
    """Returns refs_out, copy_src, copy_dst and whether pages ran out; fills the outs in place."""
    refs = refs.astype(np.int64)
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    new = refs.copy()
    for b, n in enumerate(tokens):
        for j in range(pages_of(n)):
            new[table[b, j]] -= 1
    keeper = {}
    for b, p in enumerate(parents):
        if p >= 0 and (p not in keeper or p == b):
            keeper[p] = b
    src, dst, short = [], [], False
    for b, p in enumerate(parents):
        if p < 0:
            tokens_out[b] = 0
            continue
        n = int(tokens[p])
        row = [int(x) for x in table[p, :n // PAGE]]
        kept = n
        if n % PAGE:
            last = int(table[p, n // PAGE])
            if keeper[p] == b:
                row.append(last)
            elif free:
                row.append(free.pop(0))
                new[row[-1]] = 0                     # whatever it was: its count is 1 then
                src.append(last)
                dst.append(row[-1])
            else:
                short, kept = True, n // PAGE * PAGE
        for j, page in enumerate(row):
            table_out[b, j] = page
            new[page] += 1
        tokens_out[b] = kept
    return new, src, dst, short


def take(table, tokens, now, refs):
    """Fills the table in place; returns tokens_out, refs_out, pages left and whether they ran out."""
    refs, out = refs.copy(), tokens.copy()
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    short = False
    for b in range(len(tokens)):
        have, want = pages_of(tokens[b]), pages_of(now[b])
        if want > have:
            if short or want - have > len(free):
                short = True
                continue
            for j in range(have, want):
                table[b, j] = free.pop(0)
                refs[table[b, j]] = 1
        out[b] = now[b]
    return out, refs, len(free), short


def compact(table, tokens, refs, table_out):
    used = [p for p in range(len(refs)) if refs[p] > 0]
    src = [p for p in used if p >= len(used)]
    dst = [p for p in range(len(used)) if refs[p] <= 0]
    new = np.arange(len(refs), dtype=np.int64)
    new[src] = dst
    after = refs.copy()
    after[dst] = refs[src]
    after[len(used):] = 0
    for b, n in enumerate(tokens):
        for j in range(pages_of(n)):
            table_out[b, j] = new[table[b, j]]
    return after, src, dst, new
