"""The paged-cache operators written out in float64, from their formulas in
include/locks_cache.h. Loops over sequences and heads; nothing here is shared with the
library."""

from __future__ import annotations

import numpy as np


def bf16(x):
    """float -> nearest bf16 value (ties to even), as float64."""
    import synth
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(x, np.float32))).astype(np.float64)


def norm(x, w, eps):
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rotate(x, angle, interleaved, scale):
    """x [..., 128], angle [pairs]."""
    n = angle.shape[-1]
    i = np.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    out = x.copy()
    c, s = np.cos(angle) * scale, np.sin(angle) * scale
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ib] * c + x[..., ia] * s
    return out


def pair_size(x, n, interleaved):
    """|a| + |b| of each element's pair (|x| itself past the rotated ones)."""
    i = np.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    out = np.abs(x)
    both = out[..., ia] + out[..., ib]
    out[..., ia] = both
    out[..., ib] = both
    return out


def attend(q, keys, values):
    """q [rows, 128], keys / values [tokens, 128] -> out, lse, sum p |v|, max_t sum |q k| / sqrt(128)."""
    rows = q.shape[0]
    if keys.shape[0] == 0:
        z = np.zeros((rows, 128))
        return z, np.full(rows, -np.inf), z, np.zeros(rows)
    s = q @ keys.T / np.sqrt(128.0)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    size = (np.abs(q) @ np.abs(keys).T).max(1) / np.sqrt(128.0)
    return p @ values / l, (m + np.log(l))[:, 0], p @ np.abs(values) / l, size


def mass(scores, seq_pages, old, decay):
    new = {}
    for b, n in enumerate(seq_pages):
        s = scores[b, :, :n].astype(np.float64)
        s = np.where(np.isnan(s) | np.isposinf(s), -np.inf, s)
        share = np.zeros((s.shape[0], n))
        for h in range(s.shape[0]):
            if n and np.any(s[h] > -np.inf):
                e = np.exp(s[h] - s[h].max())
                share[h] = e / e.sum()
        kept = old[b, :n].astype(np.float64) * decay if decay != 0 else 0.0
        new[b] = kept + share.mean(0)
    return new


def evict(mass_row, table_row, n, keep, sink, recent, extra):
    """One sequence: kept table, kept mass, evicted physical pages."""
    free = [j for j in range(sink, n - recent)]

    def key(j):
        m = float(mass_row[j])
        return (0, 0.0, j) if np.isnan(m) else (1, m + 0.0, j)

    gone = sorted(sorted(free, key=key)[:max(0, n - keep)])
    out = set(gone)
    rest = [j for j in range(min(n + extra, len(mass_row))) if j not in out]
    return table_row[rest], mass_row[rest], table_row[gone]
