"""GPU tests of the paged-cache operators against their float64 forms (cache_ref).

Tolerances are counted from the arithmetic (a rounding is off by half a step, u = 2^-24
in fp32 and 2^-8 in bf16, relative to the value):

* append: 17 u times |a| + |b| of the rotated pair. Norm: 12 u (the sum of 128 squares in
  12 levels, halved by the root: 6; rsqrt 4; two products 2). Angle and sincospi: 3 u.
  Rotation: 2 u. Then the rounding of the output type.
* prefix attention: scores are off by at most e = 2^-15 max_t sum |q k| / sqrt(128): q as
  two bf16 parts keeps it to 2^-16 (half a bf16 step of half a bf16 step), the products'
  256 fp32 additions to 256 u = 2^-16. A weight is then off by 2 e relative (itself and
  the normaliser) and by 2^-8 for its own rounding; 2^-20 covers exp2 and the sums.
* mass: a share is off by 2 u |s - m| for its exponent, as much for the normaliser, plus
  16 u for exp2, the products and the sums over up to 16 heads.
"""

import numpy as np
import pytest
import torch

from tests import cache_ref as ref
import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV, bf16_out

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8


def f64(t):
    t = t.view(torch.bfloat16) if t.dtype == torch.int16 else t
    return t.double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ append

def append_case(tokens, seqs, hq, hkv, itype, seed, start=None, axes=1, far=0, max_index=200):
    g = gen(seed)
    pages = (max_index + 15) // 16
    phys = seqs * pages + 3
    table = torch.randperm(phys, generator=g, device=DEV)[:seqs * pages].view(seqs, pages).int().contiguous()
    rows = torch.randperm(seqs * max_index, generator=g, device=DEV)[:tokens]       # distinct cache rows
    qkv = torch.randn((tokens, hq + 2 * hkv, 128), generator=g, device=DEV).mul_(1.5).to(itype)
    return dict(dims=L.make_dims(seqs, hq, hkv, pages, phys), q=qkv[:, :hq], k=qkv[:, hq:hq + hkv],
                v=qkv[:, hq + hkv:], token_seq=(rows // max_index).int(), cache_index=(rows % max_index).int(),
                positions=torch.randint(0, 300, (axes, tokens), generator=g, device=DEV, dtype=torch.int32) + far,
                page_table=table, k_cache=torch.randn((phys, hkv, 16, 128), generator=g, device=DEV).bfloat16(),
                v_cache=torch.randn((phys, hkv, 16, 128), generator=g, device=DEV).bfloat16())


def inv_freq(rot, base=500000.0):
    n = rot // 2
    return [base ** (-i / n) for i in range(n)]


def check_append(c, rope, freqs, axis, inter, scale, qw, kw, eps, q_type, dtype_u):
    tokens, hq = c["q"].shape[:2]
    q_out = torch.full((tokens, hq, 128), 7.0, dtype=q_type, device=DEV)
    k_ref, v_ref = f64(c["k_cache"]), f64(c["v_cache"])
    k_tol, v_tol = np.zeros_like(k_ref), np.zeros_like(v_ref)
    q_ref = f64(q_out)
    q_tol = np.zeros_like(q_ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    L.locks_append_tokens(c["dims"], rope, c["q"], c["k"], c["v"], c["positions"], c["cache_index"], c["page_table"],
                          q_out, c["k_cache"], c["v_cache"], token_seq=c["token_seq"], q_weight=qw, k_weight=kw,
                          eps=eps, workspace=ws)
    q, k, v = f64(c["q"]), f64(c["k"]), f64(c["v"])
    qn = ref.norm(q, None if qw is None else f64(qw), eps)
    kn = ref.norm(k, None if kw is None else f64(kw), eps)
    pos, index = c["positions"].cpu().numpy(), c["cache_index"].cpu().numpy()
    seq, table = c["token_seq"].cpu().numpy(), c["page_table"].cpu().numpy()
    n = len(freqs)
    for t in range(tokens):
        if index[t] < 0:
            continue
        # whole turns off in extended precision: 2^31 radians leave a double 2^-22 of one
        angle = np.array([int(pos[axis[i], t]) * np.longdouble(freqs[i]) for i in range(n)], np.longdouble)
        angle = np.fmod(angle, 8 * np.arctan(np.longdouble(1))).astype(np.float64)
        page, row = table[seq[t], index[t] // 16], index[t] % 16
        s = max(1.0, abs(scale))
        q_ref[t] = ref.rotate(qn[t], angle, inter, scale)
        q_tol[t] = 17 * U * s * ref.pair_size(qn[t], n, inter)
        k_ref[page, :, row] = ref.rotate(kn[t], angle, inter, scale)
        k_tol[page, :, row] = 17 * U * s * ref.pair_size(kn[t], n, inter) + UB * np.abs(k_ref[page, :, row])
        v_ref[page, :, row] = v[t]
        v_tol[page, :, row] = UB * np.abs(v[t])
    if q_type == torch.bfloat16:
        q_tol += UB * np.abs(q_ref) * (q_tol > 0)
    assert np.all(np.abs(f64(q_out) - q_ref) <= q_tol)
    assert np.all(np.abs(f64(c["k_cache"]) - k_ref) <= k_tol)        # untouched rows: exactly as they were
    assert np.all(np.abs(f64(c["v_cache"]) - v_ref) <= v_tol)
    assert L.locks_get_device_status(ws) == 0


@pytest.mark.parametrize("tokens,seqs,hq,hkv", [(1, 1, 32, 8), (7, 3, 32, 2), (129, 5, 20, 4), (64, 64, 1, 1),
                                                (33, 2, 128, 8)])
@pytest.mark.parametrize("itype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rot,inter,axes,normed", [(128, False, 1, True), (64, True, 1, False), (96, False, 3, True),
                                                   (16, True, 4, True)])
def test_append(tokens, seqs, hq, hkv, itype, rot, inter, axes, normed):
    c = append_case(tokens, seqs, hq, hkv, itype, seed=tokens + rot, axes=axes)
    freqs = inv_freq(rot)
    axis = [i % axes for i in range(rot // 2)]
    w = (1 + 0.3 * torch.randn((2, 128), generator=gen(1), device=DEV)) if normed else (None, None)
    rope = L.make_rope(rot, freqs, interleaved=inter, axis=axis, num_axes=axes)
    check_append(c, rope, freqs, axis, inter, 1.0, w[0], w[1], 1e-5,
                 torch.float32 if tokens % 2 else torch.bfloat16, U)


def test_append_many_tokens_take_the_other_launch_shape():
    c = append_case(3001, 4, 32, 8, torch.bfloat16, seed=5, max_index=1000)
    freqs = inv_freq(128)
    check_append(c, L.make_rope(128, freqs), freqs, [0] * 64, False, 1.0, None, torch.ones(128, device=DEV), 1e-6,
                 torch.float32, U)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 301, -5000])
def test_append_far_positions_and_scale(far):
    """Angles of a million and of 2^31 radians keep full precision (the tolerance does not grow)."""
    c = append_case(65, 3, 8, 2, torch.float32, seed=9, far=far)
    freqs = [1.0, -0.75] + inv_freq(124)
    check_append(c, L.make_rope(128, freqs, scale=1.25), freqs, [0] * 64, False, 1.25, None, None, 1e-6,
                 torch.float32, U)


def test_append_padding_rows_no_rotation_and_keys_only():
    c = append_case(40, 4, 8, 2, torch.bfloat16, seed=3)
    c["cache_index"][5] = -1
    c["cache_index"][30:] = -7
    c["q"][30:] = float("nan")
    c["token_seq"][31] = 99                       # not read for padding
    check_append(c, None, [], [], False, 1.0, None, None, 1e-6, torch.float32, U)
    before = c["k_cache"].clone()
    c["k"][:, 0] = 2.0
    L.locks_append_tokens(c["dims"], None, None, c["k"], c["v"], None, c["cache_index"], c["page_table"], None,
                          c["k_cache"], c["v_cache"], token_seq=c["token_seq"])
    changed = (c["k_cache"] != before).any(-1)
    assert int(changed[:, 0].sum()) == 29 and int(changed[:, 1].sum()) == 0


def test_append_one_token_per_sequence_without_token_seq_and_strides():
    c = append_case(6, 6, 8, 2, torch.float16, seed=4)
    c["token_seq"] = torch.arange(6, dtype=torch.int32, device=DEV)
    freqs = inv_freq(128)
    wide = torch.randn((6, 3, 8, 128), generator=gen(2), device=DEV).half()
    c["q"] = wide[:, 1]                           # rows 24 heads apart
    c["k"] = torch.randn((1, 2, 128), generator=gen(3), device=DEV).half().expand(6, 2, 128)    # stride 0
    want = {n: c[n].clone() for n in ("k_cache", "v_cache")}
    check_append(c, L.make_rope(128, freqs), freqs, [0] * 64, False, 1.0, None, None, 0.0, torch.float32, U)
    q_out = torch.empty((6, 8, 128), device=DEV)
    L.locks_append_tokens(c["dims"], L.make_rope(128, freqs), c["q"], c["k"], c["v"], c["positions"][0],
                          c["cache_index"], c["page_table"], q_out, want["k_cache"], want["v_cache"])
    assert torch.equal(want["k_cache"], c["k_cache"]) and torch.equal(want["v_cache"], c["v_cache"])


def test_append_bad_indices_skip_the_token():
    c = append_case(8, 2, 8, 2, torch.bfloat16, seed=6)
    c["token_seq"][0] = 2
    c["token_seq"][1] = -1
    c["cache_index"][2] = 16 * c["dims"].max_pages_per_seq
    c["cache_index"][3] = (1 << 31) - 1
    lp = int(c["cache_index"][4]) // 16
    bad_seq = int(c["token_seq"][4])
    c["page_table"][bad_seq, lp] = c["dims"].num_phys_pages
    same = [t for t in range(5, 8) if int(c["token_seq"][t]) == bad_seq and int(c["cache_index"][t]) // 16 == lp]
    k0 = c["k_cache"].clone()
    q_out = torch.full((8, 8, 128), 3.0, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    L.locks_append_tokens(c["dims"], None, c["q"], c["k"], c["v"], None, c["cache_index"], c["page_table"], q_out,
                          c["k_cache"], c["v_cache"], token_seq=c["token_seq"], workspace=ws)
    assert L.locks_get_device_status(ws) == -6
    skipped = {0, 1, 2, 3, 4} | set(same)
    for t in range(8):
        if t in skipped:
            assert torch.all(q_out[t] == 3.0)
        else:
            assert torch.equal(q_out[t], c["q"][t].float())
    assert int((c["k_cache"] != k0).any(-1).any(1).sum()) == 8 - len(skipped)


# ------------------------------------------------------------------ prefix attention

def prefix_case(groups, own, hq, hkv, seed, q_type=torch.float32, max_prefix_pages=None, spare=0, scale=1.0):
    """groups: [(sequences, prefix tokens)], own: tokens per sequence (more sequences than the
    groups hold: the rest belong to none)."""
    g = gen(seed)
    B, G = len(own), len(groups)
    pp = max([(n + 15) // 16 for _, n in groups] + [0]) + spare if max_prefix_pages is None else max_prefix_pages
    mp = max([(n + 15) // 16 for n in own] + [0]) + spare
    phys = G * pp + B * mp + 2
    perm = torch.randperm(phys, generator=g, device=DEV).int()
    k = torch.randn((phys, hkv, 16, 128), generator=g, device=DEV)
    k += 0.5 * torch.randn((1, hkv, 1, 128), generator=g, device=DEV)
    start = np.concatenate([[0], np.cumsum([n for n, _ in groups])]).astype(np.int32)
    c = dict(dims=L.make_dims(B, hq, hkv, mp, phys), groups=groups, own=own,
             q=(scale * torch.randn((B, hq, 128), generator=g, device=DEV)).to(q_type), k=k.bfloat16(),
             v=torch.randn((phys, hkv, 16, 128), generator=g, device=DEV).bfloat16(),
             prefix_table=perm[:G * pp].view(G, pp).contiguous(),
             prefix_tokens=torch.tensor([n for _, n in groups], dtype=torch.int32, device=DEV),
             group_start=torch.from_numpy(start).to(DEV),
             page_table=perm[G * pp:G * pp + B * mp].view(B, mp).contiguous(),
             seq_tokens=torch.tensor(own, dtype=torch.int32, device=DEV))
    c["out"] = torch.full((B, hq, 128), float("nan"), device=DEV).bfloat16()
    c["lse"] = torch.full((B, hq), float("nan"), device=DEV)
    c["ws"] = L.alloc_prefix_workspace(c["dims"], G, DEV)
    c["ws"][256:] = 0xff                          # scratch may hold anything (here NaN)
    return c


def run_prefix(c, stream=None):
    L.locks_prefix_attention(c["dims"], c["q"], c["k"], c["v"], c["prefix_table"], c["prefix_tokens"],
                             c["group_start"], c["page_table"], c["seq_tokens"], c["out"], c["ws"], lse=c["lse"],
                             stream=stream)


def prefix_ref(c):
    hq, hkv = c["dims"].num_q_heads, c["dims"].num_kv_heads
    g = hq // hkv
    q, k, v = f64(c["q"]), f64(c["k"]), f64(c["v"])
    pt, ot = c["prefix_table"].cpu().numpy(), c["page_table"].cpu().numpy()
    ptok, own = c["prefix_tokens"].cpu().numpy(), c["seq_tokens"].cpu().numpy()
    start = c["group_start"].cpu().numpy()
    B = q.shape[0]
    out, lse = np.zeros((B, hq, 128)), np.full((B, hq), -np.inf)
    w, size = np.zeros((B, hq, 128)), np.zeros((B, hq))
    for b in range(B):
        rows = []
        for i in range(len(ptok)):
            if start[i] <= b < start[i + 1]:
                rows += [(pt[i, t // 16], t % 16) for t in range(ptok[i])]
        rows += [(ot[b, t // 16], t % 16) for t in range(own[b])]
        pg, rw = np.array([r[0] for r in rows], int), np.array([r[1] for r in rows], int)
        for h in range(hkv):
            sl = slice(h * g, (h + 1) * g)
            out[b, sl], lse[b, sl], w[b, sl], size[b, sl] = ref.attend(q[b, sl], k[pg, h, rw], v[pg, h, rw])
    return out, lse, w, size


def check_prefix(c, repeat=True):
    run_prefix(c)
    out, lse, w, size = prefix_ref(c)
    assert L.locks_get_device_status(c["ws"]) == 0
    e = 2.0 ** -15 * size
    got, got_lse = f64(c["out"]), f64(c["lse"])
    tol = (2 * e[..., None] + UB + 2.0 ** -20) * w + UB * np.abs(out)
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - out).max(), int(bad.sum()))
    none = np.isneginf(lse)
    assert np.array_equal(none, np.isneginf(got_lse)) and np.all(got[none] == 0)
    with np.errstate(invalid="ignore"):
        far = np.abs(got_lse - lse) > e + 2.0 ** -20 * (1 + np.abs(lse))
    assert not far[~none].any()
    if repeat:
        first, first_lse = c["out"].clone(), c["lse"].clone()
        run_prefix(c)
        assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])


@pytest.mark.parametrize("prefix", [1, 16, 100, 127, 128, 129, 256, 300, 2049])
def test_prefix_lengths(prefix):
    check_prefix(prefix_case([(2, prefix)], [0, 5], 8, 2, seed=prefix))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (32, 8), (32, 2), (20, 4), (16, 1), (128, 8)])
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_prefix_head_layouts(hq, hkv, q_type):
    check_prefix(prefix_case([(3, 777)], [33, 0, 150], hq, hkv, seed=hq + hkv, q_type=q_type))


@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seqs", [32, 33, 70])
def test_prefix_row_blocks(seqs, q_type):
    """128 rows of one block; a block more; a GQA group across two blocks (g = 5)."""
    check_prefix(prefix_case([(seqs, 700)], [i % 40 for i in range(seqs)], 8, 2, seed=seqs, q_type=q_type))
    check_prefix(prefix_case([(seqs, 300)], [0] * seqs, 20, 4, seed=seqs + 1, q_type=q_type))


def test_prefix_groups_and_sequences_outside_them():
    check_prefix(prefix_case([(3, 500), (0, 60), (1, 0), (4, 1025), (1, 7)], [0, 1, 200, 16, 0, 31, 128, 500, 9, 0, 77, 0],
                             16, 4, seed=3, spare=2))


def test_prefix_without_any_tokens_or_groups():
    check_prefix(prefix_case([(2, 0)], [0, 0], 8, 2, seed=1, spare=1))
    c = prefix_case([], [0, 3, 700], 8, 2, seed=2)
    c["prefix_table"] = c["prefix_table"][:0]
    check_prefix(c)
    c["prefix_table"] = None
    first = c["out"].clone()
    run_prefix(c)
    assert torch.equal(first, c["out"])


def test_prefix_many_sequences_many_groups():
    """More units than a warp holds at a time, most of them without own tokens."""
    groups = [(1 + i % 3, (i * 37) % 400) for i in range(45)]
    n = sum(s for s, _ in groups)
    own = [(b * 13) % 90 if b % 7 == 0 else 0 for b in range(n + 20)]
    check_prefix(prefix_case(groups, own, 4, 1, seed=8))


def test_prefix_thousands_of_sequences():
    groups = [(1 + i % 20, (i * 29) % 60) for i in range(260)]
    n = sum(s for s, _ in groups)
    check_prefix(prefix_case(groups, [(b * 7) % 41 if b % 3 else 0 for b in range(n + 300)], 2, 1, seed=18))


def test_cache_of_more_than_2_31_elements():
    """Rows appended to the last pages of a 9 GB pool, and attended there."""
    phys, hkv, hq = 140001, 8, 32
    kc = torch.empty((phys, hkv, 16, 128), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    kc[-40:] = float("nan")
    vc[-40:] = float("nan")
    assert kc.numel() > 2 ** 31
    dims = L.make_dims(2, hq, hkv, 3, phys)
    table = (phys - 1 - torch.arange(6, device=DEV)).view(2, 3).int().contiguous()
    own = [45, 20]
    seq = torch.tensor([0] * 45 + [1] * 20, dtype=torch.int32, device=DEV)
    index = torch.tensor(list(range(45)) + list(range(20)), dtype=torch.int32, device=DEV)
    qkv = torch.randn((65, hq + 2 * hkv, 128), generator=gen(3), device=DEV).bfloat16()
    L.locks_append_tokens(dims, None, None, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], None, index, table, None, kc, vc,
                          token_seq=seq)
    for t in (0, 44, 45, 64):
        page, row = int(table[int(seq[t]), int(index[t]) // 16]), int(index[t]) % 16
        assert torch.equal(kc[page, :, row], qkv[t, hq:hq + hkv]) and torch.equal(vc[page, :, row], qkv[t, hq + hkv:])
    q = torch.randn((2, hq, 128), generator=gen(4), device=DEV)
    out = torch.empty((2, hq, 128), dtype=torch.bfloat16, device=DEV)
    ws = L.alloc_prefix_workspace(dims, 0, DEV)
    L.locks_prefix_attention(dims, q, kc, vc, None, None, None, table, torch.tensor(own, dtype=torch.int32, device=DEV),
                             out, ws)
    assert L.locks_get_device_status(ws) == 0
    at = [0, 45, 65]
    for b in range(2):
        x = f64(qkv[at[b]:at[b + 1]])
        for h in range(hkv):
            want = ref.attend(f64(q[b, 4 * h:4 * h + 4]), x[:, hq + h], x[:, hq + hkv + h])[0]
            assert np.abs(f64(out[b, 4 * h:4 * h + 4]) - want).max() < 2e-2


def test_prefix_long_split_over_all_ctas():
    check_prefix(prefix_case([(5, 70001)], [3000, 1, 0, 20, 555], 8, 1, seed=11))


def test_prefix_rows_behind_the_end_are_never_used():
    """NaN and infinities behind the last token of every list, in and after its page."""
    for dtype in (torch.float32, torch.bfloat16):
        c = prefix_case([(2, 261), (1, 5)], [19, 0, 130], 8, 2, seed=7, spare=2, q_type=dtype)
        used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool, device=DEV)
        for tab, n in list(zip(c["prefix_table"], [261, 5])) + list(zip(c["page_table"], [19, 0, 130])):
            for t in range(n):
                used[int(tab[t // 16]), t % 16] = True
        behind = ~used[:, None, :].expand(-1, 2, -1)
        clean = {n: c[n].clone() for n in ("k", "v")}
        run_prefix(c)
        first, first_lse = c["out"].clone(), c["lse"].clone()
        for kk, vv in ((float("nan"), float("nan")), (float("inf"), -float("inf"))):
            c["k"], c["v"] = clean["k"].clone(), clean["v"].clone()
            c["k"][behind] = kk
            c["v"][behind] = vv
            run_prefix(c)
            assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])


def test_prefix_steep_and_growing_scores():
    """Large scores whose maximum keeps growing along the prefix (the accumulator is rescaled)
    and one dominant key at the very end."""
    c = prefix_case([(3, 1500)], [40, 0, 9], 8, 2, seed=5, scale=3.0)
    pt = c["prefix_table"][0].long()
    ramp = torch.linspace(0.0, 3.0, pt.numel() * 16, device=DEV).view(-1, 1, 16, 1)
    c["k"][pt] = (c["k"][pt].float() * ramp).bfloat16()
    check_prefix(c)
    c["k"][pt[-1], :, 1499 % 16] = (4 * c["q"][0, ::4]).bfloat16()
    check_prefix(c)


def test_prefix_nonfinite_values_stay_in_their_rows():
    """A NaN in one sequence's own tokens or query reaches that sequence alone."""
    c = prefix_case([(4, 300)], [20, 20, 20, 20], 8, 2, seed=6)
    run_prefix(c)
    first = c["out"].clone()
    c["v"][int(c["page_table"][1, 0]), 0, 3] = float("nan")
    c["q"][2, 5] = float("nan")
    run_prefix(c)
    got = c["out"]
    assert torch.equal(got[0], first[0]) and torch.equal(got[3], first[3])
    assert torch.isnan(got[1, :4].float()).all() and torch.equal(got[1, 4:], first[1, 4:])
    assert torch.isnan(got[2, 5].float()).all() and torch.equal(got[2, :5], first[2, :5])


def test_prefix_bad_lengths_bounds_and_pages():
    c = prefix_case([(2, 300), (2, 100)], [20, 30, 0, 7], 8, 2, seed=9)
    for name, at, value, as_if in (("seq_tokens", 1, 16 * c["dims"].max_pages_per_seq + 1, 0),
                                   ("seq_tokens", 0, -1, 0), ("prefix_tokens", 0, -5, 0),
                                   ("prefix_tokens", 1, 1 << 30, 0), ("group_start", 2, 5, 2),
                                   ("group_start", 0, -1, None)):
        kept = c[name].clone()
        c[name][at] = value
        c["ws"][:256] = 0
        run_prefix(c)
        assert L.locks_get_device_status(c["ws"]) == -6, name
        got, got_lse = c["out"].clone(), c["lse"].clone()
        if as_if is not None:
            c[name][at] = as_if
        else:                                     # the first group is dropped
            c["group_start"][0] = 2
        c["ws"][:256] = 0
        run_prefix(c)
        assert L.locks_get_device_status(c["ws"]) == 0
        assert torch.equal(got, c["out"]) and torch.equal(got_lse, c["lse"]), name
        c[name].copy_(kept)
    # overlapping groups: the later one is dropped
    c["group_start"].copy_(torch.tensor([0, 3, 2], dtype=torch.int32))
    c["ws"][:256] = 0
    run_prefix(c)
    assert L.locks_get_device_status(c["ws"]) == -6
    # a page out of range is read as page 0
    c = prefix_case([(2, 300)], [20, 30], 8, 2, seed=10)
    c["page_table"][0, 1] = -3
    c["prefix_table"][0, 2] = c["dims"].num_phys_pages
    run_prefix(c)
    assert L.locks_get_device_status(c["ws"]) == -6
    got = c["out"].clone()
    c["page_table"][0, 1] = 0
    c["prefix_table"][0, 2] = 0
    run_prefix(c)
    assert torch.equal(got, c["out"])


def test_prefix_agrees_with_attention_over_all_pages():
    """Own tokens alone, whole pages: what locks_sparse_attention gives with every page kept."""
    c = prefix_case([], [320, 160], 8, 2, seed=12)
    c["prefix_table"] = None
    run_prefix(c)
    sel = torch.arange(20, dtype=torch.int32, device=DEV).expand(2, 2, 20).contiguous()
    n = torch.tensor([[20, 20], [10, 10]], dtype=torch.int32, device=DEV)
    out = torch.empty((2, 8, 128), dtype=torch.int16, device=DEV)
    lse = torch.empty((2, 8), device=DEV)
    L.locks_sparse_attention(c["dims"], c["q"], c["k"], c["v"], c["page_table"], sel, n, 20, out, lse=lse)
    assert np.abs(bf16_out(out) - f64(c["out"])).max() < 2e-2
    assert (lse - c["lse"]).abs().max() < 1e-4


def test_prefix_in_a_graph_follows_its_lengths_and_two_calls_overlap():
    c = prefix_case([(3, 400), (2, 900)], [10, 200, 0, 64, 3], 16, 4, seed=13, spare=2)
    d = prefix_case([(4, 5000)], [50] * 4, 32, 8, seed=14)
    run_prefix(c), run_prefix(d)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run_prefix(c)
    for step in range(3):
        c["seq_tokens"] += 1
        c["prefix_tokens"] -= 7
        c["group_start"][1] = 3 - step % 2
        want = prefix_ref(c)[0]
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):             # another call with a workspace of its own beside it
            run_prefix(d)
        torch.cuda.synchronize()
        assert np.abs(f64(c["out"]) - want).max() < 2e-2
    check_prefix(d)


# ------------------------------------------------------------------ mass

def check_mass(scores, seq, old, decay, partials=None, dims=None, in_place=False):
    B, hq, P = scores.shape
    dims = L.make_dims(B, hq, next(h for h in (1, 2, 4, 8) if hq % h == 0 and hq // h <= 16), P, 1) if dims is None else dims
    ws = L.alloc_mass_workspace(dims, DEV)
    ws[256:] = 0xff
    mass = old.clone()
    out = mass if in_place else torch.full_like(mass, -3.0)
    L.locks_accumulate_mass(dims, scores, seq, mass, out, ws, decay=decay, lse_partials=partials)
    assert L.locks_get_device_status(ws) == 0
    n = seq.cpu().numpy()
    want = ref.mass(scores.cpu().numpy(), n, old.cpu().numpy(), decay)
    got = out.cpu().numpy().astype(np.float64)
    for b in range(B):
        s = scores[b, :, :n[b]].cpu().numpy().astype(np.float64)
        s = np.where(np.isfinite(s), s, 0.0)
        depth = np.ptp(s) if s.size else 0.0
        kept = np.abs(old[b, :n[b]].cpu().numpy().astype(np.float64) * decay) if decay else 0.0
        tol = (16 + 4 * depth) * U * np.abs(want[b]) + 2 * U * kept + 1e-38
        assert np.all(np.abs(got[b, :n[b]] - want[b]) <= tol), (b, np.abs(got[b, :n[b]] - want[b]).max())
        rest = old[b, n[b]:].cpu().numpy() if in_place else np.float32(-3.0)
        assert np.all(got[b, n[b]:] == rest)
    return out


@pytest.mark.parametrize("B,hq,P", [(1, 1, 1), (1, 32, 8192), (3, 32, 1001), (2, 16, 2050), (1, 128, 515), (5, 8, 4),
                                    (1, 4, 40003)])
@pytest.mark.parametrize("decay", [1.0, 0.9, 0.0])
def test_mass(B, hq, P, decay):
    g = gen(P)
    scores = 3 * torch.randn((B, hq, P), generator=g, device=DEV)
    seq = torch.randint(0, P + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    seq[0] = P
    for b in range(B):
        scores[b, :, int(seq[b]):] = float("nan")             # never read
    old = torch.rand((B, P), generator=g, device=DEV)
    if decay == 0.0:
        old[:] = float("nan")                                 # not read either
        old_ref = torch.zeros_like(old)
        dims = L.make_dims(B, hq, 8 if hq == 128 else 2 if hq == 32 else 1, P, 1)
        ws, out = L.alloc_mass_workspace(dims, DEV), torch.zeros_like(old)
        L.locks_accumulate_mass(dims, scores, seq, old, out, ws, decay=0.0)
        other = torch.zeros_like(old)
        L.locks_accumulate_mass(dims, scores, seq, old_ref, other, ws, decay=1.0)
        assert torch.equal(out, other)
        return
    check_mass(scores, seq, old, decay)
    check_mass(scores, seq, old, decay, in_place=True)
    seq.zero_()
    check_mass(scores, seq, old, decay)


def test_mass_unaligned_rows():
    base = torch.randn(2 * 8 * 400 + 1, generator=gen(2), device=DEV)
    seq = torch.tensor([400, 123], dtype=torch.int32, device=DEV)
    old = torch.rand((2, 400), generator=gen(3), device=DEV)
    check_mass(base[1:].view(2, 8, 400), seq, old, 1.0)


def test_mass_nonfinite_scores_add_nothing():
    s = torch.randn((2, 4, 300), generator=gen(4), device=DEV)
    s[0, 0, 5] = float("nan")
    s[0, 1, 6] = float("inf")
    s[0, 2, 7] = -float("inf")
    s[0, 3] = -float("inf")
    s[1, 0] = float("nan")
    s[1, 1, :200] = 1e30
    seq = torch.tensor([300, 250], dtype=torch.int32, device=DEV)
    check_mass(s, seq, torch.zeros((2, 300), device=DEV), 1.0)


def test_mass_bad_lengths_skip_the_sequence():
    s = torch.randn((3, 4, 64), generator=gen(4), device=DEV)
    seq = torch.tensor([65, 20, -1], dtype=torch.int32, device=DEV)
    dims = L.make_dims(3, 4, 1, 64, 1)
    ws = L.alloc_mass_workspace(dims, DEV)
    out = torch.full((3, 64), 9.0, device=DEV)
    L.locks_accumulate_mass(dims, s, seq, torch.zeros((3, 64), device=DEV), out, ws)
    assert L.locks_get_device_status(ws) == -6
    assert torch.all(out[0] == 9) and torch.all(out[2] == 9) and torch.all(out[1, 20:] == 9)
    assert abs(float(out[1, :20].sum()) - 1) < 1e-5


@pytest.mark.parametrize("hq,hkv,P", [(32, 8, 700), (32, 2, 3001), (4, 1, 64)])
def test_mass_from_the_scorers_partials(hq, hkv, P):
    """With locks_score_pages' partials, the mass of the scores it wrote."""
    g = gen(hq + P)
    B = 2
    dims = L.make_dims(B, hq, hkv, P, B * P)
    summ = L.Summaries.empty(B * P, hkv, DEV)
    summ.mu.random_(-127, 128, generator=g)
    summ.coef.random_(-127, 128, generator=g)
    summ.scales[..., 0] = torch.tensor(0.01, dtype=torch.float16).view(torch.int16)
    table = torch.randperm(B * P, generator=g, device=DEV).view(B, P).int()
    seq = torch.tensor([P, P // 2], dtype=torch.int32, device=DEV)
    q = torch.randn((B, hq, 128), generator=g, device=DEV)
    scores = torch.zeros((B, hq, P), device=DEV)
    partials = torch.zeros(L.locks.lse_partials_shape(dims), device=DEV)
    L.locks_score_pages(dims, q, summ, table, seq, scores, lse_partials=partials)
    old = torch.rand((B, P), generator=g, device=DEV)
    a = check_mass(scores, seq, old, 0.75, partials=partials, dims=dims)
    b = check_mass(scores, seq, old, 0.75, dims=dims)
    assert (a - b).abs().max() <= 1e-6


# ------------------------------------------------------------------ eviction

def check_evict(mass, table, seq, keep, sink, recent, extra, in_place=False, status=0):
    B, P = mass.shape
    dims = L.make_dims(B, 1, 1, P, 1 << 20)
    cap = max(1, P - keep)
    m0, t0, s0 = mass.cpu().numpy(), table.cpu().numpy(), seq.cpu().numpy()
    mass, table, seq = mass.clone(), table.clone(), seq.clone()
    mo, to, so = (mass, table, seq) if in_place else (torch.full_like(mass, -5.0), torch.full_like(table, -5),
                                                      torch.full_like(seq, -5))
    ev = torch.full((B, cap), -7, dtype=torch.int32, device=DEV)
    ne = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    L.locks_evict_pages(dims, mass, table, seq, keep, mo, to, so, ev, ne, sink_pages=sink, recent_pages=recent,
                        extra_pages=extra, workspace=ws)
    assert L.locks_get_device_status(ws) == status
    mo, to, so, ev, ne = (x.cpu().numpy() for x in (mo, to, so, ev, ne))
    for b in range(B):
        if not 0 <= s0[b] <= P:
            assert ne[b] == 0 and np.all(ev[b] == -7)
            continue
        wt, wm, we = ref.evict(m0[b], t0[b], int(s0[b]), keep, sink, recent, extra)
        assert ne[b] == len(we) and so[b] == s0[b] - len(we)
        assert np.array_equal(to[b, :len(wt)], wt) and np.array_equal(mo[b, :len(wm)], wm, equal_nan=True)
        assert np.array_equal(ev[b, :len(we)], we) and np.all(ev[b, len(we):] == -7)
        if in_place:
            assert np.array_equal(to[b, len(wt):], t0[b, len(wt):])
        else:
            assert np.all(to[b, len(wt):] == -5) and np.all(mo[b, len(wm):] == -5)


def evict_case(B, P, seed, ties=0.3):
    g = gen(seed)
    mass = torch.exp(3 * torch.randn((B, P), generator=g, device=DEV))
    mass[torch.rand((B, P), generator=g, device=DEV) < ties] = 0.0
    return mass, torch.randint(0, 1 << 20, (B, P), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("B,P,keep,sink,recent,extra", [
    (1, 1, 0, 0, 0, 0), (1, 1, 1, 0, 0, 3), (3, 17, 5, 1, 2, 0), (8, 260, 250, 1, 4, 1), (2, 4096, 4000, 4, 64, 2),
    (2, 4097, 100, 0, 0, 4), (1, 65540, 60000, 4, 128, 4), (3, 20000, 19999, 0, 0, 0), (2, 9000, 0, 0, 0, 2),
    (2, 700, 5, 2, 3, 0)])
def test_evict(B, P, keep, sink, recent, extra):
    mass, table = evict_case(B, P, seed=P)
    seq = torch.tensor([max(0, P - extra - 3 * b) for b in range(B)], dtype=torch.int32, device=DEV)
    for in_place in (False, True):
        check_evict(mass, table, seq, keep, sink, recent, extra, in_place)
    check_evict(mass, table, (seq // 3).int(), keep, sink, recent, extra)
    check_evict(mass, table, torch.zeros_like(seq), keep, sink, recent, extra)


def test_evict_ties_zeros_and_nonfinite_masses():
    for P in (500, 10000):
        mass, table = evict_case(4, P, seed=1)
        mass[0] = 0.25                                        # all equal: the lowest pages go
        mass[1, ::2] = -0.0                                   # as +0
        mass[1, 1::2] = 0.0
        mass[2, ::7] = float("nan")                           # before everything
        mass[2, 1::7] = -float("inf")
        mass[2, 2::7] = float("inf")
        mass[3] = -mass[3]
        seq = torch.full((4,), P - 1, dtype=torch.int32, device=DEV)
        for keep in (P - 2, P // 2, 30):
            check_evict(mass, table, seq, keep, 3, 5, 1)


def test_evict_largest_table():
    mass, table = evict_case(1, 393216, seed=2)
    seq = torch.tensor([393210], dtype=torch.int32, device=DEV)
    check_evict(mass, table, seq, 300000, 4, 16, 6, in_place=True)


def test_evict_bad_lengths_skip_the_sequence():
    for P in (100, 5000):
        mass, table = evict_case(3, P, seed=3)
        seq = torch.tensor([P + 1, P, -1], dtype=torch.int32, device=DEV)
        check_evict(mass, table, seq, P // 2, 1, 1, 0, status=-6)


def test_evict_in_a_graph_until_the_window_holds():
    """A captured in-place eviction, replayed as the window grows page by page."""
    P, keep = 64, 40
    mass, table = evict_case(2, P, seed=4)
    dims = L.make_dims(2, 1, 1, P, 1 << 20)
    seq = torch.tensor([20, 40], dtype=torch.int32, device=DEV)
    ev = torch.empty((2, P - keep), dtype=torch.int32, device=DEV)
    ne = torch.empty(2, dtype=torch.int32, device=DEV)

    def call():
        L.locks_evict_pages(dims, mass, table, seq, keep, mass, table, seq, ev, ne, sink_pages=1, recent_pages=2)

    state = [t.clone() for t in (mass, table, seq)]
    call()
    for t, o in zip((mass, table, seq), state):
        t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for step in range(30):
        seq += 1
        m0, t0, s0 = mass.cpu().numpy(), table.cpu().numpy(), seq.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            wt, wm, we = ref.evict(m0[b], t0[b], int(s0[b]), keep, 1, 2, 0)
            assert int(seq[b]) == len(wt) <= keep and int(ne[b]) == len(we)
            assert np.array_equal(table[b, :len(wt)].cpu().numpy(), wt)
