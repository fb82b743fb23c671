"""GPU tests of the packed cache (packing, unpacking, attention over packed pages) against the
float64 forms in pool_ref.

Codes and unpacked values are compared exactly: the definition rounds (x - zero) / scale once.
(A quotient of bf16 values is either on a border between two codes or 2^-20 away from it at
least as long as x and zero lie within 2^12 of each other, which the inputs here do.)

Attention, counted from the arithmetic (u = 2^-24, half a step of fp32; half a step of bf16 is
2^-8 of the value):
* scores: off by e = 2^-15 max_t sum |q| (|zero| + |scale code|) / sqrt(128). q as two parts
  keeps it to 2^-16 (bf16 parts, recent tokens); the sums have up to 64 + 16 additions, cut off
  rather than rounded at worst: 160 u < 2^-16.
* weights: 2 e (itself and the normaliser), 2^-11 for their rounding to fp16, 2^-19 for exp2 and the
  product with the scale; sums over n pages another 2 u for each.
* out: that times sum p (|zero| + |scale code|), and 2^-8 of itself.
"""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import DEV, bf16_out

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ packing

def cache_pair(pages, hkv, seed, kind="normal"):
    g = gen(seed)
    k, v = (torch.randn((pages, hkv, 16, 128), generator=g, device=DEV) for _ in range(2))
    if kind == "grid":                               # many quotients on borders between codes
        k, v = (torch.round(x * 3) for x in (k, v))
    elif kind == "outliers":
        k = k * torch.exp(2 * torch.randn((1, hkv, 1, 128), generator=g, device=DEV)) + 3
        v = v * 1e-3 + 1
    elif kind == "large":
        k, v = k * 2.0 ** 100, v * 2.0 ** 118
    elif kind == "small":
        k, v = k * 2.0 ** -100, v * 2.0 ** -124
    elif kind == "flat":                             # constant groups, groups with one other value
        k = torch.full_like(k, -1.25)
        k[..., 5] = 7
        k[:, :, 3] = 0
        v = torch.full_like(v, 2.0 ** -130)
        v[:, :, ::2] = 3
    return k.bfloat16(), v.bfloat16()


def check_units(units, k, v):
    for x, group, (code, scale, zero) in zip((k, v), (32, 64), ref.fields(units)):
        c, s, z = ref.codes_of(x, group)
        assert np.array_equal(s, scale) and np.array_equal(z, zero)
        bad = c != code
        assert not bad.any(), (int(bad.sum()), x[bad][:4], s[bad][:4], z[bad][:4], code[bad][:4], c[bad][:4])


@pytest.mark.parametrize("kind", ["normal", "grid", "outliers", "large", "small", "flat"])
@pytest.mark.parametrize("hkv", [1, 8])
def test_pack_and_unpack(kind, hkv):
    n, pool = 9, 13
    k, v = cache_pair(pool, hkv, 5, kind)
    dims = L.make_dims(1, hkv, hkv, 1, pool)
    src = torch.randperm(pool, generator=gen(1), device=DEV)[:n].int()
    dst = torch.randperm(n + 2, generator=gen(2), device=DEV)[:n].int()
    packed = torch.full((n + 2, hkv, L.LOCKS_PACKED_BYTES), 0xA5, dtype=torch.uint8, device=DEV)
    L.locks_pack_pages(dims, k, v, src, dst, n, packed)
    units = packed.cpu().numpy()
    check_units(units[dst.long().cpu()], f64(k[src.long()]), f64(v[src.long()]))
    rest = np.setdiff1d(np.arange(n + 2), dst.cpu().numpy())
    assert (units[rest] == 0xA5).all()
    ko, vo = (torch.full_like(x, 9.0) for x in (k, v))
    L.locks_unpack_pages(dims, packed, dst, src, n, ko, vo)
    rest = np.setdiff1d(np.arange(pool), src.cpu().numpy())
    for got, want, old in zip((ko, vo), ref.unpack(units[dst.long().cpu()]), (k, v)):
        got = f64(got)
        assert np.array_equal(got[src.cpu().numpy()], ref.cache_ref.bf16(want))
        assert (got[rest] == 9.0).all()
    # half a step of the codes, or 2^-8 of the range where the scale was rounded down; the output's
    # rounding; ranges that are too small for a scale
    for got, x, group in ((ko, k, 32), (vo, v, 64)):
        x = f64(x[src.long()])
        _, s, _ = ref.codes_of(x, group)
        err = np.abs(f64(got)[src.cpu().numpy()] - x)
        assert (err <= s * (0.5 + 15 * 2.0 ** -8) + np.abs(x) * 2.0 ** -7 + 15 * 2.0 ** -126).all()


def test_pack_many_pages_and_none():
    k, v = cache_pair(700, 2, 3)
    dims = L.make_dims(1, 4, 2, 1, 700)
    packed = torch.zeros((700, 2, 2432), dtype=torch.uint8, device=DEV)
    ids = torch.arange(700, dtype=torch.int32, device=DEV)
    L.locks_pack_pages(dims, k, v, ids, None, 0, packed)
    assert int(packed.max()) == 0
    L.locks_pack_pages(dims, k, v, ids, None, 700, packed)
    check_units(packed.cpu().numpy(), f64(k), f64(v))


def test_pack_lists_with_padding_and_bad_ids():
    k, v = cache_pair(6, 2, 4)
    dims = L.make_dims(1, 4, 2, 1, 6)
    packed = torch.full((4, 2, 2432), 7, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    L.locks_pack_pages(dims, k, v, i32([3, -1, 5, 2]), i32([0, 1, -1, 3]), 4, packed, workspace=ws)
    assert L.locks_get_device_status(ws) == 0
    units = packed.cpu().numpy()
    check_units(units[[0, 3]], f64(k[[3, 2]]), f64(v[[3, 2]]))
    assert (units[1:3] == 7).all()
    for src, dst in (([6], [0]), ([0], [4]), ([2 ** 31 - 1], [1])):
        ws.zero_()
        L.locks_pack_pages(dims, k, v, i32(src), i32(dst), 1, packed, workspace=ws)
        assert L.locks_get_device_status(ws) == -6
        assert np.array_equal(packed.cpu().numpy(), units)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        ws.zero_()
        L.locks_unpack_pages(dims, packed, i32(dst), i32(src), 1, ko, vo, workspace=ws)
        assert L.locks_get_device_status(ws) == -6 and float(ko.abs().max()) == 0 == float(vo.abs().max())


def test_pack_nonfinite_groups_unpack_to_nothing_finite():
    k, v = cache_pair(3, 1, 8)
    k[0, 0, 4, 40] = float("nan")                    # group 1 of token 4
    k[1, 0, 0, 127] = float("inf")
    v[2, 0, 15, 64] = -float("inf")
    v[0, 0, 2, 3] = 3e38                             # a range past fp32's
    v[0, 0, 2, 4] = -3e38
    dims = L.make_dims(1, 1, 1, 1, 3)
    packed = torch.zeros((3, 1, 2432), dtype=torch.uint8, device=DEV)
    ids = i32([0, 1, 2])
    L.locks_pack_pages(dims, k, v, ids, None, 3, packed)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    L.locks_unpack_pages(dims, packed, ids, None, 3, ko, vo)
    bad_k, bad_v = torch.zeros_like(k, dtype=torch.bool), torch.zeros_like(v, dtype=torch.bool)
    bad_k[0, 0, 4, 32:64] = True
    bad_k[1, 0, 0, 96:] = True
    bad_v[2, 0, 15, 64:] = True
    bad_v[0, 0, 2, :64] = True
    assert torch.equal(~torch.isfinite(ko), bad_k) and torch.equal(~torch.isfinite(vo), bad_v)


# ---------------------------------------------------------------- attention

def make_case(pages, recent, hq, hkv, seed=0, q_type=torch.float32, spare=0, selected=None, steep=1.0, width=None,
              zero=None):
    """pages[b] packed pages and recent[b] tokens of sequence b; selected[b][h]: logical pages."""
    g, B = gen(seed), len(pages)
    P = max(pages) if width is None else width
    R = max((r + 15) // 16 for r in recent)
    phys, num = B * P + spare + 1, B * R + 1
    u = torch.randint(0, 256, (phys, hkv, 2432), generator=g, device=DEV, dtype=torch.uint8)
    scale = 0.3 * torch.exp(0.3 * torch.randn((phys, hkv, 96), generator=g, device=DEV))
    z = -7.5 * scale + 0.5 * torch.randn((phys, hkv, 96), generator=g, device=DEV)
    if zero is not None:
        z = zero + z
    for lo, n, a in ((2048, 4, 0), (2304, 2, 64)):
        both = torch.stack([x[..., a:a + 16 * n].reshape(phys, hkv, 16, n) for x in (scale, z)], 3)
        u[..., lo:lo + 64 * n] = both.bfloat16().reshape(phys, hkv, -1).contiguous().view(torch.uint8)
    order = torch.randperm(phys, generator=g, device=DEV).int()
    u[int(order[-1])] = 0xFF                         # a page that nobody's table names: NaN scales
    c = dict(B=B, hq=hq, hkv=hkv, pages=list(pages), recent=list(recent), packed=u,
             table=order[:B * P].view(B, P).contiguous(), seq_pages=i32(pages), R=R,
             q=(steep * torch.randn((B, hq, 128), generator=g, device=DEV)).to(q_type),
             out=torch.full((B, hq, 128), 77.0, dtype=torch.bfloat16, device=DEV),
             lse=torch.full((B, hq), 77.0, device=DEV), dims=L.make_dims(B, hq, hkv, P, num), lists=selected,
             sel=None, n_sel=None)
    c["k"], c["v"] = (torch.randn((num, hkv, 16, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
    c["recent_table"] = torch.randperm(num, generator=g, device=DEV)[:B * R].view(B, R).int().contiguous()
    c["recent_tokens"] = i32(recent)
    if selected is not None:
        cap = max(1, max(len(x) for s in selected for x in s))
        sel = np.full((B, hkv, cap), -1, np.int32)
        for b in range(B):
            for h in range(hkv):
                sel[b, h, :len(selected[b][h])] = selected[b][h]
        c["sel"], c["n_sel"] = torch.from_numpy(sel).to(DEV), i32([[len(x) for x in s] for s in selected])
    c["ws"] = L.alloc_packed_workspace(c["dims"], DEV)
    return c


def run(c, **kw):
    args = dict(selected=c["sel"], n_selected=c["n_sel"], lse=c["lse"])
    if c["R"]:
        args.update(k_cache=c["k"], v_cache=c["v"], recent_table=c["recent_table"], recent_tokens=c["recent_tokens"])
    args.update(kw)
    L.locks_packed_attention(c["dims"], c["q"], c["packed"], c["table"], c["seq_pages"], c["out"], c["ws"], **args)


def tokens_of(c, b, h, units, table):
    logical = range(c["pages"][b]) if c["lists"] is None else c["lists"][b][h]
    u = units[table[b][list(logical)], h]
    (k, v), (ks, vs) = ref.unpack(u), ref.sizes(u)
    parts = [x.reshape(-1, 128) for x in (k, v, ks, vs)]
    if c["recent"][b]:
        rows = c["recent_table"][b].long()
        rk, rv = (f64(c[n][rows, h]).reshape(-1, 128)[:c["recent"][b]] for n in ("k", "v"))
        parts = [np.concatenate(p) for p in zip(parts, (rk, rv, np.abs(rk), np.abs(rv)))]
    return parts


def check(c, status=0):
    run(c)
    assert L.locks_get_device_status(c["ws"]) == status
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
            assert (np.abs(got[b, rows] - want) <= tol + 1e-30).all(), (b, h, np.abs(got[b, rows] - want).max())
            if len(parts[0]) == 0:
                assert (lse[b, rows] == -np.inf).all()
                continue
            assert (np.abs(lse[b, rows] - want_lse) <= e + 2.0 ** -22 * np.abs(want_lse) + 2.0 ** -18 + n * 2.0 ** -23
                    ).all(), (b, h)


@pytest.mark.parametrize("pages,recent", [(1, 0), (2, 1), (0, 1), (0, 16), (3, 17), (40, 31), (700, 64), (0, 0), (129, 0)])
def test_lengths_of_one_sequence(pages, recent):
    check(make_case([pages], [recent], 8, 2, seed=pages + recent))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (16, 8), (6, 2), (32, 8), (20, 4), (6, 1), (16, 2), (9, 1), (32, 2),
                                    (16, 1), (128, 8)])
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_head_layouts(hq, hkv, q_type):
    check(make_case([37, 0, 5], [20, 3, 0], hq, hkv, seed=hq + hkv, q_type=q_type))


def test_ragged_batches_and_empty_rows():
    check(make_case([0, 3, 0, 0, 250, 1, 0], [0, 0, 5, 0, 48, 0, 0], 8, 4, seed=1))
    check(make_case([0, 0], [0, 0], 4, 2, seed=2, width=3))
    n = 90
    check(make_case([(b * 17) % 23 if b % 3 else 0 for b in range(n)], [(b * 7) % 40 for b in range(n)], 8, 2, seed=3))


@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 1), (16, 1)])
def test_many_sequences(hq, hkv):
    """More sequences than a CTA has threads: each thread sums several; rows end inside warps."""
    n = 1500
    check(make_case([(b * 7) % 5 for b in range(n)], [(b * 11) % 20 if b % 4 == 0 else 0 for b in range(n)], hq, hkv,
                    seed=4))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 2), (24, 2)])
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_long_rows_over_all_ctas(hq, hkv, q_type):
    check(make_case([9001, 4, 2500], [60, 0, 33], hq, hkv, seed=hq, q_type=q_type))


def test_selected_pages():
    rng = np.random.default_rng(3)
    pages = [50, 7, 333]
    lists = [[sorted(rng.choice(n, size=min(n, k), replace=False)) for k in (7, 60)] for n in pages]
    lists[1][0] = []
    check(make_case(pages, [3, 0, 29], 16, 2, seed=5, selected=lists))
    check(make_case(pages, [0, 0, 0], 16, 2, seed=6, selected=lists))
    # any order, a page twice
    check(make_case(pages, [0, 2, 0], 8, 2, seed=7, selected=[[[4, 2], [0]], [[6], [5, 5, 1]], [[], [332, 0]]]))


def test_selected_needs_no_seq_pages():
    c = make_case([20], [0], 8, 2, seed=5, selected=[[[3, 9], [1]]])
    check(c)
    first = c["out"].clone()
    c["out"].zero_()
    L.locks_packed_attention(c["dims"], c["q"], c["packed"], c["table"], None, c["out"], c["ws"], selected=c["sel"],
                             n_selected=c["n_sel"])
    assert torch.equal(first, c["out"])


def test_no_packed_pages_at_all():
    c = make_case([0, 0], [37, 16], 8, 2, seed=9)
    c["dims"].max_pages_per_seq = 0
    check(c)
    first = c["out"].clone()
    c["out"].zero_()
    L.locks_packed_attention(c["dims"], c["q"], None, None, c["seq_pages"], c["out"], c["ws"], k_cache=c["k"],
                             v_cache=c["v"], recent_table=c["recent_table"], recent_tokens=c["recent_tokens"])
    assert torch.equal(first, c["out"])


def test_scores_that_keep_growing():
    """The maximum moves again and again, and one page at the end dominates."""
    for q_type in (torch.float32, torch.bfloat16):
        c = make_case([800], [40], 8, 2, seed=12, steep=2.0, q_type=q_type)
        sz = c["packed"][..., 2048:2304].contiguous().view(torch.bfloat16).view(-1, 2, 16, 2, 4)
        ramp = torch.zeros(c["packed"].shape[0], device=DEV)
        ramp[c["table"][0].long()] = torch.linspace(0, 3, 800, device=DEV)
        new = (sz.float() * ramp[:, None, None, None, None]).bfloat16()
        c["packed"][..., 2048:2304] = new.reshape(c["packed"].shape[0], 2, -1).contiguous().view(torch.uint8)
        check(c)


def test_keys_with_a_large_common_part():
    """Zeros far larger than the groups' ranges: they are counted once, not with every code."""
    check(make_case([60, 9], [5, 0], 8, 2, seed=13, zero=30.0, steep=0.3))


@pytest.mark.parametrize("size", [2.0 ** -40, 1e-6, 1e6, 2.0 ** 40])
def test_queries_of_any_size(size):
    c = make_case([30], [9], 8, 2, seed=14)
    c["q"] *= size
    sz = c["packed"][..., 2048:2304].contiguous().view(torch.bfloat16)      # keys as small as the queries are large
    c["packed"][..., 2048:2304] = (sz.float() / size).bfloat16().view(torch.uint8)
    c["k"] = (c["k"].float() / size).bfloat16()
    check(c)


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 46])
def test_values_of_any_size(size):
    c = make_case([30], [9], 8, 2, seed=15)
    sz = c["packed"][..., 2304:].contiguous().view(torch.bfloat16)
    c["packed"][..., 2304:] = (sz.float() * size).bfloat16().view(torch.uint8)
    c["v"] = (c["v"].float() * size).bfloat16()
    check(c)


def test_rows_behind_the_end_are_never_used():
    c = make_case([19, 3], [21, 7], 8, 2, seed=16)
    run(c)
    first, first_lse = c["out"].clone(), c["lse"].clone()
    used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool, device=DEV)
    for b in range(2):
        for t in range(c["recent"][b]):
            used[int(c["recent_table"][b, t // 16]), t % 16] = True
    behind = ~used[:, None].expand(-1, 2, -1)
    for x in (float("nan"), float("inf")):
        c["k"][behind] = x
        c["v"][behind] = x
        run(c)
        assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])


def test_nonfinite_tokens_reach_their_rows_alone():
    c = make_case([12, 12, 12], [20, 20, 20], 8, 2, seed=17)
    run(c)
    first = c["out"].clone()
    bad = torch.tensor([float("nan")], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    c["packed"][int(c["table"][0, 5]), 0, 2304 + 8 * 3:2304 + 8 * 3 + 2] = bad      # scale of a value's dims 0..63
    c["k"][int(c["recent_table"][1, 0]), 1, 2, 9] = float("nan")
    c["q"][2, 6] = float("nan")
    run(c)
    got, nan = c["out"].float(), torch.isnan(c["out"].float())
    assert nan[0, :4, :64].all() and not nan[0, 4:].any() and torch.equal(c["out"][0, 4:], first[0, 4:])
    assert nan[1, 4:].all() and torch.equal(c["out"][1, :4], first[1, :4])
    assert nan[2, 6].all() and torch.equal(c["out"][2, :6], first[2, :6]) and torch.equal(c["out"][2, 7], first[2, 7])
    assert torch.equal(got[0, :4, 64:], first[0, :4, 64:].float())


def test_bad_counts_and_ids():
    def fresh():
        return make_case([12, 9], [20, 5], 8, 2, seed=18, width=14)

    for name, at, value in (("seq_pages", 1, 15), ("seq_pages", 0, -1), ("recent_tokens", 0, 33),
                            ("recent_tokens", 1, -2 ** 31)):
        c = fresh()
        c[name][at] = value
        c["pages" if name == "seq_pages" else "recent"][at] = 0
        check(c, status=-6)
    for name, at, value in (("table", (0, 3), c["packed"].shape[0]), ("table", (1, 8), -1)):
        c = fresh()
        c[name][at] = value
        run(c)
        assert L.locks_get_device_status(c["ws"]) == -6
        c[name][at] = 0
        check(c, status=-6)
    c = fresh()
    c["recent_table"][0, 1] = c["k"].shape[0]
    run(c)
    assert L.locks_get_device_status(c["ws"]) == -6
    c["recent_table"][0, 1] = 0
    check(c, status=-6)
    c = make_case([12], [0], 8, 2, seed=19, selected=[[[3, 4, 5], [1, 2, 3]]])
    c["sel"][0, 0, 1] = 12                           # past the table's width: page 0
    run(c)
    assert L.locks_get_device_status(c["ws"]) == -6
    c["ws"][:256] = 0
    c["sel"][0, 0, 1] = 4
    c["n_sel"][0, 1] = 4                             # past k_cap: none
    c["lists"][0][1] = []
    check(c, status=-6)


def test_repeats_exactly_and_follows_a_captured_graph():
    c = make_case([400, 100], [20, 5], 16, 2, seed=20)
    check(c)
    first = c["out"].clone()
    for _ in range(3):
        run(c)
        assert torch.equal(first, c["out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(c)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(c)
    torch.cuda.current_stream().wait_stream(side)
    c["out"].zero_()
    graph.replay()
    assert torch.equal(first, c["out"])
    c["pages"], c["recent"] = [3, 350], [0, 30]
    c["seq_pages"].copy_(i32(c["pages"]))
    c["recent_tokens"].copy_(i32(c["recent"]))
    graph.replay()
    replayed = c["out"].clone()
    check(c)
    assert torch.equal(replayed, c["out"])


def test_two_streams_with_a_workspace_each():
    cs = [make_case([900, 30], [9, 0], 8, 2, seed=s) for s in (21, 22)]
    want = []
    for c in cs:
        check(c)
        want.append(c["out"].clone())
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cs, streams):
            run(c, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c["out"], w)


def test_a_pool_of_more_than_2_31_bytes():
    phys, hkv = 120001, 8
    packed = torch.empty((phys, hkv, 2432), dtype=torch.uint8, device=DEV)
    assert packed.numel() > 2 ** 31
    small = make_case([9], [0], 32, hkv, seed=23)
    packed[-20:] = small["packed"][0]
    ids = phys - 1 - torch.arange(9, dtype=torch.int32, device=DEV)
    packed[ids.long()] = small["packed"][small["table"][0].long()]
    run(small)
    first = small["out"].clone()
    small["packed"], small["table"] = packed, ids.view(1, 9)
    small["out"].zero_()
    run(small)
    assert torch.equal(first, small["out"])
    k, v = cache_pair(2, hkv, 3)
    dims = L.make_dims(1, hkv, hkv, 1, 2)
    L.locks_pack_pages(dims, k, v, i32([0, 1]), i32([phys - 1, phys - 7]), 2, packed)
    check_units(packed[[phys - 1, phys - 7]].cpu().numpy(), f64(k), f64(v))


def test_half_precision_of_bits_and_int16_views():
    """bf16 buffers may come as int16 bits, as elsewhere."""
    c = make_case([7], [4], 8, 2, seed=24, q_type=torch.bfloat16)
    run(c)
    first = c["out"].clone()
    bits = {n: c[n].view(torch.int16) for n in ("q", "k", "v", "out")}
    c["out"].zero_()
    L.locks_packed_attention(c["dims"], bits["q"], c["packed"], c["table"], c["seq_pages"], bits["out"], c["ws"],
                             k_cache=bits["k"], v_cache=bits["v"], recent_table=c["recent_table"],
                             recent_tokens=c["recent_tokens"])
    assert torch.equal(first, c["out"])
