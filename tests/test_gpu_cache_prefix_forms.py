"""The shared-prefix attention's forms on a GB300: one launch of clusters for few sequences; one
of single CTAs for short lists; tiles for the prefixes and pages for few own tokens; tiles for
everything. Which one a call takes follows its tables' widths, so cases of the first run on the
others too, through tables that are wider than their lists. Tolerances are test_gpu_cache's: all forms round queries,
weights and outputs alike."""
import numpy as np
import pytest
import torch

from tests import test_gpu_cache as T

pytestmark = pytest.mark.gpu

L = T.L
WIDE = 520


def wide(c, names=("prefix_table", "page_table")):
    """The same case with tables of WIDE columns: behind the lists there is no page."""
    c = dict(c)
    for name in names:
        t = c[name]
        if t.shape[1] < WIDE:
            c[name] = torch.nn.functional.pad(t, (0, WIDE - t.shape[1]), value=-1).contiguous()
    d = c["dims"]
    c["dims"] = L.make_dims(d.batch, d.num_q_heads, d.num_kv_heads, c["page_table"].shape[1], d.num_phys_pages)
    for name in ("out", "lse", "ws"):
        c[name] = c[name].clone()
    return c


def scratch_untouched(c):
    """The form of one launch leaves the workspace behind its status alone."""
    return bool((c["ws"][256:] == 255).all())


CASES = [
    # groups, own tokens, hq, hkv
    ([(2, 333)], [45, 3], 32, 8),
    ([(1, 16)], [0], 1, 1),
    ([], [1], 8, 8),
    ([(3, 777)], [33, 0, 150], 32, 8),
    ([(1, 777)], [33], 128, 8),
    ([(2, 500), (0, 60), (1, 0), (4, 1025), (1, 7)], [0, 1, 200, 16, 0, 31, 128, 500, 9, 0, 77, 0], 20, 2),
    ([(2, 2049)], [495, 496], 32, 2),                           # 160 pages
    ([(1, 8064)], [128], 16, 1),                                # 512 pages, eight warps a CTA
    ([(14, 3000)], [i * 9 for i in range(14)], 8, 1),           # as many clusters as do so
    ([(19, 8064)], [i * 5 for i in range(19)], 5, 1),           # 512 pages, four
    ([(20, 6000)], [140] * 20, 16, 1),                          # 384 pages
    ([], [511, 512, 513], 16, 4),                               # a page for each warp, one less, one more
    ([(1, 9 * i) for i in range(30)], [i % 19 for i in range(32)], 4, 1),
    ([(1, 40)] * 32, [5] * 33, 5, 1),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_both_forms(case, q_type):
    groups, own, hq, hkv = CASES[case]
    c = T.prefix_case(groups, own, hq, hkv, seed=40 + case, q_type=q_type)
    w = wide(c)
    T.check_prefix(c)
    assert scratch_untouched(c)
    T.check_prefix(w)
    assert not scratch_untouched(w)


def test_calls_past_the_limits_take_tiles():
    for groups, own, hkv in (([(1, 1)] * 33, [0] * 33, 1),        # groups (and own tokens by pages)
                             ([(1, 8065)], [128], 1),             # 513 pages
                             ([(39, 1600)], [16] * 39, 1)):       # clusters
        c = T.prefix_case(groups, own, 4 * hkv, hkv, seed=60)
        T.check_prefix(c)
        assert not scratch_untouched(c)


def test_lists_without_tokens():
    for c in (T.prefix_case([(2, 0)], [0, 0], 8, 2, seed=1, spare=1), T.prefix_case([], [0, 0, 0], 8, 2, seed=1),
              T.prefix_case([(1, 0), (1, 20)], [0, 0, 3], 8, 2, seed=1)):
        T.check_prefix(c)
        assert scratch_untouched(c)


@pytest.fixture
def tiles(monkeypatch):
    case = T.prefix_case
    monkeypatch.setattr(T, "prefix_case", lambda *a, **k: wide(case(*a, **k)))


SMALL = [T.test_prefix_groups_and_sequences_outside_them, T.test_prefix_rows_behind_the_end_are_never_used,
         T.test_prefix_steep_and_growing_scores, T.test_prefix_nonfinite_values_stay_in_their_rows,
         T.test_prefix_bad_lengths_bounds_and_pages, T.test_prefix_agrees_with_attention_over_all_pages,
         T.test_prefix_in_a_graph_follows_its_lengths_and_two_calls_overlap,
         T.test_prefix_without_any_tokens_or_groups]


@pytest.mark.parametrize("test", SMALL, ids=lambda f: f.__name__[12:])
def test_tiles_at_small_sizes(test, tiles):
    test()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (32, 8), (32, 2), (20, 4), (16, 1), (128, 8)])
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_tiles_head_layouts(hq, hkv, q_type, tiles):
    T.test_prefix_head_layouts(hq, hkv, q_type)


@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seqs", [32, 33, 70])
def test_tiles_row_blocks(seqs, q_type, tiles):
    T.test_prefix_row_blocks(seqs, q_type)


@pytest.mark.parametrize("test", [T.test_prefix_many_sequences_many_groups, T.test_prefix_thousands_of_sequences],
                         ids=lambda f: f.__name__[12:])
def test_tiles_many(test, tiles):
    test()


@pytest.mark.parametrize("prefix", [1, 16, 100, 127, 128, 129, 256, 300, 2049])
def test_tiles_lengths(prefix, tiles):
    T.test_prefix_lengths(prefix)


def test_one_launch_in_a_graph_follows_its_lengths_and_two_calls_overlap():
    c = T.prefix_case([(2, 400), (1, 900)], [10, 200, 0, 3], 16, 4, seed=13, spare=2)
    d = T.prefix_case([(2, 300)], [50] * 2, 32, 8, seed=14)
    T.run_prefix(c), T.run_prefix(d)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        T.run_prefix(c)
    for step in range(3):
        c["seq_tokens"] += 1
        c["prefix_tokens"] -= 7
        c["group_start"][1] = 2 - step % 2
        want = T.prefix_ref(c)[0]
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            T.run_prefix(d)
        torch.cuda.synchronize()
        assert np.abs(T.f64(c["out"]) - want).max() < 2e-2
    T.check_prefix(d)
    assert scratch_untouched(c) and scratch_untouched(d)


# ------------------------------------------------ own tokens by pages, behind the tiles

@pytest.fixture
def own_pages(monkeypatch):
    """Cases of 32 / 8 heads whose prefix table alone is wide."""
    case = T.prefix_case
    monkeypatch.setattr(T, "prefix_case",
                        lambda groups, own, hq, hkv, **k: wide(case(groups, own, 32, 8, **k), ("prefix_table",)))


OWN = [T.test_prefix_groups_and_sequences_outside_them, T.test_prefix_steep_and_growing_scores,
       T.test_prefix_nonfinite_values_stay_in_their_rows, T.test_prefix_bad_lengths_bounds_and_pages,
       T.test_prefix_in_a_graph_follows_its_lengths_and_two_calls_overlap]


@pytest.mark.parametrize("test", OWN, ids=lambda f: f.__name__[12:])
def test_own_pages_at_small_sizes(test, own_pages):
    test()


OWN_CASES = [
    # groups, own tokens, hq, hkv
    ([(2, 333)], [45, 3], 32, 8),                                # eight warps a CTA or four, by the width
    ([(2, 333)], [1024, 1009], 32, 8),
    ([(5, 7000), (0, 3), (30, 50)], [(i * 97) % 1025 for i in range(38)], 32, 8),
    ([(20, 200), (19, 0)], [i % 18 for i in range(45)], 64, 8),  # more than two CTAs an SM
    ([(20, 600)], [(i * 7) % 300 for i in range(20)], 8, 8),
    ([(60, 100)], [(i * 5) % 200 for i in range(61)], 20, 4),
    ([(100, 40), (99, 900)], [(i * 3) % 70 for i in range(200)], 7, 1),
    ([], [(i * 131) % 1025 for i in range(41)], 32, 8),          # no groups: no launch ahead
    ([], [16, 0, 64, 63, 65] * 9, 4, 4),
]


@pytest.mark.parametrize("case", range(len(OWN_CASES)))
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_own_pages(case, q_type):
    groups, own, hq, hkv = OWN_CASES[case]
    c = T.prefix_case(groups, own, hq, hkv, seed=80 + case, q_type=q_type)
    T.check_prefix(wide(c, ("prefix_table",)))
    if groups:
        T.check_prefix(c)


@pytest.mark.parametrize("groups", [[(2, 261), (38, 5)], []])
def test_own_pages_rows_behind_the_end_are_never_used(groups):
    own = [19, 0, 130, 16, 1] * 8
    c = T.prefix_case(groups, own, 32, 8, seed=7, spare=2)
    used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool, device=T.DEV)
    for tab, n in list(zip(c["prefix_table"], [n for _, n in groups])) + list(zip(c["page_table"], own)):
        for t in range(n):
            used[int(tab[t // 16]), t % 16] = True
    behind = ~used[:, None, :].expand(-1, 8, -1)
    clean = {n: c[n].clone() for n in ("k", "v")}
    T.run_prefix(c)
    first, first_lse = c["out"].clone(), c["lse"].clone()
    for kk, vv in ((float("nan"), float("nan")), (float("inf"), -float("inf"))):
        c["k"], c["v"] = clean["k"].clone(), clean["v"].clone()
        c["k"][behind] = kk
        c["v"][behind] = vv
        T.run_prefix(c)
        assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])


@pytest.mark.parametrize("groups", [[(30, 300), (10, 90)], []])
def test_tokens_appended_ahead_are_seen(groups):
    """Append and attention back to back, in a captured graph: own tokens are read ahead of the
    prefix launch's end, but not ahead of what came before it."""
    own = [(i * 11) % 60 for i in range(40)]
    c = T.prefix_case(groups, own, 32, 8, seed=21, spare=1)
    d = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    kv = torch.zeros((40, 16, 128), device=T.DEV).bfloat16()
    index = torch.zeros(40, dtype=torch.int32, device=T.DEV)

    def step(c, wait):
        for i in range(4):                        # four layers' worth, all in one cache
            L.locks_append_tokens(c["dims"], None, None, kv[:, :8], kv[:, 8:], None, index, c["page_table"], None, c["k"],
                                  c["v"])
            wait()
            T.run_prefix(c)
            wait()

    step(c, torch.cuda.synchronize)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, lambda: None)
    for t in range(6):
        kv.copy_(torch.randn(kv.shape, generator=T.gen(t), device=T.DEV))
        for x in (c, d):
            if t == 0:
                x["k"].copy_(d["k"]), x["v"].copy_(d["v"])
            index.copy_(x["seq_tokens"])
            x["seq_tokens"] += 1
            torch.cuda.synchronize()
            if x is c:
                graph.replay()
            else:
                step(d, torch.cuda.synchronize)
            torch.cuda.synchronize()
        assert torch.equal(c["out"], d["out"]) and torch.equal(c["lse"], d["lse"])
    T.check_prefix(c)


# ------------------------------------------------ whole lists by pages, a CTA a kv head

LIST_CASES = [
    # groups, own tokens, hq, hkv
    ([(1, 1)], [0], 1, 1),
    ([(2, 33)], [45, 3], 32, 8),                                 # 6 pages, few sequences
    ([(7, 200), (0, 90), (8, 16)], [i % 48 for i in range(17)], 8, 8),      # 16 pages
    ([(5, 1536), (3, 1)], [512] * 10, 64, 8),                    # 128 pages, eight warps a CTA
    ([(10, 700), (20, 768)], [i * 7 for i in range(40)], 32, 8),  # four, three a CTA in flight
    ([(90, 160), (0, 3), (160, 90)], [i % 60 for i in range(256)], 28, 4),  # several waves of CTAs
    ([(40, 380)], [i * 8 for i in range(48)], 32, 2),            # sixteen queries
    ([(3, 30)] * 32, [i % 90 for i in range(100)], 8, 1),        # as many groups as there may be
    ([], [(i * 50) % 2049 for i in range(60)], 16, 8),
]


@pytest.mark.parametrize("case", range(len(LIST_CASES)))
@pytest.mark.parametrize("q_type", [torch.float32, torch.bfloat16])
def test_lists_by_pages(case, q_type):
    groups, own, hq, hkv = LIST_CASES[case]
    c = T.prefix_case(groups, own, hq, hkv, seed=120 + case, q_type=q_type)
    T.check_prefix(c)
    assert scratch_untouched(c)


@pytest.fixture
def many(monkeypatch):
    """Cases of 32 / 8 heads with 40 more sequences, of no group and of one page at most."""
    case = T.prefix_case
    monkeypatch.setattr(T, "prefix_case",
                        lambda groups, own, hq, hkv, **k: case(groups, list(own) + [i % 17 for i in range(40)], 32, 8, **k))


@pytest.mark.parametrize("test", [T.test_prefix_groups_and_sequences_outside_them,
                                  T.test_prefix_nonfinite_values_stay_in_their_rows,
                                  T.test_prefix_in_a_graph_follows_its_lengths_and_two_calls_overlap],
                         ids=lambda f: f.__name__[12:])
def test_lists_by_pages_at_small_sizes(test, many):
    test()


def test_lists_by_pages_bad_lengths_bounds_and_pages():
    c = T.prefix_case([(20, 100), (20, 60)], [i % 30 for i in range(40)], 32, 8, seed=9)
    for name, at, value, as_if in (("seq_tokens", 1, 16 * c["dims"].max_pages_per_seq + 1, 0),
                                   ("seq_tokens", 0, -1, 0), ("prefix_tokens", 0, -5, 0),
                                   ("prefix_tokens", 1, 1 << 30, 0), ("group_start", 2, 41, 20),
                                   ("page_table", (3, 0), -3, 0),
                                   ("prefix_table", (1, 2), c["dims"].num_phys_pages, 0)):
        kept = c[name].clone()
        c[name][at] = value
        c["ws"][:256] = 0
        T.run_prefix(c)
        assert L.locks_get_device_status(c["ws"]) == -6, name
        got, got_lse = c["out"].clone(), c["lse"].clone()
        c[name][at] = as_if
        c["ws"][:256] = 0
        T.check_prefix(c)
        assert torch.equal(got, c["out"]) and torch.equal(got_lse, c["lse"]), name
        c[name].copy_(kept)
    assert scratch_untouched(c)


def test_lists_by_pages_rows_behind_the_end_are_never_used():
    groups, own = [(2, 261), (30, 5)], [19, 0, 30, 16, 1] * 8
    c = T.prefix_case(groups, own, 32, 8, seed=7, spare=2)
    used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool, device=T.DEV)
    for tab, n in list(zip(c["prefix_table"], [n for _, n in groups])) + list(zip(c["page_table"], own)):
        for t in range(n):
            used[int(tab[t // 16]), t % 16] = True
    behind = ~used[:, None, :].expand(-1, 8, -1)
    T.run_prefix(c)
    first, first_lse = c["out"].clone(), c["lse"].clone()
    assert scratch_untouched(c)
    c["k"][behind] = float("nan")
    c["v"][behind] = float("-inf")
    T.run_prefix(c)
    assert torch.equal(first, c["out"]) and torch.equal(first_lse, c["lse"])
