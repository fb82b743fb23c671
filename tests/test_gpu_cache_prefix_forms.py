"""The shared-prefix attention's two forms on a GB300: one launch for short lists of few
sequences, tiles for the rest. Which one a call takes follows its tables' widths, so every
case of the first runs on the second too, through tables that are wider than their lists.
Tolerances are test_gpu_cache's: both forms round queries, weights and outputs alike."""
import numpy as np
import pytest
import torch

from tests import test_gpu_cache as T

pytestmark = pytest.mark.gpu

L = T.L
WIDE = 300


def wide(c):
    """The same case with tables of WIDE columns: behind the lists there is no page."""
    c = dict(c)
    for name in ("prefix_table", "page_table"):
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
    ([(1, 4000)], [95], 16, 1),                                 # 256 pages
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
    for groups, own, hkv in (([(1, 1)] * 33, [0] * 33, 1),        # groups
                             ([(1, 4065)], [17], 1),              # 257 pages
                             ([], [16] * 39, 1)):                 # clusters
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
