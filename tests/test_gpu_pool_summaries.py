"""GPU test of the way from bf16 pages to summaries at the packed pages' ids, with pools of different sizes:
built in the part of the arrays behind the packed pool's pages, copied to the front, scored and selected."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

HQ, HKV = 16, 4


def parts(s):
    return [s.mu, s.basis, s.coef, s.scales]


def test_summaries_at_the_ids_of_packed_pages():
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    rng = np.random.default_rng(4)
    num_packed, num_bf16, seqs, pages, budget = 130, 7, 3, 40, 160
    dims, packed_dims = L.make_dims(1, HQ, HKV, 1, num_bf16), L.make_dims(seqs, HQ, HKV, pages, num_packed)
    summ = L.Summaries.empty(num_packed + num_bf16, HKV, DEV)
    for x in parts(summ):
        x.fill_(77)
    front, tail = (L.Summaries(*(x[part] for x in parts(summ))) for part in (slice(0, num_packed), slice(num_packed, None)))
    planes = L.make_planes(parts(summ))
    packed = torch.zeros((num_packed, HKV, L.LOCKS_PACKED_BYTES), dtype=torch.uint8, device=DEV)
    k, v = (torch.zeros((num_bf16, HKV, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    # the same pages in a pool of their own, at the packed pages' ids
    all_k, all_v = (torch.randn((num_packed, HKV, 16, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
    order = rng.permutation(num_packed)[:seqs * pages]
    left = [int(x) for x in order]
    while left:                                      # pages fill, a few at a time
        n = min(len(left), int(rng.integers(1, num_bf16 + 1)))
        to, left = left[:n], left[n:]
        filled = torch.from_numpy(rng.permutation(num_bf16)[:n].astype(np.int32)).to(DEV)
        ids = torch.tensor(to, dtype=torch.int32, device=DEV)
        k[filled.long()], v[filled.long()] = all_k[ids.long()], all_v[ids.long()]
        L.locks_build_summaries(dims, k, filled, n, tail)
        L.locks_copy_pages(planes, filled + num_packed, ids)
        L.locks_pack_pages(dims, k, v, filled, ids, n, packed)
    want = L.Summaries.empty(num_packed, HKV, DEV)
    used = torch.from_numpy(np.sort(order).astype(np.int32)).to(DEV)
    L.locks_build_summaries(packed_dims, all_k, used, len(used), want)
    for x, y in zip(parts(front), parts(want)):
        assert torch.equal(x[used.long()], y[used.long()])
    rest = np.setdiff1d(np.arange(num_packed), order)
    assert len(rest) and all((x[rest] == 77).all() for x in parts(front))
    direct = torch.zeros_like(packed)
    L.locks_pack_pages(packed_dims, all_k, all_v, used, None, len(used), direct)
    assert torch.equal(direct, packed)
    table = torch.from_numpy(order.astype(np.int32)).to(DEV).view(seqs, pages).contiguous()
    seq_pages = torch.tensor([40, 0, 23], dtype=torch.int32, device=DEV)
    q = 2 * torch.randn((seqs, HQ, 128), generator=g, device=DEV)
    cap, got = L.locks_k_cap(packed_dims, budget), []
    for s in (front, want):
        ws = L.alloc_workspace(packed_dims, budget, DEV)
        scores = torch.zeros((seqs, HQ, pages), device=DEV)
        sel, n_sel = (torch.zeros(x, dtype=torch.int32, device=DEV) for x in ((seqs, HKV, cap), (seqs, HKV)))
        L.locks_score_pages(packed_dims, q, s, table, seq_pages, scores, workspace=ws)
        L.locks_select_pages(packed_dims, scores, seq_pages, budget, sel, n_sel, workspace=ws)
        out = torch.zeros((seqs, HQ, 128), dtype=torch.bfloat16, device=DEV)
        pws = L.alloc_packed_workspace(packed_dims, DEV)
        L.locks_packed_attention(packed_dims, q, packed, table, seq_pages, out, pws, selected=sel, n_selected=n_sel)
        assert L.locks_get_device_status(ws) == 0 == L.locks_get_device_status(pws)
        got.append((scores, sel, n_sel, out))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert got[0][2].tolist() == [[10] * HKV, [0] * HKV, [10] * HKV] and float(got[0][3].abs().max()) > 0
