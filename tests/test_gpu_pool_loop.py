"""The packed cache and its two pools together, as a serving loop uses them. Tokens go through
locks_append_tokens into pages of the bf16 pool (locks_take_pages); a page that fills is packed into a
page of the packed pool and handed back (locks_free_pages); beams fork in both pools; eviction's pages are
freed; both pools close up in the middle of it all; and locks_packed_attention attends to what is there,
whole or by a selection. A float64 simulation follows on the host: it holds every row's tokens, and is
given nothing the GPU computed.

Tolerances are those of the attention's own tests (2 e + 2^-11 + ... of the weights, 2^-8 of the output)."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import pool_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
B, HQ, HKV, G, P, R = 5, 8, 2, 4, 12, 3
NB, NP = 40, 90                                      # pages of the bf16 pool, of the packed pool


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


class Row:
    """One sequence on the host: packed pages (keys, values, their sizes) and recent tokens."""

    def __init__(self):
        self.pages, self.recent = [], []

    def copy(self):
        r = Row()
        r.pages, r.recent = list(self.pages), list(self.recent)
        return r

    def append(self, k, v):
        self.recent.append((k, v))

    def pack(self):
        k, v = (np.stack([t[i] for t in self.recent[:16]]) for i in (0, 1))          # [16][HKV][128]
        del self.recent[:16]
        page = []
        for x, group in ((k, 32), (v, 64)):
            code, scale, zero = ref.codes_of(x, group)
            page += [zero + scale * code, np.abs(zero) + np.abs(scale * code)]
        self.pages.append(page)

    def attend(self, q, pages=None):
        use = self.pages if pages is None else [self.pages[j] for j in pages]
        k, ks, v, vs = ([p[i] for p in use] for i in range(4))
        if self.recent:
            rk, rv = (np.stack([t[i] for t in self.recent]) for i in (0, 1))
            k, v, ks, vs = k + [rk], v + [rv], ks + [np.abs(rk)], vs + [np.abs(rv)]
        join = (lambda x, h: np.concatenate(x)[:, h] if x else np.zeros((0, 128)))
        out = [ref.attend(q[h * G:(h + 1) * G], *(join(x, h) for x in (k, v, ks, vs))) for h in range(HKV)]
        return [np.concatenate([o[i] for o in out]) for i in range(4)]


def holders(table, pages, pool):
    n = np.zeros(pool, np.int64)
    for b in range(B):
        np.add.at(n, table[b, :pages[b]], 1)
    return n


def test_serving_loop_on_two_pools():
    rng = np.random.default_rng(4)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    i32 = dict(dtype=torch.int32, device=DEV)
    recent_dims, packed_dims = L.make_dims(B, HQ, HKV, R, NB), L.make_dims(B, HQ, HKV, P, NP)
    attend_dims = L.make_dims(B, HQ, HKV, P, NB)
    kc = torch.full((NB, HKV, 16, 128), float("nan"), device=DEV).bfloat16()
    vc = kc.clone()
    packed = torch.full((NP, HKV, L.LOCKS_PACKED_BYTES), 255, dtype=torch.uint8, device=DEV)
    planes, packed_planes = L.make_planes([kc, vc]), L.make_planes([packed])
    recent, recent_b = torch.zeros((B, R), **i32), torch.zeros((B, R), **i32)
    table, table_b = torch.zeros((B, P), **i32), torch.zeros((B, P), **i32)
    recent_tokens, packed_tokens = torch.zeros(B, **i32), torch.zeros(B, **i32)
    refs, prefs = torch.zeros(NB, **i32), torch.zeros(NP, **i32)
    ws, pws = L.alloc_pool_workspace(recent_dims, DEV), L.alloc_pool_workspace(packed_dims, DEV)
    aws = L.alloc_packed_workspace(attend_dims, DEV)
    out, lse = torch.zeros((B, HQ, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((B, HQ), device=DEV)
    src, dst, n, tokens_b = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(1, **i32), torch.zeros(B, **i32)
    move_src, move_dst = (torch.zeros(NP, **i32) for _ in range(2))
    mass = torch.zeros((B, P), device=DEV)
    evicted, n_evicted = torch.zeros((B, P), **i32), torch.zeros(B, **i32)
    rows = [Row() for _ in range(B)]

    def check():
        for r, p, pool, t in ((refs, recent, NB, recent_tokens), (prefs, table, NP, packed_tokens)):
            pages = [ref.pages_of(x) for x in t.tolist()]
            assert np.array_equal(holders(p.cpu().numpy(), pages, pool), r.cpu().numpy())
        for w in (ws, pws, aws):
            assert L.locks_get_device_status(w) == 0

    def attention(step):
        q = torch.randn((B, HQ, 128), generator=g, device=DEV)
        pages = [len(r.pages) for r in rows]
        seq_pages = dev(pages)
        chosen, kw = [None] * B, {}
        if step % 3 == 2:                            # a selection, the same for both kv heads
            chosen = [sorted(rng.choice(m, size=min(m, 3), replace=False)) for m in pages]
            sel = np.zeros((B, HKV, 3), np.int32)
            for b, c in enumerate(chosen):
                sel[b, :, :len(c)] = c
            kw = dict(selected=dev(sel), n_selected=dev([[len(c)] * HKV for c in chosen]))
        L.locks_packed_attention(attend_dims, q, packed, table, seq_pages, out, aws, k_cache=kc, v_cache=vc,
                                 recent_table=recent, recent_tokens=recent_tokens, lse=lse, **kw)
        for b in range(B):
            want, want_lse, weight, size = rows[b].attend(q[b].double().cpu().numpy(), chosen[b])
            e = 2.0 ** -15 * size
            tol = weight * (2 * e + 2.0 ** -11 + 2.0 ** -18)[:, None] + 2.0 ** -8 * np.abs(want)
            assert (np.abs(out[b].double().cpu().numpy() - want) <= tol + 1e-30).all(), (step, b)
            got = lse[b].double().cpu().numpy()
            if np.isinf(want_lse).any():
                assert np.array_equal(got, want_lse), (step, b)
            else:
                assert (np.abs(got - want_lse) <= e + 2.0 ** -17).all(), (step, b)

    for step in range(70):
        # tokens of this step: pages for them, and the rows themselves
        count = rng.integers(0, 10, B) if step % 5 else np.full(B, 1)
        count = np.minimum(count, 16 * R - recent_tokens.cpu().numpy())
        old = recent_tokens.cpu().numpy()
        L.locks_take_pages(recent_dims, recent, recent_tokens, dev(old + count), refs, recent_tokens, refs, ws)
        seq = np.repeat(np.arange(B), count)
        if len(seq):
            index = np.concatenate([old[b] + np.arange(count[b]) for b in range(B)])
            kv = torch.randn((len(seq), 2 * HKV, 128), generator=g, device=DEV).bfloat16()
            L.locks_append_tokens(recent_dims, None, None, kv[:, :HKV], kv[:, HKV:], None, dev(index), recent, None, kc, vc,
                                  token_seq=dev(seq))
            host = kv.double().cpu().numpy()
            for t, b in enumerate(seq):
                rows[b].append(host[t, :HKV], host[t, HKV:])
        # a full page of each row that has one moves to the packed pool
        full = [len(r.recent) >= 16 and len(r.pages) < P for r in rows]
        pages = np.array([len(r.pages) for r in rows])
        L.locks_take_pages(packed_dims, table, packed_tokens, dev(16 * (pages + full)), prefs, packed_tokens, prefs, pws)
        where = torch.from_numpy(np.minimum(pages, P - 1)).to(DEV)
        target = torch.where(torch.tensor(full, device=DEV), table.gather(1, where[:, None])[:, 0], -1).int()
        L.locks_pack_pages(recent_dims, kc, vc, recent[:, 0].contiguous(), target, B, packed)
        L.locks_free_pages(refs, recent, dev(full), refs)
        moved = torch.roll(recent, -1, 1)
        on = torch.tensor(full, device=DEV)
        recent.copy_(torch.where(on[:, None], moved, recent))
        recent_tokens -= 16 * on.int()
        for r, f in zip(rows, full):
            if f:
                r.pack()
        check()
        attention(step)
        if step % 6 == 5:                            # beams go on from others, in both pools
            parents = rng.integers(0, B, B)
            parents[rng.integers(0, B)] = -1 if step % 12 == 5 else 0
            L.locks_fork_sequences(recent_dims, recent, recent_tokens, dev(parents), refs, recent_b, tokens_b, refs, src, dst,
                                   n, ws)
            L.locks_copy_pages(planes, src, dst, n)
            recent, recent_b = recent_b, recent
            recent_tokens.copy_(tokens_b)
            L.locks_fork_sequences(packed_dims, table, packed_tokens, dev(parents), prefs, table_b, tokens_b, prefs, src, dst,
                                   n, pws)
            assert int(n) == 0                       # full pages alone
            table, table_b = table_b, table
            packed_tokens.copy_(tokens_b)
            rows = [rows[p].copy() if p >= 0 else Row() for p in parents]
            check()
            attention(step)
        if step % 8 == 7:                            # a window of the heaviest pages
            keep = 5
            mass.copy_(torch.rand((B, P), generator=g, device=DEV))
            seq_pages = dev([len(r.pages) for r in rows])
            m = mass.cpu().numpy()
            for b, r in enumerate(rows):
                kept, _, _ = ref.cache_ref.evict(m[b], np.arange(P), len(r.pages), keep, 1, 1, 0)
                r.pages = [r.pages[j] for j in kept[:min(len(r.pages), keep)]]
            L.locks_evict_pages(packed_dims, mass, table, seq_pages, keep, mass, table, seq_pages, evicted, n_evicted,
                                sink_pages=1, recent_pages=1)
            L.locks_free_pages(prefs, evicted, n_evicted, prefs)
            packed_tokens.copy_(16 * seq_pages)
            check()
            attention(step)
        if step % 10 == 9:                           # both pools close up
            for d, t, k, r, p, w in ((recent_dims, recent, recent_tokens, refs, planes, ws),
                                     (packed_dims, table, packed_tokens, prefs, packed_planes, pws)):
                new = torch.zeros(d.num_phys_pages, **i32)
                L.locks_compact_pages(d, t, k, r, t, r, move_src, move_dst, n, new, w)
                L.locks_copy_pages(p, move_src, move_dst, n)
                used = int((r > 0).sum())
                assert int((r[:used] > 0).sum()) == used
            check()
            attention(step)
    assert max(len(r.pages) for r in rows) > 0


def test_step_of_the_scorer_on_packed_pages():
    """The decode step's own selection over summaries of packed pages, and attention over what it chose:
    summaries are built from bf16 pages and go by the packed page's id."""
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    seqs, pages, budget = 3, 90, 320
    phys = seqs * pages
    kc, vc = (torch.randn((phys, HKV, 16, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
    dims = L.make_dims(seqs, HQ, HKV, pages, phys)
    ids = torch.arange(phys, dtype=torch.int32, device=DEV)
    summ = L.Summaries.empty(phys, HKV, DEV)
    L.locks_build_summaries(dims, kc, ids, phys, summ)
    packed = torch.zeros((phys, HKV, L.LOCKS_PACKED_BYTES), dtype=torch.uint8, device=DEV)
    L.locks_pack_pages(dims, kc, vc, ids, None, phys, packed)
    table = torch.randperm(phys, generator=g, device=DEV).int().view(seqs, pages).contiguous()
    seq_pages = dev([90, 11, 47])
    q = 2 * torch.randn((seqs, HQ, 128), generator=g, device=DEV)
    out, again = (torch.zeros((seqs, HQ, 128), dtype=torch.int16, device=DEV) for _ in range(2))
    cap = L.locks_k_cap(dims, budget)
    sel, n_sel = torch.zeros((seqs, HKV, cap), dtype=torch.int32, device=DEV), torch.zeros((seqs, HKV), dtype=torch.int32,
                                                                                          device=DEV)
    ws = L.alloc_workspace(dims, budget, DEV)
    L.locks_decode_step(dims, q, kc, vc, summ, table, seq_pages, budget, out, ws, selected=sel, n_selected=n_sel)
    aws = L.alloc_packed_workspace(dims, DEV)
    L.locks_packed_attention(dims, q, packed, table, seq_pages, again, aws, selected=sel, n_selected=n_sel)
    ko, vo = torch.zeros_like(kc), torch.zeros_like(vc)
    L.locks_unpack_pages(dims, packed, ids, None, phys, ko, vo)
    exact = torch.zeros_like(out)
    L.locks_sparse_attention(dims, q, ko, vo, table, sel, n_sel, cap, exact, workspace=ws)
    assert L.locks_get_device_status(ws) == 0 and L.locks_get_device_status(aws) == 0
    # unpacked pages are rounded to bf16 once more: 2^-8 of a key moves a score by 2^-8 |q||k| / sqrt(128) at most
    a, b = (x.view(torch.bfloat16).double() for x in (again, exact))
    assert float((a - b).abs().max()) < 2e-2
