"""The cache operators together, as a serving loop uses them: prompts and decode steps go
through locks_append_tokens; the step attends (locks_decode_step with tails, or
locks_prefix_attention); its scores become page mass, and locks_evict_pages keeps each
sequence within its window, its freed pages taken by the next tokens. A float64 simulation
of the cache follows on the host: it holds every token's rotated key and value by page and
is given nothing the GPU computed but the masses eviction goes by.

The attention is held to the step's own bar (2e-2; the budget keeps every page, so it is
dense attention over the tokens still in the cache)."""

import numpy as np
import pytest
import torch

import sparse_kv_page_gb300 as L
from tests import cache_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

FREQS = [10000.0 ** (-i / 64) for i in range(64)]
HQ, HKV, G = 8, 2, 4


class Sim:
    """One sequence: pages of (keys, values) [16][HKV][128], and how many tokens the last has."""

    def __init__(self):
        self.pages, self.tokens = [], 0           # tokens of the cache, not of the sequence's history

    def append(self, k, v):
        if self.tokens % 16 == 0:
            self.pages.append((np.zeros((16, HKV, 128)), np.zeros((16, HKV, 128))))
        self.pages[-1][0][self.tokens % 16] = k
        self.pages[-1][1][self.tokens % 16] = v
        self.tokens += 1

    def attend(self, q):
        k = np.concatenate([p[0] for p in self.pages])[:self.tokens]
        v = np.concatenate([p[1] for p in self.pages])[:self.tokens]
        return np.concatenate([ref.attend(q[h * G:(h + 1) * G], k[:, h], v[:, h])[0] for h in range(HKV)])


def turned(x, pos, w):
    """Normed and rotated heads of one token in float64, from the bf16 projection."""
    return ref.rotate(ref.norm(x, w, 1e-6), pos * np.array(FREQS), False, 1.0)


def test_decode_loop_with_eviction_and_recycled_pages():
    B, P, keep, sink, recent, steps = 2, 12, 6, 1, 2, 150
    rng = np.random.default_rng(3)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    phys = B * P + 1
    dims = L.make_dims(B, HQ, HKV, P, phys)
    kc = torch.full((phys, HKV, 16, 128), float("nan"), device=DEV).bfloat16()
    vc = kc.clone()
    table = torch.zeros((B, P), dtype=torch.int32, device=DEV)
    free = list(rng.permutation(phys))
    seq_pages = torch.zeros(B, dtype=torch.int32, device=DEV)
    tail = torch.zeros(B, dtype=torch.int32, device=DEV)
    mass = torch.zeros((B, P), device=DEV)
    summ = L.Summaries.empty(phys, HKV, DEV)
    qw, kw = 1 + 0.1 * torch.randn((2, 128), generator=g, device=DEV)
    rope = L.make_rope(128, FREQS)
    budget = 16 * P
    ws, mws = L.alloc_workspace(dims, budget, DEV), L.alloc_mass_workspace(dims, DEV)
    out = torch.zeros((B, HQ, 128), dtype=torch.int16, device=DEV)
    scores = torch.zeros((B, HQ, P), device=DEV)
    evicted = torch.zeros((B, P - keep), dtype=torch.int32, device=DEV)
    n_evicted = torch.zeros(B, dtype=torch.int32, device=DEV)
    sims, history = [Sim() for _ in range(B)], [0] * B

    def append(counts):
        """counts[b] new tokens of every sequence in one call; returns the queries."""
        seq = np.repeat(np.arange(B), counts)
        index, pos = [], []
        for b in range(B):
            for _ in range(counts[b]):
                at = sims[b].tokens + sum(1 for s in seq[:len(index)] if s == b)
                if at % 16 == 0:
                    table[b, at // 16] = int(free.pop())
                index.append(at)
                pos.append(history[b] + sum(1 for s in seq[:len(pos)] if s == b))
        t = len(index)
        qkv = torch.randn((t, HQ + 2 * HKV, 128), generator=g, device=DEV).mul_(1.5).bfloat16()
        q = torch.empty((t, HQ, 128), device=DEV)
        i32 = dict(dtype=torch.int32, device=DEV)
        L.locks_append_tokens(dims, rope, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:],
                              torch.tensor(pos, **i32), torch.tensor(index, **i32), table, q, kc, vc,
                              token_seq=torch.tensor(seq, **i32), q_weight=qw, k_weight=kw)
        x, w = qkv.double().cpu().numpy(), (qw.double().cpu().numpy(), kw.double().cpu().numpy())
        queries = np.zeros((t, HQ, 128))
        for i, b in enumerate(seq):
            queries[i] = turned(x[i, :HQ], pos[i], w[0])
            sims[b].append(ref.bf16(turned(x[i, HQ:HQ + HKV], pos[i], w[1])), x[i, HQ + HKV:])
            history[b] += 1
        return q, queries

    def fill():
        """Summaries of the pages that are full, off the tails."""
        ids = []
        for b in range(B):
            full = sims[b].tokens // 16
            ids += [int(table[b, j]) for j in range(int(seq_pages[b]), full)]
            seq_pages[b] = full
            tail[b] = sims[b].tokens - 16 * full
        if ids:
            L.locks_build_summaries(dims, kc, torch.tensor(ids, dtype=torch.int32, device=DEV), len(ids), summ)

    append([37, 64])                              # the prompts, one call
    fill()
    evictions = 0
    for _ in range(steps):
        q, queries = append([1, 1])
        for b in range(B):
            tail[b] = sims[b].tokens - 16 * int(seq_pages[b])
        L.locks_decode_step(dims, q, kc, vc, summ, table, seq_pages, budget, out, ws, scores=scores, tail_tokens=tail)
        L.locks_accumulate_mass(dims, scores, seq_pages, mass, mass, mws, decay=0.95)
        assert L.locks_get_device_status(ws) == 0 and L.locks_get_device_status(mws) == 0
        got = out.view(torch.bfloat16).double().cpu().numpy()
        for b in range(B):
            assert np.abs(got[b] - sims[b].attend(queries[b])).max() < 2e-2
            n = int(seq_pages[b])
            assert 0 < float(mass[b, :n].sum()) <= 20.001            # at most 1 / (1 - decay)
        fill()
        for b in range(B):
            mass[b, int(seq_pages[b]):] = 0.0     # a page starts without any
        m0, t0, n0 = mass.cpu().numpy(), table.cpu().numpy(), seq_pages.cpu().numpy()
        extra = int((tail > 0).any())             # a sequence's table row ends with its unfilled page
        L.locks_evict_pages(dims, mass, table, seq_pages, keep, mass, table, seq_pages, evicted, n_evicted,
                            sink_pages=sink, recent_pages=recent, extra_pages=extra)
        for b in range(B):
            kept_t, _, gone = ref.evict(m0[b], t0[b], int(n0[b]), keep, sink, recent, extra)
            assert int(n_evicted[b]) == len(gone) and evicted[b, :len(gone)].tolist() == gone.tolist()
            assert table[b, :len(kept_t)].tolist() == kept_t.tolist()
            where = {int(p): j for j, p in enumerate(t0[b])}
            for p in gone:                        # the freed pages are used again
                j = where[int(p)]
                sims[b].pages[j] = None
                sims[b].tokens -= 16
                free.insert(0, int(p))
                kc[int(p)] = float("nan")         # nothing may read them meanwhile
                vc[int(p)] = float("nan")
            sims[b].pages = [p for p in sims[b].pages if p is not None]
            evictions += len(gone)
    assert evictions >= 2 * (steps // 16 - 4) and max(int(n) for n in seq_pages) <= keep + 1


def test_sequences_on_a_shared_prompt():
    """One prompt in the cache once, six sequences that continue it: appended step by step and
    attended through locks_prefix_attention."""
    B, prompt, steps, own_pages = 6, 301, 35, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    pp = (prompt + 15) // 16
    phys = pp + B * own_pages + 1
    dims = L.make_dims(B, HQ, HKV, own_pages, phys)
    one = L.make_dims(1, HQ, HKV, pp, phys)       # the prompt as a sequence of its own
    kc = torch.full((phys, HKV, 16, 128), float("nan"), device=DEV).bfloat16()
    vc = kc.clone()
    perm = torch.randperm(phys, generator=g, device=DEV).int()
    prefix_table, table = perm[:pp].view(1, pp).contiguous(), perm[pp:pp + B * own_pages].view(B, own_pages).contiguous()
    rope = L.make_rope(128, FREQS)
    i32 = dict(dtype=torch.int32, device=DEV)
    sim = Sim()

    def project(t):
        qkv = torch.randn((t, HQ + 2 * HKV, 128), generator=g, device=DEV).bfloat16()
        return qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], qkv.double().cpu().numpy()

    _, k, v, x = project(prompt)                  # keys and values only
    at = torch.arange(prompt, **i32)
    L.locks_append_tokens(one, rope, None, k, v, at, at, prefix_table, None, kc, vc, token_seq=torch.zeros_like(at))
    for t in range(prompt):
        sim.append(ref.bf16(turned(x[t, HQ:HQ + HKV], t, None)), x[t, HQ + HKV:])
    sims = []
    for _ in range(B):
        s = Sim()
        s.pages, s.tokens = [(p[0].copy(), p[1].copy()) for p in sim.pages], sim.tokens
        sims.append(s)
    ws = L.alloc_prefix_workspace(dims, 1, DEV)
    tokens = torch.tensor([prompt], **i32)
    start = torch.tensor([0, B], **i32)
    own = torch.zeros(B, **i32)
    out = torch.empty((B, HQ, 128), dtype=torch.bfloat16, device=DEV)
    q_out = torch.empty((B, HQ, 128), device=DEV)
    for step in range(steps):
        q, k, v, x = project(B)
        L.locks_append_tokens(dims, rope, q, k, v, torch.full((B,), prompt + step, **i32), own, table, q_out, kc, vc)
        own += 1
        L.locks_prefix_attention(dims, q_out, kc, vc, prefix_table, tokens, start, table, own, out, ws)
        for b in range(B):
            sims[b].append(ref.bf16(turned(x[b, HQ:HQ + HKV], prompt + step, None)), x[b, HQ + HKV:])
        if step % 5 == 0 or step == steps - 1:
            got = out.double().cpu().numpy()
            for b in range(B):
                want = sims[b].attend(turned(x[b, :HQ], prompt + step, None))
                assert np.abs(got[b] - want).max() < 2e-2
    assert L.locks_get_device_status(ws) == 0
