"""Cases that measure the cache operators around the decode step: filling the paged
K/V cache (head norms and rotary positions on the way), attention of a batch that shares
a prefix, the attention mass kept per page, and eviction by that mass.

``run`` computes an operator either in its plain form (elementary torch operations in 32
bits, angles in 64) or, where ``own`` is true, through this repository's library. Head
dim 128, pages of 16 tokens and the 32/8 and 32/2 head layouts are those of the
workloads in ``synth``; context lengths run from one token to the 1M tokens of the
longest one.

Arrays: k_cache / v_cache bf16 bits [pages][kv heads][16][128], page_table int32
[sequences][pages], q fp32 or bf16 [sequences][heads][128].
"""

import math

import numpy as np
import torch

own = False

D = 128
PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence decoding at 1M tokens of context: 32/8 heads, whole heads rotated in
        # halves; nothing but latency
        dict(name="append_decode_1", op="append", tokens=1, seqs=1, hq=32, hkv=8, itype="bf16", qtype="fp32", rot=128,
             inter=False, axes=1, norm=False, start=1048575, pad=0),
        # a decode batch of 256 rows, eight of them padding, 32/2 heads, the first half of
        # each head rotated in interleaved pairs
        dict(name="append_decode_256", op="append", tokens=256, seqs=248, hq=32, hkv=2, itype="bf16", qtype="fp32",
             rot=64, inter=True, axes=1, norm=False, start=8191, pad=8),
        # a 64K-token prompt chunk of two sequences, head norms and halves
        dict(name="append_prefill_64k", op="append", tokens=65536, seqs=2, hq=32, hkv=8, itype="bf16", qtype="bf16",
             rot=128, inter=False, axes=1, norm=True, start=0, pad=0),
        # an odd prompt of text and images from fp32 activations: three position axes
        dict(name="append_axes_10007", op="append", tokens=10007, seqs=3, hq=32, hkv=8, itype="fp32", qtype="fp32",
             rot=128, inter=False, axes=3, norm=True, start=77, pad=0),
        # two short chats on a 333-token system prompt: latency
        dict(name="prefix_small", op="prefix", groups=1, seqs=2, hq=32, hkv=8, prefix=333, own_max=45, qtype="fp32"),
        # 16 questions about one 128K-token document: the cache's bytes bound it
        dict(name="prefix_128k_16", op="prefix", groups=1, seqs=16, hq=32, hkv=8, prefix=131072, own_max=1024,
             qtype="fp32"),
        # 128 samples in four groups of one 24K-token prompt each, bf16 queries: products bound it
        dict(name="prefix_24k_4x32", op="prefix", groups=4, seqs=128, hq=32, hkv=8, prefix=24576, own_max=700,
             qtype="bf16"),
        # eight readers of one 1M-token context, 32/2 heads (sixteen queries to a kv head)
        dict(name="prefix_1m_8", op="prefix", groups=1, seqs=8, hq=32, hkv=2, prefix=1048570, own_max=200,
             qtype="fp32"),
        # mass of one 128K-token sequence; of four 1M-token sequences
        dict(name="mass_128k_1", op="mass", seqs=1, hq=32, pages=8192, decay=1.0),
        dict(name="mass_1m_4", op="mass", seqs=4, hq=32, pages=65536, decay=0.98),
        # a few pages out of 4K-token windows; a tenth out of four 1M-token sequences
        dict(name="evict_window_8", op="evict", seqs=8, pages=261, keep=256, sink=1, recent=4, extra=1),
        dict(name="evict_1m_4", op="evict", seqs=4, pages=65536, keep=58982, sink=4, recent=128, extra=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "prefix", "prefix", "mass", "evict"))
    hq, hkv = rng.choice(((32, 8), (32, 8), (32, 2), (16, 8), (8, 1), (20, 4)))
    if op == "append":
        tokens = _log_int(rng, 1, 50000)
        pad = rng.choice((0, 0, min(tokens - 1, rng.randint(0, 9))))
        return dict(op=op, tokens=tokens, seqs=_log_int(rng, 1, min(256, tokens - pad)), hq=hq, hkv=hkv,
                    itype=rng.choice(("bf16", "bf16", "fp16", "fp32")), qtype=rng.choice(("fp32", "fp32", "bf16")),
                    rot=rng.choice((128, 128, 96, 64, 32)), inter=rng.random() < 0.4, axes=rng.choice((1, 1, 2, 3)),
                    norm=rng.random() < 0.5, start=_log_int(rng, 1, 20000) - 1, pad=pad)
    if op == "prefix":
        seqs = _log_int(rng, 1, 96)
        groups = rng.randint(1, min(4, seqs))
        # keys times queries stay below the largest listed case
        prefix = _log_int(rng, 1, min(200000, 250000000 // (seqs * hq * 4) // groups * 2))
        return dict(op=op, groups=groups, seqs=seqs, hq=hq, hkv=hkv, prefix=prefix,
                    own_max=_log_int(rng, 1, min(6000, 200000 // seqs)), qtype=rng.choice(("fp32", "bf16")))
    if op == "mass":
        seqs = _log_int(rng, 1, 16)
        return dict(op=op, seqs=seqs, hq=hq, pages=_log_int(rng, 1, 200000 // seqs),
                    decay=rng.choice((1.0, 0.5, round(rng.uniform(0.8, 1.0), 3))))
    seqs = _log_int(rng, 1, 64)
    pages = _log_int(rng, 2, min(65536, 260000 // seqs))
    keep = rng.randint(1, pages)
    sink = rng.randint(0, min(4, keep))
    return dict(op=op, seqs=seqs, pages=pages, keep=keep, sink=sink, recent=rng.randint(0, min(64, keep - sink)),
                extra=rng.randint(0, 4))


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _inv_freq(case):
    n = case["rot"] // 2
    return [500000.0 ** (-i / n) for i in range(n)]


def _axis(case):
    # the axes' pairs lie in blocks: the first for time, the others for height and width
    n, a = case["rot"] // 2, case["axes"]
    return [min(i * a // n, a - 1) for i in range(n)]


def _prepare_append(case, g, dev):
    T, S, hq, hkv = case["tokens"], case["seqs"], case["hq"], case["hkv"]
    live = T - case["pad"]
    it = TYPES[case["itype"]]
    i = torch.arange(live, device=dev)
    seq = i * S // live
    first = torch.searchsorted(seq, torch.arange(S, device=dev))
    index = torch.full((T,), -1, dtype=torch.int32, device=dev)
    index[:live] = (case["start"] + i - first[seq]).int()
    token_seq = torch.zeros(T, dtype=torch.int32, device=dev)
    token_seq[:live] = seq.int()
    longest = -(-live // S) + 1
    pages = (case["start"] + longest + PAGE - 1) // PAGE
    first_page = case["start"] // PAGE        # the pages before the tokens' are never touched: all share page 0
    used = pages - first_page
    phys = 1 + S * used
    table = torch.zeros((S, pages), dtype=torch.int32, device=dev)
    table[:, first_page:] = 1 + torch.randperm(S * used, generator=g, device=dev).view(S, used).int()
    pos = torch.zeros((case["axes"], T), dtype=torch.int32, device=dev)
    pos[0] = index.clamp(min=0)
    for a in range(1, case["axes"]):          # rows and columns of image patches
        pos[a] = torch.randint(0, 4096, (T,), generator=g, device=dev, dtype=torch.int32)
    # one projection's output: the queries, keys and values of a token lie beside each other
    qkv = torch.randn((T, hq + 2 * hkv, D), generator=g, device=dev).mul_(1.7).to(it)
    s = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], positions=pos, cache_index=index,
             token_seq=token_seq, page_table=table, eps=1e-6,
             inv_freq=torch.tensor(_inv_freq(case), dtype=torch.float64, device=dev),
             axis=torch.tensor(_axis(case), device=dev),
             q_out=torch.zeros((T, hq, D), dtype=TYPES[case["qtype"]], device=dev),
             k_cache=torch.randn((phys, hkv, PAGE, D), generator=g, device=dev).to(torch.bfloat16),
             v_cache=torch.randn((phys, hkv, PAGE, D), generator=g, device=dev).to(torch.bfloat16),
             q_weight=None, k_weight=None)
    if case["norm"]:
        s["q_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
        s["k_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
    if own:                                   # the sizes and the rotation that a program keeps
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(S, hq, hkv, pages, phys)
        s["rope"] = L.make_rope(case["rot"], _inv_freq(case), interleaved=case["inter"], axis=_axis(case))
    return s


def _prepare_prefix(case, g, dev):
    B, hq, hkv, G = case["seqs"], case["hq"], case["hkv"], case["groups"]
    # prefixes of different lengths, the first of the full length; each group a run of sequences
    share = torch.rand(G, generator=g, device=dev) * 0.3 + 0.7
    share[0] = 1
    ptok = (case["prefix"] * share).int().clamp(min=1)
    start = (torch.arange(G + 1, device=dev) * B // G).int()
    pp = (case["prefix"] + PAGE - 1) // PAGE
    mp = (case["own_max"] + PAGE - 1) // PAGE
    phys = G * pp + B * mp
    perm = torch.randperm(phys, generator=g, device=dev).int()
    # attention with some weight on the first tokens and on a few keys along the query's direction
    k = torch.randn((phys, hkv, PAGE, D), generator=g, device=dev)
    k += 0.3 * torch.randn((1, hkv, 1, D), generator=g, device=dev)
    s = dict(case=case, q=1.5 * torch.randn((B, hq, D), generator=g, device=dev), k_cache=k.to(torch.bfloat16),
             v_cache=torch.randn((phys, hkv, PAGE, D), generator=g, device=dev).to(torch.bfloat16),
             prefix_table=perm[:G * pp].view(G, pp).contiguous(), prefix_tokens=ptok, group_start=start,
             page_table=perm[G * pp:].view(B, mp).contiguous(),
             seq_tokens=torch.randint(0, case["own_max"] + 1, (B,), generator=g, device=dev, dtype=torch.int32),
             out=torch.zeros((B, hq, D), dtype=torch.bfloat16, device=dev), lse=torch.zeros((B, hq), device=dev))
    s["q"] = s["q"].to(TYPES[case["qtype"]])
    if own:                                   # the sizes and the workspace that a program keeps
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, hq, hkv, mp, phys)
        s["ws"] = L.alloc_prefix_workspace(s["dims"], G)
    return s


def _prepare_mass(case, g, dev):
    B, hq, P = case["seqs"], case["hq"], case["pages"]
    scores = 1.5 * torch.randn((B, hq, P), generator=g, device=dev) + 3
    seq = torch.randint(max(1, P - 64), P + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    s = dict(case=case, scores=scores, seq_pages=seq, mass=torch.rand((B, P), generator=g, device=dev) / P,
             mass_out=torch.zeros((B, P), device=dev))
    if own:
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, hq, 1 if hq <= 16 else 2, P, B * P)
        s["ws"] = L.alloc_mass_workspace(s["dims"])
    return s


def _prepare_evict(case, g, dev):
    B, P, extra = case["seqs"], case["pages"], case["extra"]
    width = P + extra
    # accumulated masses span decades; a quarter of the pages never drew any and tie at zero
    mass = torch.exp(3 * torch.randn((B, width), generator=g, device=dev)) / P
    mass = torch.where(torch.rand((B, width), generator=g, device=dev) < 0.25, torch.zeros_like(mass), mass)
    seq = torch.randint(max(0, P - 9), P + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    s = dict(case=case, mass=mass, seq_pages=seq,
             page_table=torch.randperm(B * width, generator=g, device=dev).view(B, width).int(),
             mass_out=torch.full((B, width), -1.0, device=dev),
             table_out=torch.full((B, width), -1, dtype=torch.int32, device=dev),
             seq_out=torch.zeros(B, dtype=torch.int32, device=dev),
             evicted=torch.full((B, max(1, width - case["keep"])), -1, dtype=torch.int32, device=dev),
             n_evicted=torch.zeros(B, dtype=torch.int32, device=dev))
    if own:
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, 1, 1, width, B * width)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed)
    return {"append": _prepare_append, "prefix": _prepare_prefix, "mass": _prepare_mass,
            "evict": _prepare_evict}[case["op"]](case, g, dev)


# ------------------------------------------------------------------- runs

def _rotate(x, cos, sin, rot, inter):
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _normed(x, weight, eps):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight


def _append(s):
    case = s["case"]
    live, rot, inter = case["tokens"] - case["pad"], case["rot"], case["inter"]
    angle = s["positions"][:, :live][s["axis"]].T.double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"][:live] = _rotate(_normed(s["q"][:live], s["q_weight"], s["eps"]), cos, sin, rot, inter)
    k = _rotate(_normed(s["k"][:live], s["k_weight"], s["eps"]), cos, sin, rot, inter)
    index = s["cache_index"][:live].long()
    page = s["page_table"][s["token_seq"][:live].long(), index // PAGE].long()
    s["k_cache"][page, :, index % PAGE] = k.to(torch.bfloat16)
    s["v_cache"][page, :, index % PAGE] = s["v"][:live].to(torch.bfloat16)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _weights(logits):
    """exp(logits - max) and its maximum and sum over the last axis; no tokens: 0, -inf, 0."""
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p, m, p.sum(-1, keepdim=True)


def _prefix(s):
    case = s["case"]
    B, hq, hkv, G = case["seqs"], case["hq"], case["hkv"], case["groups"]
    g, scale, dev = hq // hkv, 1 / math.sqrt(D), s["q"].device
    q = s["q"].float()
    # the prefix: the queries of a group's sequences side by side (padded to the largest group)
    members = -(-B // G)
    start = s["group_start"].long()
    b = torch.arange(B, device=dev)
    group = torch.searchsorted(start, b, right=True) - 1
    place = b - start[group]
    who = (start[:-1, None] + torch.arange(members, device=dev)).clamp(max=B - 1)
    qg = q[who].view(G, members, hkv, g, D).transpose(1, 2).reshape(G, hkv, members * g, D)
    table = s["prefix_table"].long()
    kp = s["k_cache"][table].float().transpose(1, 2).reshape(G, hkv, -1, D)
    logits = qg @ kp.transpose(-1, -2) * scale
    past = torch.arange(logits.shape[-1], device=dev) >= s["prefix_tokens"][:, None]
    p, m, l = _weights(logits.masked_fill_(past[:, None, None], -math.inf))
    vp = s["v_cache"][table].float().transpose(1, 2).reshape(G, hkv, -1, D)
    acc = p @ vp

    def of_sequences(x):
        return x.view(G, hkv, members, g, -1)[group, :, place]

    acc, m, l = of_sequences(acc), of_sequences(m), of_sequences(l)
    # each sequence's own tokens
    table = s["page_table"].long()
    ko = s["k_cache"][table].float().transpose(1, 2).reshape(B, hkv, -1, D)
    vo = s["v_cache"][table].float().transpose(1, 2).reshape(B, hkv, -1, D)
    logits = q.view(B, hkv, g, D) @ ko.transpose(-1, -2) * scale
    past = torch.arange(logits.shape[-1], device=dev) >= s["seq_tokens"][:, None]
    po, mo, lo = _weights(logits.masked_fill_(past[:, None, None], -math.inf))
    both = torch.maximum(m, mo)
    safe = torch.where(both == -math.inf, torch.zeros_like(both), both)
    wp, wo = torch.exp(m - safe), torch.exp(mo - safe)
    l = l * wp + lo * wo
    out = (acc * wp + (po @ vo) * wo) / torch.where(l == 0, torch.ones_like(l), l)
    s["out"].copy_(out.view(B, hq, D))
    s["lse"].copy_((both + torch.log(l)).view(B, hq))
    return s["out"], s["lse"]


def _mass(s):
    case = s["case"]
    dev = s["scores"].device
    past = torch.arange(case["pages"], device=dev) >= s["seq_pages"][:, None]
    x = s["scores"].masked_fill(past[:, None], -math.inf)
    p, _, l = _weights(x)
    new = s["mass"] * case["decay"] + (p / l).mean(1)
    s["mass_out"].copy_(torch.where(past, s["mass_out"], new))
    return s["mass_out"]


def _evict(s):
    case = s["case"]
    B, width = s["mass"].shape
    dev = s["mass"].device
    j = torch.arange(width, device=dev)
    n = s["seq_pages"].long()[:, None]
    out = (n - case["keep"]).clamp(min=0)
    held = (j < case["sink"]) | (j >= n - case["recent"])
    order = torch.sort(s["mass"].masked_fill(held, math.inf), dim=1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand(B, -1).contiguous())
    gone = (rank < out) & ~held
    kept = ~gone & (j < n + case["extra"])
    to = torch.where(kept, kept.cumsum(1) - 1, width)

    def packed(x, where, old):
        wide = torch.cat((old, old.new_zeros(B, 1)), 1)
        return wide.scatter_(1, where, x)[:, :old.shape[1]]

    s["table_out"].copy_(packed(s["page_table"], to, s["table_out"]))
    s["mass_out"].copy_(packed(s["mass"], to, s["mass_out"]))
    cap = s["evicted"].shape[1]
    s["evicted"].copy_(packed(s["page_table"], torch.where(gone, gone.cumsum(1) - 1, cap), s["evicted"]))
    s["n_evicted"].copy_(out[:, 0])
    s["seq_out"].copy_((n - out)[:, 0])
    return s["table_out"], s["mass_out"], s["seq_out"], s["evicted"], s["n_evicted"]


def _run_own(s):
    import sparse_kv_page_gb300 as L
    case = s["case"]
    if case["op"] == "append":
        L.locks_append_tokens(s["dims"], s["rope"], s["q"], s["k"], s["v"], s["positions"], s["cache_index"],
                              s["page_table"], s["q_out"], s["k_cache"], s["v_cache"], token_seq=s["token_seq"],
                              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if case["op"] == "prefix":
        L.locks_prefix_attention(s["dims"], s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_tokens"],
                                 s["group_start"], s["page_table"], s["seq_tokens"], s["out"], s["ws"], lse=s["lse"])
        return s["out"], s["lse"]
    if case["op"] == "mass":
        L.locks_accumulate_mass(s["dims"], s["scores"], s["seq_pages"], s["mass"], s["mass_out"], s["ws"],
                                decay=case["decay"])
        return s["mass_out"]
    L.locks_evict_pages(s["dims"], s["mass"], s["page_table"], s["seq_pages"], case["keep"], s["mass_out"],
                        s["table_out"], s["seq_out"], s["evicted"], s["n_evicted"], sink_pages=case["sink"],
                        recent_pages=case["recent"], extra_pages=case["extra"])
    return s["table_out"], s["mass_out"], s["seq_out"], s["evicted"], s["n_evicted"]


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "prefix": _prefix, "mass": _mass, "evict": _evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ floors

def work(case):
    op = case["op"]
    if op == "append":
        live, hq, hkv = case["tokens"] - case["pad"], case["hq"], case["hkv"]
        size_in = 4 if case["itype"] == "fp32" else 2
        size_q = 4 if case["qtype"] == "fp32" else 2
        rows = hq + 2 * hkv
        flops = live * ((hq + hkv) * D * 3 + (4 * (hq + hkv) * D if case["norm"] else 0))
        return {"bytes": live * (rows * D * size_in + hq * D * size_q + 2 * hkv * D * 2 + 4 * (case["axes"] + 3)),
                "flops": flops}
    if op == "prefix":
        B, hq, hkv, G = case["seqs"], case["hq"], case["hkv"], case["groups"]
        # the prefixes of groups after the first are 0.85 of the first's length on average,
        # the own tokens half of the most
        prefix = case["prefix"] * (1 + 0.85 * (G - 1))
        own_tokens = B * case["own_max"] / 2
        q = B * hq * D
        return {"bytes": (prefix + own_tokens) * hkv * D * 4 + q * (4 if case["qtype"] == "fp32" else 2) + q * 2,
                "flops": 4 * D * hq * (B * prefix / G + own_tokens)}
    if op == "mass":
        n = case["seqs"] * case["pages"]
        return {"bytes": n * 4 * (case["hq"] + 2), "flops": n * case["hq"] * 6}
    n = case["seqs"] * (case["pages"] + case["extra"])
    return {"bytes": n * 8 + n * 8, "flops": n * 4}


# ------------------------------------------------------------------ 64 bits

def _exact_append(case, s):
    live, rot = case["tokens"] - case["pad"], case["rot"]
    pos = s["positions"].double()
    turn = torch.stack([torch.polar(torch.ones(live, dtype=torch.float64, device=pos.device), pos[a, :live] * f)
                        for a, f in zip(_axis(case), _inv_freq(case))], 1)[:, None]

    def of(x, w):
        x = x[:live].double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        pair = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["inter"] else \
            x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat((z.flatten(-2), x[..., rot:]), -1)

    q = s["q_out"].double()
    q[:live] = of(s["q"], s["q_weight"])
    index = s["cache_index"][:live].long()
    slot = s["page_table"][s["token_seq"][:live].long(), index.div(PAGE, rounding_mode="floor")].long()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[slot, :, index % PAGE] = of(s["k"], s["k_weight"])
    vc[slot, :, index % PAGE] = s["v"][:live].double()
    return q, kc, vc


def _exact_prefix(case, s):
    B, hq, hkv = case["seqs"], case["hq"], case["hkv"]
    g = hq // hkv
    out = torch.zeros((B, hq, D), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    start, ptok, own_tokens = (s[n].tolist() for n in ("group_start", "prefix_tokens", "seq_tokens"))

    def tokens(cache, table, h, n):
        pages = table[:(n + PAGE - 1) // PAGE].long()
        return cache[pages, h].reshape(-1, D)[:n].double()

    for i, n in enumerate(ptok):
        for h in range(hkv):
            kp, vp = (tokens(s[c], s["prefix_table"][i], h, n) for c in ("k_cache", "v_cache"))
            for b in range(start[i], start[i + 1]):
                ko, vo = (tokens(s[c], s["page_table"][b], h, own_tokens[b]) for c in ("k_cache", "v_cache"))
                q = s["q"][b, h * g:(h + 1) * g].double() / math.sqrt(D)
                x = torch.cat((q @ kp.T, q @ ko.T), 1)
                lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                out[b, h * g:(h + 1) * g] = w[:, :n] @ vp + w[:, n:] @ vo
    return out, lse


def _exact_mass(case, s):
    new = s["mass_out"].double()
    for b, n in enumerate(s["seq_pages"].tolist()):
        share = torch.softmax(s["scores"][b, :, :n].double(), 1).mean(0)
        new[b, :n] = case["decay"] * s["mass"][b, :n].double() + share
    return new


def _exact_evict(case, s):
    mass, table = s["mass"].cpu().numpy(), s["page_table"].cpu().numpy()
    t, m, e = (s[n].cpu().numpy().copy() for n in ("table_out", "mass_out", "evicted"))
    seq, left, gone_n = s["seq_pages"].cpu().numpy(), [], []
    for b, n in enumerate(seq.tolist()):
        free = np.arange(case["sink"], n - case["recent"])
        out = np.sort(free[np.lexsort((free, mass[b, free]))][:max(0, n - case["keep"])])
        rest = np.setdiff1d(np.arange(min(n + case["extra"], mass.shape[1])), out)
        t[b, :rest.size], m[b, :rest.size] = table[b, rest], mass[b, rest]
        e[b, :out.size] = table[b, out]
        left.append(n - out.size)
        gone_n.append(out.size)
    return t, m.astype(np.float64), np.array(left, np.int32), e, np.array(gone_n, np.int32)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prefix": _exact_prefix, "mass": _exact_mass,
            "evict": _exact_evict}[case["op"]](case, s)
