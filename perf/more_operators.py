"""Cases that measure the operators of a cache in 4 bits and of its page pool: packing full
pages to 4 bits and back, decode attention over packed pages (all of them or the selected
ones) with recent bf16 tokens behind, and the pool's page calls: forking sequences,
freeing and taking pages, compacting the pool, with the page copies they ask for.

``run`` computes an operator either in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through this repository's library. Head dim 128, pages of
16 tokens and the 32/8 and 32/2 head layouts are those of the workloads in ``synth``;
context lengths run from a few tokens to the 1M tokens of the longest one.

A packed unit, one page of one kv head, is 2432 bytes: the 4-bit codes of its keys and
values in the order of the tensor cores' fragments, then for every token bf16 scales and
zeros, one of each to 32 dims of a key and to 64 dims of a value: value = zero + scale * code.
"""

import math

import numpy as np
import torch

own = False

D = 128
PAGE = 16
UNIT = 2432
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the pages of a decode batch that fill in one step, 32/8 heads; latency
        dict(name="pack_step_24", op="pack", pages=24, hkv=8),
        # the pages of a 64K-token prompt
        dict(name="pack_prompt_64k", op="pack", pages=4096, hkv=8),
        # two short chats: latency
        dict(name="attend_small", op="attend", seqs=2, hq=32, hkv=8, tokens=347, recent=2, budget=0, qtype="fp32"),
        # a decode batch at 128K tokens of context, dense: the cache's bytes
        dict(name="attend_128k_16", op="attend", seqs=16, hq=32, hkv=8, tokens=131072, recent=2, budget=0,
             qtype="bf16"),
        # two sequences of 1M tokens, 32/2 heads: sixteen queries to a kv head
        dict(name="attend_1m_2", op="attend", seqs=2, hq=32, hkv=2, tokens=1048560, recent=1, budget=0, qtype="fp32"),
        # the decode step's attention: 2048 selected tokens of eight 256K-token sequences
        dict(name="attend_selected_8", op="attend", seqs=8, hq=32, hkv=8, tokens=262144, recent=2, budget=2048,
             qtype="fp32"),
        # a beam search step: eight requests of four beams at 4K tokens, two layers' caches
        dict(name="fork_beams_32", op="fork", groups=8, width=4, tokens=4009, shared=0.8, samples=False, hkv=8,
             layers=2, planes="kv"),
        # 64 samples drawn from each of two 128K-token prompts, four layers of a 32/2 model
        dict(name="fork_samples_128k", op="fork", groups=2, width=64, tokens=131001, shared=1.0, samples=True, hkv=2,
             layers=4, planes="kv"),
        # a step of a busy server: a few sequences end, others grow
        dict(name="free_take_step", op="churn", done=3, grow=29, pages=261, pool=16384, shared=0.3),
        # a pool of 16M tokens: 48 long sequences end, 48 others come
        dict(name="free_take_16m", op="churn", done=48, grow=48, pages=8192, pool=1048576, shared=0.25),
        # a small pool closes up
        dict(name="compact_2k", op="compact", pool=2048, used=0.4, seqs=16, hkv=8, layers=1, planes="packed"),
        # a 1M-token pool, three fifths of it in use, closes up: page copies
        dict(name="compact_64k", op="compact", pool=65536, used=0.6, seqs=64, hkv=4, layers=1, planes="kv"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("pack", "attend", "attend", "attend", "fork", "churn", "compact"))
    hq, hkv = rng.choice(((32, 8), (32, 8), (32, 2), (16, 8), (8, 1), (20, 4)))
    if op == "pack":
        return dict(op=op, pages=_log_int(rng, 1, 32768 // hkv), hkv=hkv)
    if op == "attend":
        seqs = _log_int(rng, 1, 96)
        budget = rng.choice((0, 0, 512, 2048))
        most = min(1 << 20, 2000000 // seqs)    # bytes and products stay below the largest listed case's
        return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, tokens=_log_int(rng, 1, most), recent=rng.randint(0, 4),
                    budget=budget, qtype=rng.choice(("fp32", "bf16")))
    planes = rng.choice(("kv", "kv", "packed"))
    if op == "fork":
        groups, width = _log_int(rng, 1, 16), rng.randint(1, 16)
        return dict(op=op, groups=groups, width=width, tokens=_log_int(rng, 1, 100000 // (groups * width)),
                    shared=round(rng.uniform(0.5, 1.0), 2), samples=rng.random() < 0.4, hkv=hkv,
                    layers=rng.randint(1, 3), planes=planes)
    if op == "churn":
        pool = _log_int(rng, 64, 1000000)
        done, grow = rng.randint(1, 64), rng.randint(1, 64)
        return dict(op=op, done=done, grow=grow, pages=max(1, pool // 4 // max(done, grow) - rng.randint(0, 3)),
                    pool=pool + 64, shared=round(rng.uniform(0, 0.6), 2))
    pool = _log_int(rng, 70, 32768)
    return dict(op=op, pool=pool, used=round(rng.uniform(0.1, 0.95), 2), seqs=rng.randint(1, 48), hkv=hkv,
                layers=1, planes=planes)


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _lengths(case):
    """Packed pages and recent tokens of every sequence: of like sizes, none alike."""
    most = _pages(case["tokens"])
    pages = [most - (b * 7919 + b // 3) % (most // 6 + 1) for b in range(case["seqs"])]
    recent = [(b * 37 + 13) % (PAGE * case["recent"] + 1) for b in range(case["seqs"])]
    return pages, recent


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _prepare_pack(case, g, dev):
    n, hkv = case["pages"], case["hkv"]
    pool = n + n // 2 + 1

    def cache(heads_differ):
        # some channels are far larger than the others, as those of keys are
        x = torch.randn((pool, hkv, PAGE, D), generator=g, device=dev)
        x *= torch.exp(heads_differ * torch.randn((1, hkv, 1, D), generator=g, device=dev))
        x += torch.randn((1, hkv, 1, D), generator=g, device=dev) * heads_differ
        return x.to(torch.bfloat16)

    s = dict(case=case, k_cache=cache(0.6), v_cache=cache(0.1),
             src=torch.randperm(pool, generator=g, device=dev)[:n].int(),
             dst=torch.randperm(n, generator=g, device=dev).int(),
             k_out=torch.zeros((n, hkv, PAGE, D), dtype=torch.bfloat16, device=dev),
             v_out=torch.zeros((n, hkv, PAGE, D), dtype=torch.bfloat16, device=dev))
    if own:                                   # the packed pool and the sizes that a program keeps
        import sparse_kv_page_gb300 as L
        s["packed"] = torch.zeros((n, hkv, UNIT), dtype=torch.uint8, device=dev)
        s["dims"] = L.make_dims(1, hkv, hkv, 1, pool)
        s["out_dims"] = L.make_dims(1, hkv, hkv, 1, n)
    return s


def _packed_pool(units, g, dev):
    """Random units: codes spread as those of normal values are, scales and zeros to match."""
    pool = torch.empty((units, UNIT), dtype=torch.uint8, device=dev)
    spread = torch.randn(1 << 17, generator=g, device=dev).mul_(3.4).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
    table = spread[::2] | (spread[1::2] << 4)                   # of 64K bytes, drawn from by 16 bits
    step = 1 << 16
    for u in range(0, units, step):
        n = min(step, units - u)
        pick = torch.randint(0, 1 << 16, (n, 2048), generator=g, device=dev, dtype=torch.int32)
        pool[u:u + n, :2048] = table[pick]
        scale = 0.29 * torch.exp(0.2 * torch.randn((n, 96), generator=g, device=dev))
        zero = -7.5 * scale + 0.1 * torch.randn((n, 96), generator=g, device=dev)
        # a token's scales, then its zeros: four of either for its key, two for its value
        both = [torch.stack([x[:, a:b].view(n, PAGE, -1) for x in (scale, zero)], 2)
                for a, b in ((0, 64), (64, 96))]
        pool[u:u + n, 2048:] = torch.cat([x.flatten(1) for x in both], 1).to(torch.bfloat16).view(torch.uint8)
    return pool


def _prepare_attend(case, g, dev):
    B, hq, hkv, rp = case["seqs"], case["hq"], case["hkv"], case["recent"]
    pages, recent = _lengths(case)
    P = max(pages)
    phys = B * P + 1
    s = dict(case=case, q=(1.3 * torch.randn((B, hq, D), generator=g, device=dev)).to(TYPES[case["qtype"]]),
             packed=_packed_pool(phys * hkv, g, dev).view(phys, hkv, UNIT),
             page_table=torch.randperm(phys, generator=g, device=dev)[:B * P].view(B, P).int(),
             seq_pages=torch.tensor(pages, dtype=torch.int32, device=dev),
             out=torch.zeros((B, hq, D), dtype=torch.bfloat16, device=dev), lse=torch.zeros((B, hq), device=dev),
             selected=None, n_selected=None, k_cache=None, v_cache=None, recent_table=None, recent_tokens=None)
    if case["budget"]:
        cap = min(case["budget"] // PAGE, P)
        k = torch.minimum(s["seq_pages"], torch.tensor(cap, device=dev))
        draw_ = torch.rand((B, hkv, P), generator=g, device=dev)
        draw_ = draw_.masked_fill(torch.arange(P, device=dev) >= s["seq_pages"][:, None, None], -1.0)
        picked = draw_.topk(cap, -1).indices
        picked = picked.masked_fill(torch.arange(cap, device=dev) >= k[:, None, None], P).sort(-1).values
        s["selected"] = picked.clamp(max=P - 1).int()
        s["n_selected"] = k[:, None].expand(B, hkv).contiguous()
    if rp:
        s["k_cache"], s["v_cache"] = (torch.randn((B * rp, hkv, PAGE, D), generator=g, device=dev).to(torch.bfloat16)
                                      for _ in range(2))
        s["recent_table"] = torch.randperm(B * rp, generator=g, device=dev).view(B, rp).int()
        s["recent_tokens"] = torch.tensor(recent, dtype=torch.int32, device=dev)
    if own:                                   # the sizes and the workspace that a program keeps
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, hq, hkv, P, B * rp)
        s["ws"] = L.alloc_packed_workspace(s["dims"])
    return s


def _planes(case, pool, g, dev):
    if case["planes"] == "kv":
        return [torch.randint(-32768, 32768, (pool, case["hkv"], PAGE, D), generator=g, device=dev, dtype=torch.int16)
                for _ in range(2 * case["layers"])]
    return [torch.randint(0, 256, (pool, case["hkv"], UNIT), generator=g, device=dev, dtype=torch.uint8)
            for _ in range(case["layers"])]


def _prepare_fork(case, g, dev):
    G, W, T = case["groups"], case["width"], case["tokens"]
    B, P = G * W, _pages(T)
    row = torch.arange(B, device=dev)
    first = row // W * W
    tokens = T - first * 31 % (T // 3 + 1)                      # the beams of a request are of one length
    if case["samples"]:                                         # only the prompts are there yet
        tokens = torch.where(row == first, tokens, 0)
        parent = first
    else:
        parent = first + torch.randint(0, W, (B,), generator=g, device=dev)
    n = (tokens + PAGE - 1) // PAGE
    full = tokens // PAGE
    shared = (full * case["shared"]).long()                     # leading pages that a request's rows share
    # one page to a request for a shared place, one to a row for the others
    col = torch.arange(P, device=dev)
    cell = torch.where(col < shared[:, None], first[:, None], row[:, None]) * P + col
    held = col < n[:, None]
    some = torch.zeros(B * P + 1, dtype=torch.bool, device=dev)
    some[torch.where(held, cell, B * P).flatten()] = True
    some[B * P] = False
    pool = int(some.sum()) + B + 7
    perm = torch.randperm(pool, generator=g, device=dev)
    table = torch.where(held, perm[some.long().cumsum(0)[cell] - 1], -1)
    refs = torch.zeros(pool + 1, dtype=torch.int64, device=dev)
    refs.index_add_(0, torch.where(held, table, pool).flatten(), torch.ones(B * P, dtype=torch.int64, device=dev))
    s = dict(case=case, page_table=table.int(), seq_tokens=tokens.int(), parents=parent.int(),
             refs=refs[:pool].int().contiguous(), table_out=torch.full((B, P), -1, dtype=torch.int32, device=dev),
             tokens_out=torch.zeros(B, dtype=torch.int32, device=dev),
             refs_out=torch.zeros(pool, dtype=torch.int32, device=dev),
             copy_src=torch.full((B,), -1, dtype=torch.int32, device=dev),
             copy_dst=torch.full((B,), -1, dtype=torch.int32, device=dev),
             n_copies=torch.zeros(1, dtype=torch.int32, device=dev), planes=_planes(case, pool, g, dev))
    if own:                                   # what a program keeps: sizes, the list of caches, a workspace
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, case["hkv"], case["hkv"], P, pool)
        s["pool_planes"] = L.make_planes(s["planes"])
        s["ws"] = L.alloc_pool_workspace(s["dims"])
    return s


def _prepare_churn(case, g, dev):
    done, grow, n, pool = case["done"], case["grow"], case["pages"], case["pool"]
    perm = torch.randperm(pool, generator=g, device=dev).int()
    shared = int(n * case["shared"])
    col, row = torch.arange(n, device=dev), torch.arange(done, device=dev)[:, None]
    count = (n - row * 5 % (n // 4 + 1)).clamp(min=shared)      # pages of the sequences that end
    # the leading pages are a prompt that all of them share, and another sequence too
    lists = perm[torch.where(col < shared, col, shared + row * n + col)]
    refs = torch.zeros(pool + 1, dtype=torch.int64, device=dev)
    refs.index_add_(0, torch.where(col < count, lists.long(), pool).flatten(),
                    torch.ones(done * n, dtype=torch.int64, device=dev))
    refs = refs[:pool]
    refs[perm[:shared].long()] += 1
    rest = perm[shared + done * n:]                             # of the other pages, a third are held by others
    refs[rest[:(rest.numel() - 2 * grow) // 3].long()] = 1
    b = torch.arange(grow, device=dev)
    old = b * 53 % (PAGE * (n // 8 + 1))
    if pool < 100000:                                           # decoding sequences: a token or a chunk each
        new = old + torch.where(b % 5 == 0, 40, 1).clamp(max=PAGE * n)
    else:
        new = old + PAGE * n // 2 - b * 17
    width = int(_pages(PAGE * (n // 8 + 1) + max(40, PAGE * n)))
    s = dict(case=case, refs=refs.int().contiguous(), lists=lists.contiguous(),
             counts=count[:, 0].int().contiguous(), refs_mid=torch.zeros(pool, dtype=torch.int32, device=dev),
             page_table=torch.full((grow, width), -1, dtype=torch.int32, device=dev), seq_tokens=old.int(),
             new_tokens=torch.maximum(new, old).int(), tokens_out=torch.zeros(grow, dtype=torch.int32, device=dev),
             refs_out=torch.zeros(pool, dtype=torch.int32, device=dev),
             n_free=torch.zeros(1, dtype=torch.int32, device=dev))
    if own:                                   # the sizes and the workspace that a program keeps
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(grow, 1, 1, width, pool)
        s["ws"] = L.alloc_pool_workspace(s["dims"])
    return s


def _prepare_compact(case, g, dev):
    pool, B = case["pool"], case["seqs"]
    used = max(1, int(pool * case["used"]))
    W = max(1, used // B)
    # the sequences' pages lie anywhere in the pool; the first page of all is one shared page
    perm = torch.randperm(pool, generator=g, device=dev).int()
    n = (W - torch.arange(B, device=dev) * 3 % (W // 4 + 1))[:, None]
    col = torch.arange(W, device=dev)
    table = perm[torch.arange(B * W, device=dev).view(B, W).clamp(max=pool - 1)]
    table[:, 0] = perm[0]
    held = col < n
    refs = torch.zeros(pool + 1, dtype=torch.int64, device=dev)
    refs.index_add_(0, torch.where(held, table.long(), pool).flatten(),
                    torch.ones(B * W, dtype=torch.int64, device=dev))
    half = max(1, pool // 2)
    s = dict(case=case, page_table=torch.where(held, table, -1),
             seq_tokens=(n[:, 0] * PAGE - torch.arange(B, device=dev) % PAGE).int(),
             refs=refs[:pool].int().contiguous(), table_out=torch.full((B, W), -1, dtype=torch.int32, device=dev),
             refs_out=torch.zeros(pool, dtype=torch.int32, device=dev),
             move_src=torch.full((half,), -1, dtype=torch.int32, device=dev),
             move_dst=torch.full((half,), -1, dtype=torch.int32, device=dev),
             n_moves=torch.zeros(1, dtype=torch.int32, device=dev),
             new_page=torch.zeros(pool, dtype=torch.int32, device=dev), planes=_planes(case, pool, g, dev))
    if own:                                   # what a program keeps: sizes, the list of caches, a workspace
        import sparse_kv_page_gb300 as L
        s["dims"] = L.make_dims(B, case["hkv"], case["hkv"], W, pool)
        s["pool_planes"] = L.make_planes(s["planes"])
        s["ws"] = L.alloc_pool_workspace(s["dims"])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed)
    return {"pack": _prepare_pack, "attend": _prepare_attend, "fork": _prepare_fork, "churn": _prepare_churn,
            "compact": _prepare_compact}[case["op"]](case, g, dev)


# ------------------------------------------------------------------- runs

def _quantised(x, group):
    """x in groups along its last axis, as zero + scale * code in 32 bits."""
    x = x.float().unflatten(-1, (-1, group))
    zero, most = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((most - zero) / 15).to(torch.bfloat16).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    step = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = torch.where(scale == 0, torch.zeros_like(x), torch.round((x - zero) / step).clamp(0, 15))
    return (zero + scale * code).flatten(-2)


def _pack(s):
    src, dst = s["src"].long(), s["dst"].long()
    # packed page dst[i] comes from page src[i], and goes on to page dst[i] of the output
    s["k_out"][dst] = _quantised(s["k_cache"][src], 32).to(torch.bfloat16)
    s["v_out"][dst] = _quantised(s["v_cache"][src], 64).to(torch.bfloat16)
    return s["k_out"], s["v_out"]


def _unpacked(units):
    """Packed units [..., 2432] as fp32 keys and values [..., 16, 128]."""
    lead = units.shape[:-1]
    n = len(lead)

    def nibbles(lo):
        x = units[..., lo:lo + 1024].reshape(*lead, 2, 8, 4, 4, 2, 2)
        return torch.stack((x & 15, x >> 4), -1)

    def pairs(lo, groups):
        x = units[..., lo:lo + 64 * groups].contiguous().view(torch.bfloat16).float()
        x = x.view(*lead, PAGE, 2, groups, 1)
        return x[..., 0, :, :], x[..., 1, :, :]

    def order(x, axes):
        return x.permute(*range(n), *(n + a for a in axes)).reshape(*lead, PAGE, D).float()

    # keys: [step / 4][token % 8][pair of dims][step % 4][dim % 2][token / 8][dim / 8 % 2]
    k = order(nibbles(0), (5, 1, 0, 3, 6, 2, 4))
    # values: [step / 4][dim % 8][pair of tokens][step % 4][token % 2][token / 8][dim / 8 % 2]
    v = order(nibbles(1024), (5, 2, 4, 0, 3, 6, 1))
    ks, kz = pairs(2048, 4)
    vs, vz = pairs(2304, 2)
    k = (kz + ks * k.unflatten(-1, (4, 32))).flatten(-2)
    v = (vz + vs * v.unflatten(-1, (2, 64))).flatten(-2)
    return k, v


def _attend(s):
    case = s["case"]
    B, hq, hkv = case["seqs"], case["hq"], case["hkv"]
    g = hq // hkv
    pages, recent = _lengths(case)
    heads = torch.arange(hkv, device=s["q"].device)[:, None]
    for b in range(B):
        if s["selected"] is None:
            units = s["packed"][s["page_table"][b, :pages[b]].long()].transpose(0, 1)
        else:
            n = min(pages[b], s["selected"].shape[2])
            units = s["packed"][s["page_table"][b][s["selected"][b, :, :n].long()].long(), heads]
        k, v = _unpacked(units)
        k, v = k.reshape(hkv, -1, D), v.reshape(hkv, -1, D)
        if case["recent"]:
            of = s["recent_table"][b].long()
            k, v = (torch.cat((x, s[c][of].transpose(0, 1).reshape(hkv, -1, D)[:, :recent[b]].float()), 1)
                    for x, c in ((k, "k_cache"), (v, "v_cache")))
        x = s["q"][b].float().view(hkv, g, D) @ k.transpose(1, 2) / math.sqrt(D)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        s["out"][b] = (p @ v / l).view(hq, D).to(torch.bfloat16)
        s["lse"][b] = (m + torch.log(l)).view(hq)
    return s["out"], s["lse"]


def _copy_planes(planes, src, dst, n):
    """planes[dst[i]] = planes[src[i]] for i < n; the lists' rest asks for the first pair again."""
    on = torch.arange(src.numel(), device=src.device) < n
    zero = torch.zeros_like(src[:1])
    a, b = (torch.where(on, x, torch.where(n > 0, x[:1], zero)).long() for x in (src, dst))
    for p in planes:
        p[b] = p[a]


def _free_ids(refs):
    """Page ids, the free ones first and ascending."""
    return torch.sort((refs != 0).int(), stable=True).indices


def _fork(s):
    table, tokens, parent = s["page_table"], s["seq_tokens"].long(), s["parents"].long()
    B, P = table.shape
    dev = table.device
    row, col = torch.arange(B, device=dev), torch.arange(P, device=dev)
    # of the rows that continue a row, itself or else the first keeps its last page
    order = torch.where(parent == row, 0, row + 1)
    keeper = torch.full((B,), B + 1, device=dev).scatter_reduce(0, parent, order, "amin")
    children = torch.zeros(B, dtype=torch.int64, device=dev).index_add_(0, parent, torch.ones_like(parent))
    full, part = tokens // PAGE, tokens % PAGE != 0
    fresh = part[parent] & (order != keeper[parent])
    rank = fresh.long().cumsum(0) - 1
    ids = _free_ids(s["refs"])
    page = ids[rank.clamp(min=0)]
    last = table.gather(1, full[:, None].clamp(max=P - 1))[:, 0].long()
    out = torch.where(col < (full + part)[parent][:, None], table[parent], s["table_out"])
    new = torch.where(fresh[:, None] & (col == full[parent][:, None]), page[:, None].int(), out)
    s["table_out"].copy_(new)
    s["tokens_out"].copy_(tokens[parent])
    refs = s["refs"].long()
    spare = torch.cat((refs, refs.new_zeros(1)))
    pool = refs.numel()
    held = col < full[:, None]
    spare.index_add_(0, torch.where(held, table.long(), pool).flatten(),
                     (held * (children - 1)[:, None]).flatten())
    spare.index_add_(0, torch.where(part, last, pool), ((children > 0).long() - 1) * part)
    spare.index_add_(0, torch.where(fresh, page, pool), fresh.long())
    s["refs_out"].copy_(spare[:pool])
    for name, x in (("copy_src", last[parent]), ("copy_dst", page)):
        wide = torch.cat((s[name].long(), s[name].new_zeros(1).long()))
        s[name].copy_(wide.scatter(0, torch.where(fresh, rank, B), x)[:B])
    s["n_copies"].copy_(fresh.sum()[None])
    _copy_planes(s["planes"], s["copy_src"], s["copy_dst"], s["n_copies"])
    return (s["table_out"], s["tokens_out"], s["refs_out"], s["copy_src"], s["copy_dst"], s["n_copies"], *s["planes"])


def _churn(s):
    lists, refs = s["lists"].long(), s["refs"]
    dev, pool = refs.device, refs.numel()
    on = torch.arange(lists.shape[1], device=dev) < s["counts"][:, None]
    mid = torch.cat((refs, refs.new_zeros(1)))
    mid.index_add_(0, torch.where(on, lists, pool).flatten(), -on.int().flatten())
    s["refs_mid"].copy_(mid[:pool])
    old = (s["seq_tokens"].long() + PAGE - 1) // PAGE
    need = (s["new_tokens"].long() + PAGE - 1) // PAGE - old
    upto = need.cumsum(0)
    ids = _free_ids(s["refs_mid"])
    free = (s["refs_mid"] == 0).sum()
    served = (need == 0) | (upto <= free)
    need = torch.where(served, need, 0)
    col = torch.arange(s["page_table"].shape[1], device=dev)
    at = col - old[:, None]
    mine = (at >= 0) & (at < need[:, None])
    rank = ((upto - need)[:, None] + at).clamp(0, pool - 1)
    s["page_table"].copy_(torch.where(mine, ids[rank].int(), s["page_table"]))
    s["tokens_out"].copy_(torch.where(served, s["new_tokens"], s["seq_tokens"]))
    taken = torch.arange(pool, device=dev) < need.sum()
    s["refs_out"][ids] = torch.where(taken, 1, s["refs_mid"][ids]).int()
    s["n_free"].copy_((free - need.sum())[None])
    return s["refs_mid"], s["page_table"], s["tokens_out"], s["refs_out"], s["n_free"]


def _compact(s):
    refs, table = s["refs"], s["page_table"]
    pool, dev = refs.numel(), refs.device
    page = torch.arange(pool, device=dev)
    used = refs > 0
    end = used.sum()
    hole, high = ~used & (page < end), used & (page >= end)
    dst = torch.sort((~hole).int(), stable=True).indices[:pool // 2]
    src = torch.sort((~high).int(), stable=True).indices[:pool // 2]
    n = high.sum()
    half = s["move_src"].numel()
    on = torch.arange(half, device=dev) < n
    src, dst = (torch.nn.functional.pad(x, (0, half - x.numel())) for x in (src, dst))
    s["move_src"].copy_(torch.where(on, src, s["move_src"]))
    s["move_dst"].copy_(torch.where(on, dst, s["move_dst"]))
    s["n_moves"].copy_(n[None])
    new = torch.cat((page, page[:1])).scatter(0, torch.where(on, src, pool), dst)[:pool]
    s["new_page"].copy_(new)
    out = torch.cat((refs, refs[:1])).scatter(0, torch.where(on, dst, pool), refs[src])
    s["refs_out"].copy_(out.scatter(0, torch.where(on, src, pool), torch.zeros_like(refs[src]))[:pool])
    held = torch.arange(table.shape[1], device=dev) < ((s["seq_tokens"] + PAGE - 1) // PAGE)[:, None]
    s["table_out"].copy_(torch.where(held, new[table.clamp(min=0).long()].int(), s["table_out"]))
    _copy_planes(s["planes"], s["move_src"], s["move_dst"], s["n_moves"])
    return (s["table_out"], s["refs_out"], s["move_src"], s["move_dst"], s["n_moves"], s["new_page"], *s["planes"])


def _run_own(s):
    import sparse_kv_page_gb300 as L
    op = s["case"]["op"]
    if op == "pack":
        n = s["case"]["pages"]
        L.locks_pack_pages(s["dims"], s["k_cache"], s["v_cache"], s["src"], s["dst"], n, s["packed"])
        L.locks_unpack_pages(s["out_dims"], s["packed"], s["dst"], s["dst"], n, s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if op == "attend":
        L.locks_packed_attention(s["dims"], s["q"], s["packed"], s["page_table"], s["seq_pages"], s["out"], s["ws"],
                                 selected=s["selected"], n_selected=s["n_selected"], k_cache=s["k_cache"],
                                 v_cache=s["v_cache"], recent_table=s["recent_table"],
                                 recent_tokens=s["recent_tokens"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "fork":
        L.locks_fork_sequences(s["dims"], s["page_table"], s["seq_tokens"], s["parents"], s["refs"], s["table_out"],
                               s["tokens_out"], s["refs_out"], s["copy_src"], s["copy_dst"], s["n_copies"], s["ws"])
        L.locks_copy_pages(s["pool_planes"], s["copy_src"], s["copy_dst"], s["n_copies"])
        return (s["table_out"], s["tokens_out"], s["refs_out"], s["copy_src"], s["copy_dst"], s["n_copies"],
                *s["planes"])
    if op == "churn":
        L.locks_free_pages(s["refs"], s["lists"], s["counts"], s["refs_mid"])
        L.locks_take_pages(s["dims"], s["page_table"], s["seq_tokens"], s["new_tokens"], s["refs_mid"],
                           s["tokens_out"], s["refs_out"], s["ws"], n_free=s["n_free"])
        return s["refs_mid"], s["page_table"], s["tokens_out"], s["refs_out"], s["n_free"]
    L.locks_compact_pages(s["dims"], s["page_table"], s["seq_tokens"], s["refs"], s["table_out"], s["refs_out"],
                          s["move_src"], s["move_dst"], s["n_moves"], s["new_page"], s["ws"])
    L.locks_copy_pages(s["pool_planes"], s["move_src"], s["move_dst"], s["n_moves"])
    return (s["table_out"], s["refs_out"], s["move_src"], s["move_dst"], s["n_moves"], s["new_page"], *s["planes"])


def run(state):
    if own:
        return _run_own(state)
    return {"pack": _pack, "attend": _attend, "fork": _fork, "churn": _churn,
            "compact": _compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ floors

def _page_bytes(case):
    return case["layers"] * case["hkv"] * (2 * PAGE * D * 2 if case["planes"] == "kv" else UNIT)


def work(case):
    op = case["op"]
    if op == "pack":
        units = case["pages"] * case["hkv"]
        return {"bytes": units * 2 * (UNIT + 4 * PAGE * D), "flops": units * PAGE * D * 2 * 6}
    if op == "attend":
        hq, hkv = case["hq"], case["hkv"]
        pages, recent = _lengths(case)
        if case["budget"]:
            pages = [min(p, case["budget"] // PAGE) for p in pages]
        q = case["seqs"] * hq * D
        return {"bytes": sum(pages) * hkv * UNIT + sum(recent) * hkv * D * 4 + sum(pages) * 4
                + q * (4 if case["qtype"] == "fp32" else 2) + q * 2,
                "flops": 4 * D * hq * (sum(pages) * PAGE + sum(recent))}
    if op == "fork":
        B, P = case["groups"] * case["width"], _pages(case["tokens"])
        # the last page of about every second beam is copied, of a prompt's samples for all but one
        copies = B - case["groups"] if case["samples"] else B * 0.4
        read = case["groups"] if case["samples"] else B
        return {"bytes": (read + B) * P * 4 + 2 * 4 * B * P + 2 * copies * _page_bytes(case), "flops": B * P}
    if op == "churn":
        listed_ = case["done"] * case["pages"]
        return {"bytes": 4 * 4 * case["pool"] + 4 * listed_ + 4 * case["grow"], "flops": case["pool"]}
    moved = case["used"] * (1 - case["used"]) * case["pool"]
    return {"bytes": 2 * moved * _page_bytes(case) + 4 * 3 * case["pool"] + 8 * case["used"] * case["pool"],
            "flops": case["pool"]}


# ------------------------------------------------------------------ 64 bits

def _exact_pack(case, s):
    def values(cache, group):
        x = cache[s["src"].long()].double()
        x = x.reshape(*x.shape[:-1], D // group, group)
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        step = torch.div(hi - lo, 15.0).bfloat16().double()
        code = torch.nan_to_num(torch.div(x - lo, step)).round().clamp(0, 15)
        out = torch.empty(x.shape[:-2] + (D,), dtype=torch.float64, device=x.device)
        out[s["dst"].long()] = (lo + step * code).reshape(out.shape)
        return out

    return values(s["k_cache"], 32), values(s["v_cache"], 64)


def _exact_attend(case, s):
    B, hq, hkv = case["seqs"], case["hq"], case["hkv"]
    g = hq // hkv
    dev = s["q"].device
    out = torch.zeros((B, hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=dev)
    t, d = torch.arange(PAGE, device=dev)[:, None], torch.arange(D, device=dev)[None]

    def place(row, col):
        """Byte and shift of an element: row and column of the tensor cores' fragment."""
        word, lane = col // 16, 4 * (row % 8) + col % 8 // 2
        bit = 16 * (col % 2) + 4 * (col // 8 % 2) + 8 * (row // 8)
        return word // 4 * 512 + lane * 16 + word % 4 * 4 + bit // 8, bit % 8

    k_byte, k_bit = place(t, d)
    word, lane = d // 16, 4 * (d % 8) + t % 8 // 2
    bit = 16 * (t % 2) + 4 * (d % 16 // 8) + 8 * (t // 8)
    v_byte, v_bit = 1024 + word // 4 * 512 + lane * 16 + word % 4 * 4 + bit // 8, bit % 8

    def of(units, byte, shift, lo, group):
        code = (units[:, byte.flatten()].int() >> shift.flatten()) & 15
        pair = units[:, lo:lo + 64 * (D // group)].contiguous().view(torch.bfloat16).double()
        pair = pair.view(-1, PAGE, 2, D // group).repeat_interleave(group, 3)
        return (pair[:, :, 1] + pair[:, :, 0] * code.view(-1, PAGE, D).double()).view(-1, D)

    pages, recent = _lengths(case)
    for b in range(B):
        for h in range(hkv):
            logical = torch.arange(pages[b], device=dev)
            if s["selected"] is not None:
                logical = s["selected"][b, h, :min(pages[b], s["selected"].shape[2])].long()
            ids = s["page_table"][b].long()[logical]
            q = s["q"][b, h * g:(h + 1) * g].double() / math.sqrt(D)
            xs, vs = [], []
            for i in range(0, ids.numel(), 16384):
                units = s["packed"][ids[i:i + 16384], h]
                xs.append(q @ of(units, k_byte, k_bit, 2048, 32).T)
                vs.append(of(units, v_byte, v_bit, 2304, 64))
            if case["recent"]:
                rows = s["recent_table"][b].long()
                xs.append(q @ s["k_cache"][rows, h].reshape(-1, D)[:recent[b]].double().T)
                vs.append(s["v_cache"][rows, h].reshape(-1, D)[:recent[b]].double())
            x = torch.cat(xs, 1)
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, 1)
            out[b, h * g:(h + 1) * g] = torch.softmax(x, 1) @ torch.cat(vs)
    return out, lse


def _host(s, *names):
    return [s[n].cpu().numpy().copy() for n in names]


def _moved(s, src, dst):
    planes = [p.cpu().numpy().copy() for p in s["planes"]]
    for p in planes:
        p[dst] = p[src]
    return planes


def _exact_fork(case, s):
    table, tokens, parents, refs, out = _host(s, "page_table", "seq_tokens", "parents", "refs", "table_out")
    free = iter(np.flatnonzero(refs == 0))
    new_refs, new_tokens = refs.copy(), np.zeros_like(tokens)
    src, dst, kept = [], [], {}
    for b, p in enumerate(parents):
        if p not in kept or p == b:
            kept[p] = b
    for b in range(tokens.size):
        new_refs[table[b, :_pages(tokens[b])]] -= 1
    for b, p in enumerate(parents):
        n = _pages(tokens[p])
        row = table[p, :n].copy()
        if tokens[p] % PAGE and kept[p] != b:
            src.append(row[-1])
            row[-1] = next(free)
            dst.append(row[-1])
        out[b, :n] = row
        new_refs[row] += 1
        new_tokens[b] = tokens[p]
    lists = [np.concatenate((np.array(x, np.int32), np.full(tokens.size - len(x), -1, np.int32))) for x in (src, dst)]
    return (out, new_tokens, new_refs, *lists, np.array([len(src)], np.int32),
            *_moved(s, np.array(src, np.int64), np.array(dst, np.int64)))


def _exact_churn(case, s):
    refs, lists, counts, table, old, new = _host(s, "refs", "lists", "counts", "page_table", "seq_tokens",
                                                 "new_tokens")
    for b, n in enumerate(counts):
        np.subtract.at(refs, lists[b, :n], 1)
    mid, free, tokens = refs.copy(), np.flatnonzero(refs == 0), old.copy()
    at, left = 0, True
    for b in range(old.size):
        have, want = _pages(int(old[b])), _pages(int(new[b]))
        if want > have:
            left = left and at + want - have <= free.size
            if not left:
                continue
            table[b, have:want] = free[at:at + want - have]
            refs[table[b, have:want]] = 1
            at += want - have
        tokens[b] = new[b]
    return mid, table, tokens, refs, np.array([free.size - at], np.int32)


def _exact_compact(case, s):
    table, tokens, refs, out, src, dst = _host(s, "page_table", "seq_tokens", "refs", "table_out", "move_src",
                                               "move_dst")
    used = np.flatnonzero(refs)
    gone = used[used >= used.size]
    into = np.setdiff1d(np.arange(used.size), used)
    src[:gone.size], dst[:gone.size] = gone, into
    new = np.arange(refs.size, dtype=np.int32)
    new[gone] = into
    for b, n in enumerate(tokens):
        out[b, :_pages(n)] = new[table[b, :_pages(n)]]
    after = np.zeros_like(refs)
    after[new[used]] = refs[used]
    return (out, after, src, dst, np.array([gone.size], np.int32), new, *_moved(s, gone, into))


def exact(case, seed):
    s = prepare(case, seed)
    return {"pack": _exact_pack, "attend": _exact_attend, "fork": _exact_fork, "churn": _exact_churn,
            "compact": _exact_compact}[case["op"]](case, s)
