"""Attention over whole contexts and the tables it runs on, as measured cases with a plain form of each.

Four operators, in the order in which a step of a speculative server calls them:

``tables``     block tables and slot maps from request lengths: new blocks for the pages that the
               step's tokens need, and per new token its position, slot and request.
``tree_mask``  who sees whom among the drafted tokens of a tree, as bits, and their positions,
               from each node's parent.
``window``     attention of every new token over the paged attention cache, causal, within a
               sliding window and over a few first tokens that stay visible.
``tree``       attention of drafted tokens over all of a request's earlier tokens and over their
               own ancestors in the tree.

All heads share the token's one latent: keys are its 576 dims, values its first 512. The cache is the
644-byte-per-token one: blocks of ``bs`` tokens, each block ``stride`` bytes, the e4m3 latent of token i
at ``512 i``, its rotated bf16 position dims at ``512 bs + 128 i``, its four E8M0 scale codes at
``640 bs + 4 i`` (a code c scales its 128 dims by 2^(c - 127)).

``run`` computes the plain form in elementary torch operations, or calls the library when ``own`` is set.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
LATENT, PE, QK = 512, 64, 576
SCALE = 192 ** -0.5


def _round_up(a, b):
    return -(-a // b) * b


def kv_block_stride(bs):
    return _round_up(bs * 644, 512)


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 128 requests with long contexts: latency
        {"name": "tables, decode", "op": "tables", "requests": 128, "new": 1, "context": 131072, "block": 64, "pad": 0},
        # a chunked prefill of 256 ragged prompts, padded to the rows of a captured graph
        {"name": "tables, chunk", "op": "tables", "requests": 256, "new": 224, "context": 32768, "block": 64, "pad": 512},
        # eight requests that draft 16 tokens each: latency
        {"name": "tree mask, small", "op": "tree_mask", "requests": 8, "nodes": 16, "words": 1},
        # a full batch with trees of 64 tokens
        {"name": "tree mask, batch", "op": "tree_mask", "requests": 128, "nodes": 64, "words": 2},
        # one user's decode step, every head: latency
        {"name": "window, one row", "op": "window", "requests": 1, "rows": 1, "heads": 128, "context": 32768,
         "window": 4096, "sinks": 4, "block": 64},
        # decode of 128 requests on a server that holds 16 heads
        {"name": "window, decode 128x16", "op": "window", "requests": 128, "rows": 1, "heads": 16, "context": 32768,
         "window": 1024, "sinks": 4, "block": 64},
        # ragged rows of five requests, an odd number of heads, small blocks, some contexts shorter than the window
        {"name": "window, odd", "op": "window", "requests": 5, "rows": 37, "heads": 20, "context": 777, "window": 333,
         "sinks": 7, "block": 16},
        # a prefill chunk of four prompts, every head
        {"name": "window, chunk", "op": "window", "requests": 4, "rows": 512, "heads": 128, "context": 8192,
         "window": 1024, "sinks": 4, "block": 64},
        # one user, eight drafted tokens over a long context, every head
        {"name": "tree, one request", "op": "tree", "requests": 1, "nodes": 8, "heads": 128, "context": 32768, "block": 64},
        # few heads and ragged contexts, small blocks
        {"name": "tree, odd", "op": "tree", "requests": 7, "nodes": 13, "heads": 20, "context": 1500, "block": 16},
        # sixteen requests with larger trees on a server that holds 16 heads
        {"name": "tree, 16x32", "op": "tree", "requests": 16, "nodes": 32, "heads": 16, "context": 16384, "block": 64},
        # a batch of 64 with trees of eight tokens, 64 heads
        {"name": "tree, 64x8", "op": "tree", "requests": 64, "nodes": 8, "heads": 64, "context": 8192, "block": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "tree_mask", "window", "window", "window", "tree", "tree", "tree"])
    block = rng.choice([16, 32, 64, 64, 128])
    if op == "tables":
        B = _log_int(rng, 1, 512)
        return {"op": op, "requests": B, "new": _log_int(rng, 1, max(1, 49152 // B)),
                "context": _log_int(rng, 16, 65536), "block": block, "pad": rng.choice([0, _log_int(rng, 1, 512)])}
    if op == "tree_mask":
        nodes = _log_int(rng, 1, 128)
        return {"op": op, "requests": _log_int(rng, 1, max(1, 8192 // nodes)), "nodes": nodes,
                "words": -(-nodes // 32) + rng.choice([0, 0, 1])}
    heads = rng.choice([_log_int(rng, 1, 128), 16, 32, 64, 128])
    budget = 200 * 1000 * 1000  # pairs of a row's head and a token, below the largest listed case
    if op == "window":
        window, sinks = _log_int(rng, 8, 4096), rng.choice([0, 4, _log_int(rng, 1, 64)])
        requests = _log_int(rng, 1, 128)
        most = max(1, min(budget // heads, 2000 * 1000) // ((window + sinks) * requests))
        rows = rng.choice([1, _log_int(rng, 1, min(most, 1024))])
        return {"op": op, "requests": requests, "rows": rows, "heads": heads,
                "context": max(rows, _log_int(rng, 64, 32768)), "window": window, "sinks": sinks, "block": block}
    requests, nodes = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
    most = max(nodes, budget // (heads * nodes * requests))
    return {"op": op, "requests": requests, "nodes": nodes, "heads": heads,
            "context": max(nodes, _log_int(rng, 64, min(most, 32768)) if most > 64 else most), "block": block}


# Ragged sizes are those of the case, the same for every seed.

def _contexts(B, L, least=1):
    """Lengths between half of the longest and the longest."""
    return [max(least, L - (b * 7919 + b * b * 31) % (L // 2 + 1)) for b in range(B)]


def _row_counts(case):
    """New tokens of each request: ragged where there are several, and one request of many sits out."""
    B = case["requests"]
    n = case["nodes"] if case["op"] in ("tree", "tree_mask") else case["new"] if case["op"] == "tables" else case["rows"]
    counts = [n - (b * 2659 + b * b * 17) % (n // 2 + 1) for b in range(B)]
    if B > 16:
        counts[B // 2] = 0
    return counts


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cumulated(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def _random_cache(blocks, bs, g):
    """An attention cache whose every token holds a quantised random latent."""
    cache = torch.zeros(blocks, kv_block_stride(bs), dtype=torch.uint8, device=DEV)
    lat = torch.randn(blocks * bs, 4, 128, generator=g, device=DEV)
    lat = lat * torch.exp(0.3 * torch.randn(blocks * bs, 4, 1, generator=g, device=DEV))
    code = torch.ceil(torch.log2(lat.abs().amax(dim=2) / 448)).clamp(-127, 7)
    val = (lat / torch.exp2(code)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[:, :512 * bs] = val.view(blocks, bs * 512)
    pe = torch.randn(blocks, bs * 64, generator=g, device=DEV).bfloat16()
    cache[:, 512 * bs:640 * bs] = pe.view(torch.uint8)
    cache[:, 640 * bs:644 * bs] = (code + 127).to(torch.uint8).view(blocks, bs * 4)
    return cache


def _prepare_tables(case, seed):
    g = _gen(seed)
    B, bs = case["requests"], case["block"]
    new = _row_counts(case)
    # cached lengths of any remainder in their last block
    cached = [int(v) for v in torch.randint(0, case["context"] + 1, (B,), generator=g, device=DEV).tolist()]
    held = [-(-c // bs) + (1 if b % 3 == 0 else 0) for b, c in enumerate(cached)]  # some kept a block of drafted tokens
    need = sum(max(0, -(-(c + n) // bs) - h) for c, n, h in zip(cached, new, held))
    pages = -(-(case["context"] + max(new)) // bs) + 1
    total = sum(held) + need
    ids = torch.randperm(total + 37, generator=g, device=DEV).int()
    table = torch.full((B, pages), -1, dtype=torch.int32, device=DEV)
    taken = torch.tensor(held, device=DEV)
    has = torch.arange(pages, device=DEV)[None] < taken[:, None]
    table[has] = ids[:sum(held)]
    n_rows = sum(new) + case["pad"]

    def ints(n, dtype=torch.int32):
        return torch.zeros(n, dtype=dtype, device=DEV)

    return {"bs": bs, "cached_lens": _int32(cached), "new_lens": _int32(new), "held_pages": _int32(held),
            "free_blocks": ids[sum(held):].contiguous(), "free_start": _int32([5]), "table": table,
            "ctx_lens": ints(B), "cu_rows": ints(B + 1), "cu_ctx": ints(B + 1), "held_out": ints(B), "free_end": ints(1),
            "positions": ints(n_rows), "slots": ints(n_rows, torch.int64), "row_to_req": ints(n_rows), "row_ke": ints(n_rows)}


def _random_parents(counts, g):
    """Each node's parent in its request: an earlier node, or -1. Deep and bushy at once, as drafters grow them."""
    parts = []
    for n in counts:
        i = torch.arange(n, device=DEV)
        back = 1 + torch.floor(torch.rand(n, generator=g, device=DEV) ** 2 * torch.clamp(i, max=8)).long()
        parts.append((i - back).clamp(min=-1))
    return torch.cat(parts).int()


def _prepare_tree_mask(case, seed):
    g = _gen(seed)
    counts = _row_counts(case)
    n = sum(counts)
    base = torch.randint(0, 131072, (case["requests"],), generator=g, device=DEV, dtype=torch.int32)
    return {"parents": _random_parents(counts, g), "cu": _int32(_cumulated(counts)), "base": base,
            "mask": torch.zeros(n, case["words"], dtype=torch.int32, device=DEV),
            "positions": torch.zeros(n, dtype=torch.int32, device=DEV)}


def _prepare_attention(case, seed):
    g = _gen(seed)
    B, H, bs = case["requests"], case["heads"], case["block"]
    counts = _row_counts(case)
    lens = _contexts(B, case["context"], max(counts))
    per = -(-max(lens) // bs)
    need = [-(-n // bs) for n in lens]
    ids = torch.randperm(sum(need) + 3, generator=g, device=DEV).int()
    table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)
    has = torch.arange(per, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table[has] = ids[:sum(need)]
    T = sum(counts)
    s = {"bs": bs, "cache": _random_cache(sum(need) + 3, bs, g), "table": table, "cu": _int32(_cumulated(counts)),
         "lens": _int32(lens), "q": (2 * torch.randn(T, H, QK, generator=g, device=DEV)).bfloat16(),
         "out": torch.zeros(T, H, LATENT, dtype=torch.bfloat16, device=DEV),
         "lse": torch.zeros(T, H, dtype=torch.float32, device=DEV), "counts": counts, "ctx": lens, "ws": {}}
    if case["op"] == "window":
        s["window"], s["sinks"] = case["window"], case["sinks"]
    else:
        s["most"] = max(counts)
        s["mask"] = _bits_of(_ancestors(_random_parents(counts, g).long(), s["cu"].long(), T, _round_up(max(counts), 32)))
    return s


def prepare(case, seed):
    op = case["op"]
    s = {"tables": _prepare_tables, "tree_mask": _prepare_tree_mask}.get(op, _prepare_attention)(case, seed)
    s["op"] = op
    return s


# ------------------------------------------------------------------------------ plain forms

def _ancestors(parents, cu, n, width):
    """[n, width] truth values: node m of the row's request is the row itself or one of its ancestors."""
    row = torch.arange(n, device=DEV)
    req = torch.searchsorted(cu[1:], row, right=True)
    at = row - cu[req]
    up = torch.eye(width, device=DEV).repeat(cu.shape[0] - 1, 1, 1)  # of each request: node, and node one step up
    child = parents >= 0
    up[req[child], at[child], parents[child]] = 1
    steps = 1
    while steps < width:  # paths of up to twice the length
        up = (torch.bmm(up, up) > 0).float()
        steps *= 2
    return up[req, at] > 0


def _bits_of(seen):
    """Rows of 32-bit words, bit m % 32 of word m // 32 for column m."""
    w = seen.view(seen.shape[0], -1, 32).long() << torch.arange(32, device=seen.device)
    w = w.sum(dim=2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _plain_tables(s):
    bs, free = s["bs"], s["free_blocks"].long()
    cached, new, held = s["cached_lens"].long(), s["new_lens"].long(), s["held_pages"].long()
    ctx = cached + new
    need = ((ctx + bs - 1) // bs - held).clamp(min=0)
    upto = need.cumsum(0)
    start = s["free_start"].long()
    page = torch.arange(s["table"].shape[1], device=DEV)[None]
    fresh = (page >= held[:, None]) & (page < (held + need)[:, None])
    at = (start + upto - need)[:, None] + page - held[:, None]
    table = torch.where(fresh, free[at.clamp(0, free.shape[0] - 1)].int(), s["table"])
    cu = torch.zeros(new.shape[0] + 1, dtype=torch.long, device=DEV)
    cu[1:] = new.cumsum(0)
    cu_ctx = torch.zeros_like(cu)
    cu_ctx[1:] = ctx.cumsum(0)
    row = torch.arange(s["positions"].shape[0], device=DEV)
    real = row < cu[-1]
    req = torch.searchsorted(cu[1:], row, right=True).clamp(max=new.shape[0] - 1)
    pos = torch.where(real, cached[req] + row - cu[req], torch.zeros_like(row))
    slot = table.long()[req, pos // bs] * bs + pos % bs
    return {"table": table, "ctx_lens": ctx.int(), "cu_rows": cu.int(), "cu_ctx": cu_ctx.int(),
            "held": (held + need).int(), "free_end": (start + upto[-1]).int(), "positions": pos.int(),
            "slots": torch.where(real, slot, torch.full_like(slot, -1)),
            "row_to_req": torch.where(real, req, torch.zeros_like(req)).int(),
            "row_ke": torch.where(real, pos + 1, torch.zeros_like(pos)).int()}


def _plain_tree_mask(s):
    cu = s["cu"].long()
    n, words = s["mask"].shape
    seen = _ancestors(s["parents"].long(), cu, n, 32 * words)
    base = s["base"].long()[torch.searchsorted(cu[1:], torch.arange(n, device=DEV), right=True)]
    return {"mask": _bits_of(seen), "positions": (base + seen.sum(dim=1) - 1).int()}


def _tokens(cache, bs, slot):
    """The 576 dims of the tokens in ``slot`` (any shape, all >= 0), in 32 bits."""
    blk, off = slot // bs, slot % bs
    val = cache[:, :512 * bs].unflatten(1, (bs, 512))[blk, off].view(torch.float8_e4m3fn).float()
    pe = cache[:, 512 * bs:640 * bs].unflatten(1, (bs, 128))[blk, off].view(torch.bfloat16).float()
    code = cache[:, 640 * bs:644 * bs].unflatten(1, (bs, 4))[blk, off].float()
    lat = val.unflatten(-1, (4, 128)) * torch.exp2(code - 127)[..., None]
    return torch.cat([lat.flatten(-2), pe], dim=-1)


def _softmax_rows(logit, visible):
    """Weights and log-sum-exp along the last dim of what is visible; zeros and -inf where nothing is."""
    logit = logit.masked_fill(~visible, -math.inf)
    top = logit.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(logit - top)
    total = p.sum(dim=-1, keepdim=True)
    return p / total.clamp(min=1e-30), (torch.log(total) + top).squeeze(-1)


def _plain_window(s):
    bs, W, S = s["bs"], s["window"], s["sinks"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    row = torch.arange(s["q"].shape[0], device=DEV)[:, None]
    req = torch.searchsorted(cu[1:], row, right=True)
    pos = lens[req] - cu[req + 1] + row
    # each row has a list of its own: the first tokens, then those of its window that are none of them
    far = torch.arange(S, device=DEV)[None].expand(row.shape[0], S)
    near = pos - torch.arange(W, device=DEV)[None]
    visible = torch.cat([far <= pos, near >= S], dim=1)
    key = torch.cat([far, near], dim=1).clamp(min=0).minimum(pos)
    k = _tokens(s["cache"], bs, table[req, key // bs] * bs + key % bs)
    p, lse = _softmax_rows(torch.bmm(s["q"].float(), k.transpose(1, 2)) * SCALE, visible[:, None, :])
    s["out"].copy_(torch.bmm(p, k[:, :, :LATENT]))
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tree(s):
    bs, H, most = s["bs"], s["q"].shape[1], s["most"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    B, T = lens.shape[0], s["q"].shape[0]
    # the requests side by side, as many rows and tokens for each as the longest has
    row = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:], row, right=True)
    at = row - cu[req]
    q = torch.zeros(B, most, H, QK, device=DEV)
    q[req, at] = s["q"].float()
    key = torch.arange(table.shape[1] * bs, device=DEV)[None].minimum(lens[:, None] - 1)
    k = _tokens(s["cache"], bs, torch.gather(table, 1, key // bs) * bs + key % bs)
    token = torch.arange(key.shape[1], device=DEV)
    node = token - (lens - cu[1:] + cu[:-1])[req][:, None]
    bits = torch.gather(s["mask"].long(), 1, (node // 32).clamp(0, s["mask"].shape[1] - 1)) >> (node % 32)
    visible = torch.zeros(B, most, 1, key.shape[1], dtype=torch.bool, device=DEV)
    visible[req, at, 0] = (node < 0) | ((bits & 1 == 1) & (token < lens[req][:, None]))
    logit = torch.bmm(q.view(B, most * H, QK), k.transpose(1, 2)).view(B, most, H, -1) * SCALE
    p, lse = _softmax_rows(logit, visible)
    out = torch.bmm(p.view(B, most * H, -1), k[:, :, :LATENT]).view(B, most, H, LATENT)
    s["out"].copy_(out[req, at])
    s["lse"].copy_(lse[req, at])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ the library's calls

def _own(s):
    import sparse_attention_indexer_fp8_gb300 as idx
    op = s["op"]
    if op == "tables":
        idx.idx_build_tables(s["cached_lens"], s["new_lens"], s["free_blocks"], s["table"], s["bs"], s["ctx_lens"],
                             s["cu_rows"], s["positions"], s["slots"], held_pages=s["held_pages"], held_out=s["held_out"],
                             free_start=s["free_start"], free_end=s["free_end"], cu_ctx=s["cu_ctx"],
                             row_to_req=s["row_to_req"], row_ke=s["row_ke"])
        return {"table": s["table"], "ctx_lens": s["ctx_lens"], "cu_rows": s["cu_rows"], "cu_ctx": s["cu_ctx"],
                "held": s["held_out"], "free_end": s["free_end"], "positions": s["positions"], "slots": s["slots"],
                "row_to_req": s["row_to_req"], "row_ke": s["row_ke"]}
    if op == "tree_mask":
        idx.idx_tree_mask(s["parents"], s["cu"], s["mask"], base_lens=s["base"], positions=s["positions"])
        return {"mask": s["mask"], "positions": s["positions"]}
    if "buf" not in s["ws"]:  # a user's program keeps the workspace of its shapes
        n = idx.idx_paged_attention_workspace_bytes(s["q"].shape[0], s["lens"].shape[0], s["q"].shape[1])
        s["ws"]["buf"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device) if n else None
    if op == "window":
        idx.idx_window_attention(s["q"], s["cache"], s["bs"], s["table"], s["cu"], s["lens"], s["out"], SCALE,
                                 s["window"], sinks=s["sinks"], lse=s["lse"], ws=s["ws"]["buf"])
    else:
        idx.idx_tree_attention(s["q"], s["cache"], s["bs"], s["table"], s["cu"], s["lens"], s["mask"], s["out"], SCALE,
                               lse=s["lse"], ws=s["ws"]["buf"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "tree_mask": _plain_tree_mask, "window": _plain_window,
            "tree": _plain_tree}[state["op"]](state)


# ------------------------------------------------------------------------------ work

def work(case):
    op, B = case["op"], case["requests"]
    counts = _row_counts(case)
    T = sum(counts)
    if op == "tables":
        rows = T + case["pad"]
        fresh = T / case["block"]  # blocks taken, on average
        return {"bytes": rows * 20 + fresh * 8 + B * 28, "flops": 4 * rows}
    if op == "tree_mask":
        return {"bytes": T * (8 + 4 * case["words"]) + B * 8, "flops": T * max(counts)}
    H, bs = case["heads"], case["block"]
    pairs, tokens = 0, 0
    for n, L in zip(counts, _contexts(B, case["context"], max(counts))):
        if n == 0:
            continue
        if op == "window":
            W, S = case["window"], case["sinks"]
            for p in range(L - n, L):
                pairs += min(p + 1, W) + min(S, max(0, p + 1 - W))
            tokens += min(L, n + W - 1) + min(S, max(0, L - n - W + 1))
        else:
            pairs += n * (L - n) + n * min(n, 6)  # a path through a tree of drafted tokens is a handful long
            tokens += L
    mask = T * 4 * -(-max(counts) // 32) if op == "tree" else 0
    return {"bytes": tokens * (644 + 4 / bs) + T * H * (2 * QK + 2 * LATENT + 4) + mask,
            "flops": 2 * H * pairs * (QK + LATENT)}


# ------------------------------------------------------------------------------ exact values

def _exact_tables(s):
    """Request by request, as a scheduler on the host would do it."""
    bs = s["bs"]
    cached, new, held = s["cached_lens"].tolist(), s["new_lens"].tolist(), s["held_pages"].tolist()
    free, at, table = s["free_blocks"].tolist(), int(s["free_start"]), s["table"].tolist()
    n_rows = s["positions"].shape[0]
    ctx, cu, cu_ctx, pos, slot, req = [], [0], [0], [], [], []
    for b in range(len(cached)):
        ctx.append(cached[b] + new[b])
        while held[b] * bs < ctx[b]:
            table[b][held[b]] = free[at]
            held[b] += 1
            at += 1
        for p in range(cached[b], ctx[b]):
            pos.append(p)
            slot.append(table[b][p // bs] * bs + p % bs)
            req.append(b)
        cu.append(len(pos))
        cu_ctx.append(cu_ctx[-1] + ctx[b])
    pad = n_rows - len(pos)
    return {"table": _int32(table), "ctx_lens": _int32(ctx), "cu_rows": _int32(cu), "cu_ctx": _int32(cu_ctx),
            "held": _int32(held), "free_end": _int32([at]), "positions": _int32(pos + [0] * pad),
            "slots": torch.tensor(slot + [-1] * pad, dtype=torch.int64, device=DEV),
            "row_to_req": _int32(req + [0] * pad), "row_ke": _int32([p + 1 for p in pos] + [0] * pad)}


def _exact_tree_mask(s):
    cu, parents, base = s["cu"].tolist(), s["parents"].tolist(), s["base"].tolist()
    words = s["mask"].shape[1]
    mask, pos = [], []
    for b in range(len(cu) - 1):
        seen, deep = [], []
        for i in range(cu[b + 1] - cu[b]):
            up = parents[cu[b] + i]
            seen.append((1 << i) | (seen[up] if up >= 0 else 0))
            deep.append(deep[up] + 1 if up >= 0 else 0)
        for v, d in zip(seen, deep):
            row = [(v >> (32 * w)) & 0xFFFFFFFF for w in range(words)]
            mask.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
            pos.append(base[b] + d)
    return {"mask": _int32(mask).view(len(pos), words), "positions": _int32(pos)}


def _exact_context(s, b):
    """Keys of all of request b's tokens, in 64 bits, decoded bit by bit from the records."""
    bs, L = s["bs"], s["ctx"][b]
    blocks = s["cache"][s["table"][b, :-(-L // bs)].long()]
    byte = blocks[:, :512 * bs].reshape(-1, 512)[:L].long()
    sign = 1.0 - 2.0 * (byte >> 7).double()
    exp, man = (byte >> 3) & 15, (byte & 7).double()
    val = torch.where(exp == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(exp.double() - 7))
    scale = torch.exp2(blocks[:, 640 * bs:644 * bs].reshape(-1, 4)[:L].double() - 127)
    lat = sign * val * scale.repeat_interleave(128, dim=1)
    pe = blocks[:, 512 * bs:640 * bs].reshape(-1, 64, 2)[:L].int()
    half = ((pe[:, :, 1] << 8) | pe[:, :, 0]) << 16
    return torch.cat([lat, half.view(torch.float32).double()], dim=1)


def _exact_attention(s):
    outs, lses = [], []
    t = 0
    H = s["q"].shape[1]
    for b, (n, L) in enumerate(zip(s["counts"], s["ctx"])):
        if n == 0:
            continue
        k = _exact_context(s, b)
        j = torch.arange(L, device=DEV)
        step = max(1, (1 << 26) // (L * H))
        for at in range(0, n, step):
            m = min(step, n - at)
            pos = torch.arange(L - n + at, L - n + at + m, device=DEV)[:, None]
            if s["op"] == "window":
                see = (j <= pos) & ((j > pos - s["window"]) | (j < s["sinks"]))
            else:
                see = (j < L - n).repeat(m, 1)
                for i in range(m):
                    words = [w & 0xFFFFFFFF for w in s["mask"][t + at + i].tolist()]
                    for node in range(n):
                        if words[node // 32] >> (node % 32) & 1:
                            see[i, L - n + node] = True
            used = torch.nonzero(see.any(dim=0)).squeeze(1)
            z = s["q"][t + at:t + at + m].double().reshape(m * H, QK) @ k[used].T * SCALE
            z = z.view(m, H, -1) + torch.where(see[:, used], 0.0, -math.inf).double()[:, None, :]
            lse = torch.logsumexp(z, dim=2)
            outs.append((torch.exp(z - lse[..., None]).view(m * H, -1) @ k[used, :LATENT]).view(m, H, LATENT))
            lses.append(lse)
        t += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "tree_mask": _exact_tree_mask}.get(case["op"], _exact_attention)(s)
