"""The operators around the indexer's selection, as measured cases with a plain form of each.

Four operators, in the order in which one layer's step calls them:

``k_insert``   LayerNorm of the indexer's k, partial RoPE, e4m3 quantisation and the insert
               into the paged 132-byte-per-token indexer cache, in one pass.
``kv_insert``  RMSNorm of the attention latent (512 dims), RoPE of its 64 position dims,
               e4m3 quantisation with one power-of-two scale per 128 dims and the insert
               into the paged 644-byte-per-token attention cache, in one pass.
``kv_gather``  read-back of that cache: the tokens of a batch of requests, dequantised to
               bf16 and packed one request after another (what a prompt's dense attention
               over an earlier context reads).
``attention``  attention of every query row over the tokens that the indexer selected for
               it, read straight from the cache through their slots; all heads share the
               token's one latent (keys are its 576 dims, values its first 512).

Attention cache, blocks of ``bs`` tokens, each block ``stride`` bytes: the e4m3 latent of
token i at ``512 i``, its rotated bf16 position dims at ``512 bs + 128 i``, and its four
E8M0 scale codes at ``640 bs + 4 i``. A code c scales its 128 dims by 2^(c - 127); the scale is
the smallest power of two >= amax / 448, its code held to [0, 134].

``run`` computes the plain form in elementary torch operations, or calls the library when
``own`` is set.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
LATENT, PE, QK = 512, 64, 576
MAX_POS = 65536


def _round_up(a, b):
    return -(-a // b) * b


def k_block_stride(bs):
    return _round_up(bs * 132, 512)


def kv_block_stride(bs):
    return _round_up(bs * 644, 512)


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 128: latency of the two inserts
        {"name": "k insert, decode", "op": "k_insert", "tokens": 128, "block": 64, "dtype": "bf16",
         "interleaved": False},
        # one prefill chunk of 8192 tokens
        {"name": "k insert, chunk", "op": "k_insert", "tokens": 8192, "block": 64, "dtype": "bf16",
         "interleaved": False},
        {"name": "kv insert, decode", "op": "kv_insert", "tokens": 128, "block": 64, "dtype": "bf16",
         "interleaved": True},
        {"name": "kv insert, chunk", "op": "kv_insert", "tokens": 8192, "block": 64, "dtype": "bf16",
         "interleaved": True},
        # a few short prompts with a cached prefix, ragged
        {"name": "kv gather, short", "op": "kv_gather", "requests": 5, "max_len": 2048, "block": 64,
         "out": "bf16"},
        # eight long contexts
        {"name": "kv gather, long", "op": "kv_gather", "requests": 8, "max_len": 32768, "block": 64,
         "out": "bf16"},
        # one user's decode step: latency
        {"name": "attention, one row", "op": "attention", "rows": 1, "heads": 128, "topk": 2048,
         "context": 32768, "block": 64},
        # a small batch with a few heads (a head-sharded server), odd sizes, short and empty lists
        {"name": "attention, odd", "op": "attention", "rows": 37, "heads": 20, "topk": 777, "context": 1500,
         "block": 16},
        # decode of 64 requests, every head
        {"name": "attention, decode 64", "op": "attention", "rows": 64, "heads": 128, "topk": 2048,
         "context": 32768, "block": 64},
        # decode of 128 requests on a server that holds 16 heads
        {"name": "attention, decode 128x16", "op": "attention", "rows": 128, "heads": 16, "topk": 2048,
         "context": 32768, "block": 64},
        # two rows for each of 128 requests (multi-token prediction), 64 heads
        {"name": "attention, decode 256x64", "op": "attention", "rows": 256, "heads": 64, "topk": 2048,
         "context": 32768, "block": 64},
        # part of a prefill chunk
        {"name": "attention, chunk", "op": "attention", "rows": 1024, "heads": 128, "topk": 2048,
         "context": 32768, "block": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["k_insert", "kv_insert", "kv_gather", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64, 64, 128])
    if op in ("k_insert", "kv_insert"):
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "block": block,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "interleaved": rng.random() < 0.5}
    if op == "kv_gather":
        return {"op": op, "requests": _log_int(rng, 1, 16), "max_len": _log_int(rng, 1, 16384), "block": block,
                "out": rng.choice(["bf16", "bf16", "fp32"])}
    heads = rng.choice([_log_int(rng, 1, 128), 16, 32, 64, 128])
    topk = rng.choice([_log_int(rng, 1, 2048), 512, 2048])
    rows = _log_int(rng, 1, 1024)
    return {"op": op, "rows": rows, "heads": heads, "topk": topk,
            "context": max(topk, _log_int(rng, 64, 32768)), "block": block}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cos_sin():
    i = torch.arange(32, dtype=torch.float64, device=DEV)
    ang = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-2.0 * i / 64)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _prepare_insert(case, seed):
    g = _gen(seed)
    n, bs, dt = case["tokens"], case["block"], _dtype(case)
    blocks = -(-n // bs) + 2
    s = {"bs": bs, "interleaved": case["interleaved"], "cos_sin": _cos_sin(), "eps": 1e-6}
    s["positions"] = torch.randint(0, MAX_POS, (n,), generator=g, device=DEV, dtype=torch.int32)
    s["slots"] = torch.randperm(blocks * bs, generator=g, device=DEV)[:n]
    # projections come out with a common offset and a spread that varies from token to token
    spread = torch.exp(0.5 * torch.randn(n, 1, generator=g, device=DEV))
    if case["op"] == "k_insert":
        x = torch.randn(n, 128, generator=g, device=DEV) * spread + 0.2 * torch.randn(1, 128, generator=g, device=DEV)
        s["k"] = x.to(dt)
        s["weight"] = 1 + 0.3 * torch.randn(128, generator=g, device=DEV)
        s["bias"] = 0.2 * torch.randn(128, generator=g, device=DEV)
        s["cache"] = torch.zeros(blocks, k_block_stride(bs), dtype=torch.uint8, device=DEV)
    else:
        x = torch.randn(n, QK, generator=g, device=DEV) * spread
        s["proj"] = x.to(dt)  # one projection: 512 latent dims, then the 64 position dims
        s["weight"] = 1 + 0.3 * torch.randn(LATENT, generator=g, device=DEV)
        s["cache"] = torch.zeros(blocks, kv_block_stride(bs), dtype=torch.uint8, device=DEV)
    return s


def _random_cache(blocks, bs, g):
    """An attention cache whose every token holds a quantised random latent."""
    stride = kv_block_stride(bs)
    cache = torch.zeros(blocks, stride, dtype=torch.uint8, device=DEV)
    lat = torch.randn(blocks * bs, 4, 128, generator=g, device=DEV)
    lat = lat * torch.exp(0.3 * torch.randn(blocks * bs, 4, 1, generator=g, device=DEV))
    code = torch.ceil(torch.log2(lat.abs().amax(dim=2) / 448)).clamp(-127, 7)
    val = (lat / torch.exp2(code)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[:, :512 * bs] = val.view(blocks, bs * 512)
    pe = torch.randn(blocks, bs * 64, generator=g, device=DEV).bfloat16()
    cache[:, 512 * bs:640 * bs] = pe.view(torch.uint8)
    cache[:, 640 * bs:644 * bs] = (code + 127).to(torch.uint8).view(blocks, bs * 4)
    return cache


def _prepare_gather(case, seed):
    g = _gen(seed)
    B, L, bs = case["requests"], case["max_len"], case["block"]
    # ragged lengths between half of the longest and the longest, the same for every seed of a case
    lens = torch.tensor([L - (b * 7919 + b * b * 31) % (L // 2 + 1) for b in range(B)], device=DEV)
    per = -(-L // bs)
    bt = torch.randperm(B * per, generator=g, device=DEV).view(B, per).int()
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = lens.cumsum(0)
    total = int(cu[-1])
    out = torch.zeros(total, QK, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
    return {"bs": bs, "cache": _random_cache(B * per, bs, g), "block_table": bt, "cu": cu, "out": out}


def _prepare_attention(case, seed):
    g = _gen(seed)
    T, H, K, L, bs = case["rows"], case["heads"], case["topk"], case["context"], case["block"]
    # up to eight contexts of at most L tokens, shared by the rows
    B = min(8, T)
    per = -(-L // bs)
    cache = _random_cache(B * per, bs, g)
    bt = torch.randperm(B * per, generator=g, device=DEV).view(B, per)
    req = torch.arange(T, device=DEV) % B
    # row t sees a context of its own length; the selection keeps K distinct tokens of it, or all
    # of a shorter one, the rest of the list -1; one row of several has no token at all
    seen = torch.randint(L // 2 + 1, L + 1, (T,), generator=g, device=DEV)
    short = torch.rand(T, generator=g, device=DEV) < 0.1
    seen = torch.where(short, torch.randint(1, L + 1, (T,), generator=g, device=DEV), seen)
    if T > 16:
        seen[T // 2] = 0
    key = torch.rand(T, L, generator=g, device=DEV)
    key = torch.where(torch.arange(L, device=DEV)[None] < seen[:, None], key, torch.full_like(key, -1.0))
    score, pos = key.topk(K, dim=1)
    slot = bt[req[:, None], pos // bs] * bs + pos % bs
    slots = torch.where(score >= 0, slot, torch.full_like(slot, -1)).int()
    q = 2 * torch.randn(T, H, QK, generator=g, device=DEV)
    return {"bs": bs, "cache": cache, "slots": slots, "q": q.bfloat16(), "scale": QK ** -0.5,
            "out": torch.zeros(T, H, LATENT, dtype=torch.bfloat16, device=DEV),
            "lse": torch.zeros(T, H, dtype=torch.float32, device=DEV), "ws": {}}


def prepare(case, seed):
    op = case["op"]
    if op in ("k_insert", "kv_insert"):
        s = _prepare_insert(case, seed)
    elif op == "kv_gather":
        s = _prepare_gather(case, seed)
    else:
        s = _prepare_attention(case, seed)
    s["op"] = op
    return s


# ------------------------------------------------------------------------------ plain forms

def _rope(x, cos, sin, interleaved):
    """Rotation of the pairs of the last dim (64): (i, i + 32), or (2i, 2i + 1)."""
    a, b = (x[:, 0::2], x[:, 1::2]) if interleaved else (x[:, :32], x[:, 32:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], dim=2).reshape(x.shape) if interleaved else torch.cat([u, v], dim=1)


def _table(s):
    row = s["cos_sin"][s["positions"].long()]
    return row[:, :32], row[:, 32:]


def _k_views(cache, bs):
    """The indexer cache's e4m3 values and fp32 scales, [blocks, bs, 128] and [blocks, bs]."""
    values = cache[:, :128 * bs].unflatten(1, (bs, 128)).view(torch.float8_e4m3fn)
    return {"k": values, "scale": cache[:, 128 * bs:132 * bs].view(torch.float32)}


def _kv_views(cache, bs):
    """The attention cache's e4m3 latents, bf16 position dims and E8M0 scales."""
    return {"latent": cache[:, :512 * bs].unflatten(1, (bs, 512)).view(torch.float8_e4m3fn),
            "pe": cache[:, 512 * bs:640 * bs].unflatten(1, (bs, 128)).view(torch.bfloat16),
            "scale": cache[:, 640 * bs:644 * bs].unflatten(1, (bs, 4)).view(torch.float8_e8m0fnu)}


def _plain_k_insert(s):
    x, bs = s["k"].float(), s["bs"]
    c = x - x.mean(dim=1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"] + s["bias"]
    cos, sin = _table(s)
    y = torch.cat([_rope(y[:, :64], cos, sin, s["interleaved"]), y[:, 64:]], dim=1)
    scale = y.abs().amax(dim=1) / 448
    code = (y / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    blk, off = s["slots"] // bs, s["slots"] % bs
    values = s["cache"][:, :128 * bs].unflatten(1, (bs, 128))
    scales = s["cache"][:, 128 * bs:132 * bs].unflatten(1, (bs, 4))
    values[blk, off] = code
    scales[blk, off] = scale[:, None].view(torch.uint8)
    return _k_views(s["cache"], bs)


def _plain_kv_insert(s):
    x, bs = s["proj"].float(), s["bs"]
    c, pe = x[:, :LATENT], x[:, LATENT:]
    y = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"]
    cos, sin = _table(s)
    pe = _rope(pe, cos, sin, s["interleaved"]).bfloat16()
    t = y.view(-1, 4, 128)
    m, e = torch.frexp(t.abs().amax(dim=2) / 448)  # m in [0.5, 1): the power of two at or above is 2^e, or 2^(e - 1)
    e = (e - (m == 0.5).int()).clamp(-127, 7)
    code = (t / torch.exp2(e.float())[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    blk, off = s["slots"] // bs, s["slots"] % bs
    s["cache"][:, :512 * bs].unflatten(1, (bs, 512))[blk, off] = code.view(-1, 512)
    s["cache"][:, 512 * bs:640 * bs].unflatten(1, (bs, 128))[blk, off] = pe.view(torch.uint8)
    s["cache"][:, 640 * bs:644 * bs].unflatten(1, (bs, 4))[blk, off] = (e + 127).to(torch.uint8)
    return _kv_views(s["cache"], bs)


def _tokens(cache, bs, slot):
    """The 576 dims of the tokens in ``slot`` (any shape, all >= 0), in 32 bits."""
    blk, off = slot // bs, slot % bs
    val = cache[:, :512 * bs].unflatten(1, (bs, 512))[blk, off].view(torch.float8_e4m3fn).float()
    pe = cache[:, 512 * bs:640 * bs].unflatten(1, (bs, 128))[blk, off].view(torch.bfloat16).float()
    code = cache[:, 640 * bs:644 * bs].unflatten(1, (bs, 4))[blk, off].float()
    lat = val.unflatten(-1, (4, 128)) * torch.exp2(code - 127)[..., None]
    return torch.cat([lat.flatten(-2), pe], dim=-1)


def _plain_kv_gather(s):
    cu, bs = s["cu"].long(), s["bs"]
    row = torch.arange(s["out"].shape[0], device=cu.device)
    req = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[req]
    slot = s["block_table"].long()[req, pos // bs] * bs + pos % bs
    s["out"].copy_(_tokens(s["cache"], bs, slot))
    return s["out"]


def _plain_attention(s):
    slot = s["slots"].long()
    valid = slot >= 0
    k = _tokens(s["cache"], s["bs"], slot.clamp(min=0))
    logit = torch.bmm(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    logit = logit.masked_fill(~valid[:, None, :], -math.inf)
    top = logit.amax(dim=2, keepdim=True).clamp(min=-3e38)
    p = torch.exp(logit - top)
    total = p.sum(dim=2, keepdim=True)
    out = torch.bmm(p, k[:, :, :LATENT]) / total.clamp(min=1e-30)
    return {"out": out.bfloat16(), "lse": (torch.log(total) + top).squeeze(2)}


# ------------------------------------------------------------------------------ the library's calls

def _own(s):
    import sparse_attention_indexer_fp8_gb300 as idx
    op = s["op"]
    if op == "k_insert":
        idx.idx_k_norm_rope_quant_and_cache(s["k"], s["weight"], s["bias"], s["eps"], s["positions"], s["cos_sin"],
                                            s["slots"], s["cache"], s["bs"], interleaved=s["interleaved"])
        return _k_views(s["cache"], s["bs"])
    if op == "kv_insert":
        idx.idx_kv_norm_rope_quant_and_cache(s["proj"][:, :LATENT], s["proj"][:, LATENT:], s["weight"], s["eps"],
                                             s["positions"], s["cos_sin"], s["slots"], s["cache"], s["bs"],
                                             interleaved=s["interleaved"])
        return _kv_views(s["cache"], s["bs"])
    if op == "kv_gather":
        idx.idx_gather_kv(s["cache"], s["bs"], s["block_table"], s["cu"], s["out"])
        return s["out"]
    if "buf" not in s["ws"]:  # a user's program keeps the workspace of its shapes
        n = idx.idx_sparse_attention_workspace_bytes(s["q"].shape[0], s["q"].shape[1], s["slots"].shape[1])
        s["ws"]["buf"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device) if n else None
    idx.idx_sparse_attention(s["q"], s["cache"], s["bs"], s["slots"], s["out"], s["scale"], lse=s["lse"],
                             ws=s["ws"]["buf"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "k_insert":
        return _plain_k_insert(state)
    if op == "kv_insert":
        return _plain_kv_insert(state)
    if op == "kv_gather":
        return _plain_kv_gather(state)
    return _plain_attention(state)


# ------------------------------------------------------------------------------ work

def _mean_list(k, lo, hi):
    """The mean of min(k, n) over the whole numbers n in [lo, hi]."""
    if k <= lo:
        return float(k)
    k = min(k, hi)
    return ((k - lo) * (k - 1 + lo) / 2 + k * (hi - k + 1)) / (hi - lo + 1)


def work(case):
    op = case["op"]
    if op in ("k_insert", "kv_insert"):
        n, sz = case["tokens"], 2 if case["dtype"] == "bf16" else 4
        dims, rec = (128, 132) if op == "k_insert" else (QK, 644)
        table = n * 256 + n * 12  # the rows of the angle table, positions and slots
        return {"bytes": n * (dims * sz + rec) + table, "flops": 12 * n * dims}
    if op == "kv_gather":
        L = case["max_len"]
        n = sum(L - (b * 7919 + b * b * 31) % (L // 2 + 1) for b in range(case["requests"]))
        return {"bytes": n * (644 + QK * (2 if case["out"] == "bf16" else 4)), "flops": n * QK}
    T, H, K, L = case["rows"], case["heads"], case["topk"], case["context"]
    # the tokens of the rows' lists, or the whole of the contexts where that is less
    listed_tokens = T * (0.9 * _mean_list(K, L // 2 + 1, L) + 0.1 * _mean_list(K, 1, L))
    tokens = min(listed_tokens, min(8, T) * L)
    return {"bytes": tokens * 644 + T * (4 * K + H * (2 * QK + 2 * LATENT + 4)),
            "flops": 2 * H * listed_tokens * (QK + LATENT)}


# ------------------------------------------------------------------------------ exact values

def _e4m3(v):
    """The e4m3 values nearest to v (ties to even mantissas), saturating at 448, in 64 bits."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _turn(x, s):
    """Rotation of 64 dims as a complex product."""
    row = s["cos_sin"].double()[s["positions"].long()]
    z = torch.complex(row[:, :32], row[:, 32:])
    p = x.view(-1, 32, 2) if s["interleaved"] else torch.stack([x[:, :32], x[:, 32:]], dim=2)
    r = torch.view_as_real(torch.view_as_complex(p.contiguous()) * z)
    return r.reshape(-1, 64) if s["interleaved"] else r.transpose(1, 2).reshape(-1, 64)


def _place(s, blocks, values):
    out = torch.zeros(blocks * s["bs"], values.shape[1], dtype=torch.float64, device=values.device)
    out[s["slots"]] = values
    return out.view(blocks, s["bs"], -1)


def _exact_k_insert(s):
    x = s["k"].double()
    y = (x - x.mean(1, True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + s["eps"])
    y = y * s["weight"].double() + s["bias"].double()
    y = torch.cat([_turn(y[:, :64], s), y[:, 64:]], dim=1)
    scale = y.abs().max(dim=1, keepdim=True).values / 448
    blocks = s["cache"].shape[0]
    return {"k": _place(s, blocks, _e4m3(y / scale)), "scale": _place(s, blocks, scale).squeeze(2)}


def _exact_kv_insert(s):
    x = s["proj"].double()
    c = x[:, :LATENT]
    y = c / torch.sqrt(c.square().mean(1, True) + s["eps"]) * s["weight"].double()
    t = y.view(-1, 4, 128)
    e = torch.ceil(torch.log2(t.abs().max(dim=2).values / 448)).clamp(-127, 7)
    blocks = s["cache"].shape[0]
    scale = _place(s, blocks, torch.exp2(e))
    scale = torch.where(scale == 0, torch.full_like(scale, 2.0 ** -127), scale)  # code 0 where nothing was written
    return {"latent": _place(s, blocks, _e4m3(t / torch.exp2(e)[:, :, None]).view(-1, LATENT)),
            "pe": _place(s, blocks, _turn(x[:, LATENT:], s)), "scale": scale}


def _exact_tokens(cache, bs, slot):
    rows = cache[slot // bs]
    off = (slot % bs)[:, None]
    byte = torch.arange(644, device=cache.device)[None]
    at = torch.where(byte < 512, off * 512 + byte,
                     torch.where(byte < 640, 512 * bs + off * 128 + byte - 512, 640 * bs + off * 4 + byte - 640))
    rec = rows.gather(1, at)
    v = rec[:, :512].int()
    exp, man = (v >> 3) & 15, (v & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(exp.double() - 10))
    lat = torch.where(v >= 128, -mag, mag).view(-1, 4, 128) * torch.exp2(rec[:, 640:].double() - 127)[:, :, None]
    return torch.cat([lat.view(-1, 512), rec[:, 512:640].contiguous().view(torch.bfloat16).double()], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "k_insert":
        return _exact_k_insert(s)
    if op == "kv_insert":
        return _exact_kv_insert(s)
    if op == "kv_gather":
        cu, bt = s["cu"].tolist(), s["block_table"].long()
        parts = []
        for b in range(len(cu) - 1):
            for at in range(0, cu[b + 1] - cu[b], 4096):
                p = torch.arange(at, min(at + 4096, cu[b + 1] - cu[b]), device=bt.device)
                parts.append(_exact_tokens(s["cache"], s["bs"], bt[b, p // s["bs"]] * s["bs"] + p % s["bs"]))
        return torch.cat(parts)
    outs, lses = [], []
    for t in range(s["q"].shape[0]):
        slot = s["slots"][t].long()
        slot = slot[slot >= 0]
        if slot.numel() == 0:
            outs.append(torch.zeros(s["q"].shape[1], LATENT, dtype=torch.float64, device=slot.device))
            lses.append(torch.full((s["q"].shape[1],), -math.inf, dtype=torch.float64, device=slot.device))
            continue
        k = _exact_tokens(s["cache"], s["bs"], slot)
        z = s["q"][t].double() @ k.T * s["scale"]
        lse = torch.logsumexp(z, dim=1)
        outs.append(torch.exp(z - lse[:, None]) @ k[:, :LATENT])
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
