"""Normalised inserts, the attention cache and the sparse attention that reads it, in fp64.

[DSA] "Indexer 内部六步" steps ②, ③ and ⑤ (k_norm, RoPE, quantisation fused with the
insert) and data-flow items 2-3 (the selection hands the main attention a slot
list). Everything is evaluated in fp64; where a quantisation follows, both the
value before it and the error that binary32 evaluation may add to it are
returned, so a check can accept exactly the codes that some value within that
error rounds to.
"""

from __future__ import annotations

import numpy as np

from .codecs import bf16_decode, e4m3_decode
from .indexer import rope_pairs

U = 2.0 ** -24          # half a binary32 step, relative
LATENT, ROPE = 512, 64
TOKEN_BYTES = 644
MAX_SCALE_EXP = 7


def rotate(x, positions, cos_sin, interleaved):
    """``x`` [n, 64] with its 32 pairs turned by the angles of each position; zeros outside the table."""
    x = np.asarray(x, dtype=np.float64)
    cs = np.asarray(cos_sin, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.int64)
    ok = (pos >= 0) & (pos < cs.shape[0])
    row = cs[np.where(ok, pos, 0)]
    c, s = row[:, :32], row[:, 32:64]
    a, b = rope_pairs(interleaved)
    y = x.copy()
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    y[~ok] = 0.0
    return y, ok


def k_norm_rope(x, weight, bias, eps, positions, cos_sin, interleaved):
    """LayerNorm and partial RoPE of the indexer's k: (y, err) [n, 128], err bounding binary32's error.

    The error, with u = 2^-24, X = max |x|, d = x - mean, s = sqrt(var + eps): the mean (a tree of seven
    additions) is within 8 u X, so d is within 10 u X; the variance is then within (20 X / s + 9) u
    relative, its reciprocal root within (10 X / s + 8) u, and y before the rotation within
    |w| / s * 10 u X + |w d| / s * (10 X / s + 11) u + u |y|. The rotation adds both members'
    errors and two roundings of each product.
    """
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(weight, dtype=np.float64)
    b = np.zeros(128) if bias is None else np.asarray(bias, dtype=np.float64)
    d = x - x.mean(axis=1, keepdims=True)
    s = np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    y = d / s * w + b
    X = np.abs(x).max(axis=1, keepdims=True)
    err = np.abs(w) / s * 10 * U * X + np.abs(w * d) / s * (10 * X / s + 11) * U + U * np.abs(y)
    rot, ok = rotate(y[:, :64], positions, cos_sin, interleaved)
    pa, pb = rope_pairs(interleaved)
    rerr = np.zeros((len(y), 64))
    both = err[:, pa] + err[:, pb] + 2 * U * (np.abs(y[:, pa]) + np.abs(y[:, pb]))
    rerr[:, pa] = both
    rerr[:, pb] = both
    y = np.concatenate([rot, y[:, 64:]], axis=1)
    err = np.concatenate([rerr, err[:, 64:]], axis=1)
    y[~ok] = 0.0
    err[~ok] = 0.0
    return y, err


def kv_norm(c, weight, eps):
    """RMSNorm of the latent: (y, err) [n, 512]. Sixteen serial and five tree additions of squares, the
    root, the quotient and two products stay within 16 u relative. weight None: y = c, exact."""
    c = np.asarray(c, dtype=np.float64)
    if weight is None:
        return c, np.zeros_like(c)
    y = c / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    return y, 16 * U * np.abs(y)


def kv_scale_exponent(amax) -> np.ndarray:
    """Exponent of the smallest power of two >= amax / 448 (the binary32 quotient), held to [-127, 7]."""
    q = (np.asarray(amax, dtype=np.float32) / np.float32(448)).astype(np.float64)
    m, e = np.frexp(q)
    e = np.where(m == 0.5, e - 1, e)
    return np.clip(np.where(q == 0, -127, e), -127, MAX_SCALE_EXP).astype(np.int64)


def kv_record(cache, block_size, slot):
    """(e4m3 codes [512], position dims [64] as bf16 bits, scale codes [4]) of one slot."""
    blk, off = divmod(int(slot), block_size)
    row = cache[blk]
    pe = row[512 * block_size + 128 * off:512 * block_size + 128 * off + 128]
    at = 640 * block_size + 4 * off
    return row[512 * off:512 * off + 512], pe.copy().view(np.uint16), row[at:at + 4]


def kv_put(cache, block_size, slot, codes, pe_bits, scale_codes):
    """Write one record (the inverse of ``kv_record``)."""
    blk, off = divmod(int(slot), block_size)
    row = cache[blk]
    row[512 * off:512 * off + 512] = codes
    row[512 * block_size + 128 * off:512 * block_size + 128 * off + 128] = np.asarray(pe_bits, np.uint16).view(np.uint8)
    row[640 * block_size + 4 * off:640 * block_size + 4 * off + 4] = scale_codes


def kv_token(cache, block_size, slot) -> np.ndarray:
    """The 576 dims that one slot stands for; NaN under scale code 255."""
    codes, pe, sc = kv_record(cache, block_size, slot)
    scale = np.where(sc == 255, np.nan, np.exp2(sc.astype(np.float64) - 127))
    return np.concatenate([e4m3_decode(codes) * np.repeat(scale, 128), bf16_decode(pe).astype(np.float64)])


def gather_kv(cache, block_size, block_table, cu_lens, starts=None) -> np.ndarray:
    """Packed read-back [cu_lens[-1], 576] (rows before cu_lens[0] are zero)."""
    cu = [int(c) for c in cu_lens]
    out = np.zeros((cu[-1], 576))
    for b in range(len(cu) - 1):
        for r in range(cu[b], cu[b + 1]):
            p = r - cu[b] + (0 if starts is None else int(starts[b]))
            blk = int(block_table[b][p // block_size])
            out[r] = kv_token(cache, block_size, blk * block_size + p % block_size)
    return out


def sparse_attention_row(q, tokens, softmax_scale):
    """Attention of one row's heads ``q`` [H, 576] over ``tokens`` [n, 576].

    Returns (out [H, 512], lse [H], out_err, lse_err): the last two bound what binary32 evaluation with the
    weights rounded once to bf16 may differ by. With A = |scale| max_j sum_d |q_d k_jd|, a logit summed in
    binary32 by an adder that may truncate is within 578 * 2^-23 A (576 terms and two products); a weight
    within e^(2 delta) - 1 of its value (its own logit and the maximum's), 2^-8 more after bf16, 2^-21
    for the exponential; sums of n terms add n 2^-23; joining parts of a list a few more roundings.
    """
    q = np.asarray(q, dtype=np.float64)
    H, n = len(q), len(tokens)
    if n == 0:
        return np.zeros((H, LATENT)), np.full(H, -np.inf), np.zeros((H, LATENT)), np.zeros(H)
    z = q @ tokens.T * softmax_scale
    A = abs(softmax_scale) * (np.abs(q) @ np.abs(tokens).T).max(axis=1)
    top = z.max(axis=1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(axis=1, keepdims=True)
    out = p @ tokens[:, :LATENT] / total
    spread = p @ np.abs(tokens[:, :LATENT]) / total
    lse = (np.log(total) + top)[:, 0]
    delta = 578 * 2.0 ** -23 * A
    rel = np.expm1(4 * delta) + 2.0 ** -8 + 2.0 ** -20 + 2 * n * 2.0 ** -23
    out_err = spread * rel[:, None] + 2.0 ** -8 * np.abs(out) * (1 + rel[:, None])
    lse_err = 2 * delta + n * 2.0 ** -23 + 2.0 ** -20 + 8 * U * np.abs(lse)
    return out, lse, out_err, lse_err


def sparse_attention(q, cache, block_size, slots, softmax_scale, n_sel=None, block_span=None):
    """``sparse_attention_row`` for every row; entries that are negative or outside the cache are skipped."""
    span = block_size if block_span is None else block_span
    rows = []
    for t in range(len(q)):
        lst = slots[t] if n_sel is None else slots[t][:max(0, int(n_sel[t]))]
        tok = [kv_token(cache, block_size, (v // span) * block_size + v % span) for v in map(int, lst)
               if v >= 0 and v // span < len(cache) and v % span < block_size]
        rows.append(sparse_attention_row(q[t], np.array(tok).reshape(len(tok), 576), softmax_scale))
    return tuple(np.stack(x) for x in zip(*rows))
