"""Step tables, trees of drafted tokens and attention over whole contexts, on the host.

Integers are computed request by request, as a scheduler would; attention in fp64, row by row over the list of
tokens that the row sees, with the error bounds of ``attention.sparse_attention_row``.
"""

from __future__ import annotations

import numpy as np

from .attention import sparse_attention_row
from .codecs import bf16_decode, e4m3_decode


def build_tables(cached, new, free, table, block_size, n_rows, held=None, start=0):
    """The outputs of one step as a dict of int64 arrays; ``table`` is copied. Inputs are in range."""
    table = np.array(table, dtype=np.int64)
    B, pages = table.shape
    held = [min(-(-c // block_size), pages) for c in cached] if held is None else [int(h) for h in held]
    at = int(start)
    ctx, rows = [], []
    for b in range(B):
        ctx.append(int(cached[b]) + int(new[b]))
        want = min(-(-ctx[b] // block_size), pages)
        for page in range(held[b], want):
            if at < len(free):
                table[b, page] = free[at]
                at += 1
                held[b] += 1
            else:
                table[b, page] = -1
        for p in range(int(cached[b]), ctx[b]):
            page = p // block_size
            block = table[b, page] if page < pages else -1
            rows.append((p, block * block_size + p % block_size if block >= 0 else -1, b, p + 1))
    cu = np.concatenate([[0], np.cumsum(np.asarray(new, dtype=np.int64))])
    rows = (rows + [(0, -1, 0, 0)] * n_rows)[:n_rows]
    pos, slot, req, ke = (np.array([r[k] for r in rows], dtype=np.int64) for k in range(4))
    return {"table": table, "ctx_lens": np.array(ctx, dtype=np.int64), "cu_rows": cu,
            "cu_ctx": np.concatenate([[0], np.cumsum(np.array(ctx, dtype=np.int64))]),
            "held": np.array(held, dtype=np.int64), "free_end": at, "positions": pos, "slots": slot,
            "row_to_req": req, "row_ke": ke}


def tree_sets(parents):
    """For each node of one tree the set of itself and its ancestors."""
    sets = []
    for i, up in enumerate(int(p) for p in parents):
        sets.append({i} | (sets[up] if 0 <= up < i else set()))
    return sets


def mask_words(sets, words):
    """int32 [n, words] with bit m % 32 of word m / 32 set for every m of a row's set."""
    out = np.zeros((len(sets), words), dtype=np.uint32)
    for i, s in enumerate(sets):
        for m in s:
            if m < 32 * words:
                out[i, m // 32] |= np.uint32(1) << np.uint32(m % 32)
    return out.view(np.int32)


def window_seen(p, window, sinks):
    """Tokens that a row at position ``p`` sees."""
    return [j for j in range(p + 1) if j > p - window or j < sinks]


def tree_seen(base, n, words_of_row):
    """Tokens that a node sees: all before ``base``, and of its n nodes those whose bit is set."""
    w = np.asarray(words_of_row, dtype=np.int32).view(np.uint32)
    return list(range(max(base, 0))) + [base + m for m in range(n) if base + m >= 0 and m < 32 * len(w)
                                        and (int(w[m // 32]) >> (m % 32)) & 1]


def context(cache, block_size, block_table_row, ctx):
    """[ctx, 576] values of a request's tokens; rows of NaN for tokens whose page is outside the cache."""
    out = np.full((ctx, 576), np.nan)
    for page in range(-(-ctx // block_size)):
        n = min(block_size, ctx - page * block_size)
        blk = int(block_table_row[page]) if page < len(block_table_row) else -1
        if blk < 0 or blk >= len(cache):
            continue
        rec = cache[blk]
        lat = e4m3_decode(rec[:512 * block_size].reshape(block_size, 512)[:n])
        pe = bf16_decode(rec[512 * block_size:640 * block_size].copy().view(np.uint16).reshape(block_size, 64)[:n])
        sc = rec[640 * block_size:644 * block_size].reshape(block_size, 4)[:n]
        scale = np.where(sc == 255, np.nan, np.exp2(sc.astype(np.float64) - 127))
        out[page * block_size:page * block_size + n] = np.concatenate([lat * np.repeat(scale, 128, axis=1), pe], axis=1)
    return out


def attention(q, tokens_of, seen_of, softmax_scale):
    """(out, lse, out_err, lse_err) of every row: ``tokens_of(t)`` is its request's context, ``seen_of(t)`` its tokens."""
    rows = []
    for t in range(len(q)):
        rows.append(sparse_attention_row(q[t], tokens_of(t)[seen_of(t)], softmax_scale))
    return tuple(np.stack(x) for x in zip(*rows))
