"""Window and tree attention where the work is shared out and joined, and at the edges of what a call may be given."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from test_gpu_paged_attention import Case, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def flagged():
    with pytest.raises(idx.IdxError, match="tree attention 0x00000001"):
        idx.idx_device_error()
    idx.idx_device_error()


# ------------------------------------------------------------------ pages that no node sees

@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("with_ws", [False, True])
def test_pages_of_nodes_that_no_row_sees_may_be_missing(H, with_ws):
    """Nodes without a bit, and nodes whose bit no row has set: their pages need no block, in the table or behind it."""
    bs, n, base = 16, 70, 600
    c = Case(H, [n, 2], [base + n, 40], bs, seed=31, extra_pages=3)
    ws = c.workspace() if with_ws else None
    first = -(-base // bs)                       # the first page of nodes alone: node 8 (600 is 8 tokens into a page)
    full = c.block_table.clone()
    last = (base + n - 1) // bs
    for missing in (-1, 2 ** 31 - 1, c.cache.shape[0]):
        c.block_table = full.clone()
        c.block_table[0, first:last + 1] = missing
        none = torch.zeros((c.T, 0), dtype=torch.int32, device=DEV)
        c.tree(none, ws=ws)                      # no words at all
        idx.idx_device_error()
        c.check(c.tree_seen(none))
        bits = np.zeros((c.T, 3), dtype=np.int32)
        bits[:, 0] = 0xFF                        # the nodes of the page that holds earlier tokens too
        c.tree(i32(bits), ws=ws)
        idx.idx_device_error()
        c.check(c.tree_seen(i32(bits)))
        bits[37, 1] = 1 << 9                     # one row sees node 41, on the page that begins with node 40
        c.tree(i32(bits), ws=ws)
        flagged()
        seen = c.tree_seen(i32(bits))
        c.check(lambda b, i: [j for j in seen(b, i) if b or j < base + 8])
        c.block_table[0, (base + 41) // bs] = full[0, (base + 41) // bs]
        c.tree(i32(bits), ws=ws)                 # with that page all is well
        idx.idx_device_error()
        c.check(seen)
    # nodes behind the words, whose pages the table does not even have
    c.block_table = full[:, :(base + 32) // bs + 1].contiguous()
    bits = np.random.default_rng(1).integers(-2 ** 31, 2 ** 31 - 1, (c.T, 1))
    bits[:, 0] &= 0xFFFFFF
    c.tree(i32(bits), ws=ws)
    idx.idx_device_error()
    c.check(c.tree_seen(i32(bits)))
    # and one that a row sees: node 60 in word 1, behind the table
    wide = np.concatenate([bits, np.zeros_like(bits)], axis=1)
    wide[50, 1] = 1 << 28
    c.tree(i32(wide), ws=ws)
    flagged()
    c.check(c.tree_seen(i32(bits)))


@pytest.mark.parametrize("with_ws", [False, True])
@pytest.mark.parametrize("pages", [2, 40])
def test_first_tokens_of_a_context_at_the_end_of_32_bits(pages, with_ws):
    """Every token is one of the first, and the context is longer than its table: what the table has counts."""
    c = Case(64, [1, 1], [64 * pages, 64 * pages], 64, seed=41)
    have = list(c.ctxs)
    c.ctxs = [2 ** 31 - 1, 64 * pages]
    c.window(2 ** 31 - 1, 2 ** 31 - 1, ws=c.workspace() if with_ws else None)
    flagged()
    c.ctxs = have
    c.check(lambda b, i: list(range(64 * pages)))


@pytest.mark.parametrize("op", ["window", "tree"])
@pytest.mark.parametrize("H,counts,ctxs,cu", [
    (128, [1] * 5, [900, 40, 300, 1000, 77], [0, 200, 260, 50, 60, 55]),       # shared out, or whole units in turn
    (16, [1] * 5, [900, 40, 300, 1000, 77], [250, 0, 250, 10, 240, 3]),
    (64, [1] * 170, [100] * 170, [(7 * b) % 251 for b in range(171)]),          # a block for each unit
    (3, [1] * 3, [500, 500, 500], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -5])])
def test_row_ranges_that_do_not_ascend_stay_inside(op, H, counts, ctxs, cu):
    """Such a call's results mean nothing, but it ends, and touches none but the rows that some range names."""
    c = Case(H, counts, ctxs, 64, seed=51, extra_pages=20)
    T, rows = 270, 261
    c.q = torch.randn(T, H, 576, device=DEV).bfloat16()
    out, lse = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, H), 7.0, device=DEV)
    mask = torch.full((T, 1), -1, dtype=torch.int32, device=DEV)[:rows]
    n = idx.idx_paged_attention_workspace_bytes(rows, len(counts), H)
    for ws in (None, torch.empty(n + 4096, dtype=torch.uint8, device=DEV)):
        guard = None if ws is None else ws[n:].fill_(171)
        part = None if ws is None else ws[:n]
        if op == "window":
            idx.idx_window_attention(c.q[:rows], c.cache, 64, c.block_table, i32(cu), i32(c.ctxs), out[:rows], 0.07, 2 ** 20, lse=lse[:rows], ws=part)
        else:
            idx.idx_tree_attention(c.q[:rows], c.cache, 64, c.block_table, i32(cu), i32(c.ctxs), mask, out[:rows], 0.07, lse=lse[:rows], ws=part)
        idx.idx_device_error()
        last = min(max(cu), rows)
        assert (out[last:] == 7).all() and (lse[last:] == 7).all()
        assert guard is None or (guard == 171).all()
    # the next call is right
    c = Case(H, counts, ctxs, 64, seed=52, extra_pages=20)
    c.window(100, 3, ws=c.workspace())
    idx.idx_device_error()
    c.check(c.window_seen(100, 3))
