"""Window and tree attention where the work is shared out and joined, and at the edges of what a call may be given."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from test_gpu_paged_attention import SCALE, Case, i32, random_mask

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


# ------------------------------------------------------------------ contexts that are cut and joined

def shared_out(c, ws, call):
    """Whether ``call`` shares the work out, which shows in the workspace: every worker notes its cut there."""
    ws.fill_(255)
    call(ws)
    return bool((ws != 255).any())


def both(c, call, check):
    """With the work shared out, which must have happened, and without; the results of the first are returned."""
    ws = c.workspace()
    assert shared_out(c, ws, call)
    check()
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(7)
    c.lse.fill_(7)
    call(None)
    check()
    return first


@pytest.mark.parametrize("H,counts,ctxs,window,sinks,bs", [
    (128, [1, 2, 1], [3000, 1700, 900], 1024, 4, 64), (16, [1] * 16, [100 + 301 * b for b in range(16)], 1024, 0, 16),
    (20, [37, 1, 0, 5], [1300, 1, 10, 2777], 1100, 7, 16), (64, [3, 2, 4], [2100, 64, 1290], 640, 200, 128),
    (65, [2, 1], [2500, 2500], 2000, 0, 32), (3, [21, 40], [999, 5000], 777, 130, 64), (1, [64, 1], [4000, 4000], 3999, 1, 64),
    (300, [1], [900], 513, 1, 16)])
def test_windows_that_are_cut(H, counts, ctxs, window, sinks, bs):
    """Ragged requests, their windows shorter than their contexts, some contexts shorter than the window."""
    c = Case(H, counts, ctxs, bs, seed=H + 60, before=2, behind=3)
    both(c, lambda ws: c.window(window, sinks, ws=ws), lambda: c.check(c.window_seen(window, sinks)))
    idx.idx_device_error()


@pytest.mark.parametrize("H", [8, 128])
@pytest.mark.parametrize("op", ["window", "tree"])
def test_strides_of_rows_that_are_joined(op, H):
    """Slices of larger tensors; what lies between stays."""
    c = Case(H, [5, 9], [900, 777], 64, seed=63)
    qb = torch.full((c.T, H + 2, 600), float("nan"), dtype=torch.bfloat16, device=DEV)
    qb[:, 1:-1, 8:584] = c.q
    ob = torch.full((c.T, H + 3, 528), 5.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((c.T, H + 1), 5.0, dtype=torch.float32, device=DEV)
    tb = torch.full((2, c.block_table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    tb[:, :-3] = c.block_table
    masks = torch.full((c.T, 4), -1, dtype=torch.int32, device=DEV)
    masks[:, 1:3] = random_mask(c.counts, 2, np.random.default_rng(4))
    cu, ctx = i32(c.cu), i32(c.ctxs)

    def call(ws):
        if op == "window":
            idx.idx_window_attention(qb[:, 1:-1, 8:584], c.cache, 64, tb[:, :-3], cu, ctx, ob[:, 2:-1, 8:520], SCALE, 600,
                                     sinks=2, lse=lb[:, 1:], ws=ws)
        else:
            idx.idx_tree_attention(qb[:, 1:-1, 8:584], c.cache, 64, tb[:, :-3], cu, ctx, masks[:, 1:3], ob[:, 2:-1, 8:520],
                                   SCALE, lse=lb[:, 1:], ws=ws)
        c.out, c.lse = ob[:, 2:-1, 8:520].contiguous(), lb[:, 1:].contiguous()

    both(c, call, lambda: c.check(c.window_seen(600, 2) if op == "window" else c.tree_seen(masks[:, 1:3])))
    idx.idx_device_error()
    ob[:, 2:-1, 8:520] = 5.0
    assert (ob == 5).all() and (lb[:, 0] == 5).all()
    # heads outside, rows inside
    qb = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    ob = torch.zeros(H, c.T, 512, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    ws = c.workspace()
    idx.idx_window_attention(qb, c.cache, 64, c.block_table, cu, ctx, ob, SCALE, 600, sinks=2, ws=ws)
    idx.idx_device_error()
    c.out, c.lse = ob.contiguous(), torch.full_like(c.lse, 7.0)
    idx.idx_window_attention(qb, c.cache, 64, c.block_table, cu, ctx, c.out, SCALE, 600, sinks=2, lse=c.lse, ws=ws)
    assert torch.equal(c.out, ob)
    c.check(c.window_seen(600, 2))


def poison(c, b, j, kind):
    rec, bs, off = c.cache[int(c.table[b, j // c.bs])], c.bs, j % c.bs
    if kind == "latent":
        rec[640 * bs + 4 * off + 2] = 255
        rec[512 * off + 256:512 * off + 384] = 0
    else:
        rec[512 * bs + 128 * off:512 * bs + 128 * off + 2] = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("kind", ["latent", "position"])
@pytest.mark.parametrize("H,rows", [(128, 6), (16, 24), (3, 50), (64, 40)])
def test_tokens_that_are_not_finite_in_cut_contexts(H, rows, kind):
    """A NaN token in one part makes the rows that see it NaN, through the join, and no other row."""
    window, ctx, bs = 1200, 2000, 16
    c = Case(H, [rows, 1], [ctx, 1300], bs, seed=64)
    p0 = ctx - rows                                # position of the first row
    poison(c, 0, p0 - window + 3, kind)            # seen by rows 0, 1 and 2
    poison(c, 0, ctx - 2, kind)                    # by the last two
    poison(c, 0, 100, kind)                        # by none
    bad = [0, 1, 2, rows - 2, rows - 1]
    clean = [t for t in range(rows + 1) if t not in bad]

    def check():
        assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
        c.check(c.window_seen(window, 2), clean)

    both(c, lambda ws: c.window(window, 2, ws=ws), check)
    idx.idx_device_error()
    # of drafted nodes: seen by itself and by those below it
    mask = random_mask(c.counts, 2, np.random.default_rng(H))
    base = ctx - rows
    c = Case(H, [rows, 1], [ctx, 1300], bs, seed=65)
    poison(c, 0, base + 1, kind)
    seen = c.tree_seen(mask)
    bad = [i for i in range(rows) if base + 1 in seen(0, i)]
    clean = [t for t in range(rows + 1) if t not in bad]
    assert bad and len(clean) > 1

    def check_tree():
        assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
        c.check(seen, clean)

    both(c, lambda ws: c.tree(mask, ws=ws), check_tree)
    idx.idx_device_error()


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("bs", [16, 128])
def test_pages_that_are_missing_in_cut_contexts(H, bs):
    """Single pages, all pages of several tiles, the first and the last, and the end of the table."""
    c = Case(H, [3, 2], [3000, 1400], bs, seed=66)
    pages = 3000 // bs
    gone = {0: {0, 3} | set(range(pages // 4, pages // 2)), 1: {0, 1400 // bs}}
    c.block_table[0, sorted(gone[0])] = i32([[-1, c.cache.shape[0], -2 ** 31, 2 ** 31 - 1][i % 4] for i in range(len(gone[0]))])
    c.block_table[1, sorted(gone[1])] = -1
    mask = i32(np.full((5, 1), -1))
    full = c.tree_seen(mask)

    def check(seen):
        flagged()
        c.check(lambda b, i: [j for j in seen(b, i) if j // bs not in gone[b]])

    both(c, lambda ws: c.tree(mask, ws=ws), lambda: check(full))
    both(c, lambda ws: c.window(2900, 5, ws=ws), lambda: check(c.window_seen(2900, 5)))
    # pages behind the window may be missing without an error
    first = (3000 - 3) - 1200 + 1
    c = Case(H, [3], [3000], bs, seed=67)
    dead = [p for p in range(pages) if p > 4 // bs and (p + 1) * bs <= first]
    c.block_table[0, dead] = -1
    both(c, lambda ws: c.window(1200, 5, ws=ws), lambda: c.check(c.window_seen(1200, 5)))
    idx.idx_device_error()
    # a context longer than its table
    c = Case(H, [3], [3000], bs, seed=68)
    c.block_table = c.block_table[:, :2048 // bs].contiguous()

    def check_short():
        flagged()
        c.check(lambda b, i: list(range(2048)))

    both(c, lambda ws: c.window(10 ** 6, 0, ws=ws), check_short)


def test_rows_that_see_nothing_in_cut_contexts():
    """Requests without a context, rows before a context's first token, masks without a bit, beside long contexts."""
    c = Case(16, [1, 1, 5, 2, 0, 3], [0, 1900, 3, -4, 77, 1000], 16, seed=69)
    empty = [0, 2, 3, 7, 8]
    both(c, lambda ws: c.window(900, 1, ws=ws), lambda: c.check(c.window_seen(900, 1)))
    assert not c.out[empty].any() and torch.isneginf(c.lse[empty]).all()
    mask = i32(np.full((c.T, 1), -1))
    both(c, lambda ws: c.tree(mask, ws=ws), lambda: c.check(c.tree_seen(mask)))
    idx.idx_device_error()
    # a request of nodes alone, over ten tiles: some see nothing at all, some nothing of most parts
    c = Case(16, [600, 2], [600, 300], 64, seed=70, extra_pages=40)
    words = np.zeros((c.T, 19), dtype=np.int64)
    rng = np.random.default_rng(7)
    words[200:400] = rng.integers(-2 ** 31, 2 ** 31 - 1, (200, 19))
    words[100:150, 7] = 1 << 4
    words[550:600, 18] = 1
    mask = i32(words)
    both(c, lambda ws: c.tree(mask, ws=ws), lambda: c.check(c.tree_seen(mask)))
    idx.idx_device_error()
    assert not c.out[:100].any() and torch.isneginf(c.lse[400:550]).all()


def test_masks_of_any_bits_in_cut_contexts():
    c = Case(20, [40, 3, 70], [640, 3, 900], 16, seed=71)
    words = np.random.default_rng(8).integers(-2 ** 31, 2 ** 31 - 1, (c.T, 2))
    words[3] = 0
    for mask in (i32(words), torch.zeros((c.T, 0), dtype=torch.int32, device=DEV), i32(np.full((c.T, 32), -1))[:, :31]):
        both(c, lambda ws: c.tree(mask, ws=ws), lambda: c.check(c.tree_seen(mask)))
    idx.idx_device_error()


# ------------------------------------------------------------------ whole units in turn

@pytest.mark.parametrize("with_ws", [False, True])
@pytest.mark.parametrize("H,counts,ctxs,window,sinks,bs", [
    (128, [40, 30, 20], [300, 100, 700], 90, 4, 64),             # two units a row, 186 in all, of ragged windows
    (128, [100, 0, 70], [100, 50, 70], 2 ** 31 - 1, 0, 16),      # prompts from their first token
    (16, [500, 0, 203], [900, 10, 203], 200, 7, 32), (64, [160, 1], [161, 500], 40, 0, 128), (33, [70, 90, 3], [800, 90, 64], 130, 65, 16),
    (5, [12] * 155, [20 + 5 * b for b in range(155)], 100, 2, 64), (200, [50], [600], 600, 0, 64)])
def test_windows_of_whole_units_in_turn(H, counts, ctxs, window, sinks, bs, with_ws):
    """More units than the GPU has blocks: each takes several, the last rows' first, and fetches one while it ends another."""
    c = Case(H, counts, ctxs, bs, seed=H + 80, before=1, behind=2)
    c.window(window, sinks, ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    c.check(c.window_seen(window, sinks))


def test_tokens_that_are_not_finite_with_units_in_turn():
    """A unit's NaN tokens leave nothing behind for the block's next unit."""
    c = Case(128, [120, 60], [400, 90], 64, seed=90)
    p0 = 400 - 120
    for j in (p0 + 10, p0 + 70):
        poison(c, 0, j, "latent")
    window = 20
    bad = [i for i in range(120) if any(p0 + i - window < j <= p0 + i for j in (p0 + 10, p0 + 70))]
    c.window(window, 0)
    idx.idx_device_error()
    assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
    c.check(c.window_seen(window, 0), [t for t in range(180) if t not in bad])


@pytest.mark.parametrize("op", ["window", "tree"])
@pytest.mark.parametrize("H,counts", [(16, [3, 0, 1, 7] * 50), (64, [1] * 200)])
def test_more_requests_than_share_their_work(op, H, counts):
    ctxs = [max(n, (37 * b) % 400) for b, n in enumerate(counts)]
    c = Case(H, counts, ctxs, 32, seed=91, before=1, behind=1)
    assert c.workspace() is None
    if op == "window":
        c.window(150, 3)
        c.check(c.window_seen(150, 3))
    else:
        mask = random_mask(counts, 1, np.random.default_rng(2), 1, 1)
        c.tree(mask)
        c.check(c.tree_seen(mask))
    idx.idx_device_error()


# ------------------------------------------------------------------ captured calls that share their work

def test_captured_calls_that_are_cut():
    """Two calls with one workspace in a graph, and a second graph with its own: replayed back to back, on two streams at
    once, beside an eager call, over lengths that change between replays."""
    made = [[Case(128, [2, 1], [2600, 1500], 64, seed=100), Case(16, [8, 5], [1800, 2900], 64, seed=101)],
            [Case(64, [1] * 6, [900 + 300 * b for b in range(6)], 64, seed=102), Case(20, [9], [5000], 64, seed=103)],
            [Case(128, [4], [3000], 64, seed=104), Case(16, [3], [4000], 64, seed=105)]]
    for k, pair in enumerate(made):
        size = max(idx.idx_paged_attention_workspace_bytes(c.T, len(c.counts), c.H) for c in pair)
        for c in pair:
            c.ws = torch.empty(size, dtype=torch.uint8, device=DEV) if c is pair[0] else pair[0].ws
            c.cu_dev, c.ctx_dev, c.full = i32(c.cu), i32(c.ctxs), list(c.ctxs)
        pair[1].mask = random_mask(pair[1].counts, 1, np.random.default_rng(k))

    def run(pair, stream=None):
        a, b = pair
        idx.idx_window_attention(a.q, a.cache, a.bs, a.block_table, a.cu_dev, a.ctx_dev, a.out, SCALE, 1100, sinks=4, lse=a.lse,
                                 ws=a.ws, stream=stream)
        idx.idx_tree_attention(b.q, b.cache, b.bs, b.block_table, b.cu_dev, b.ctx_dev, b.mask, b.out, SCALE, lse=b.lse, ws=b.ws,
                               stream=stream)

    for pair in made:
        for c in pair:
            call = (lambda ws, c=c: c.window(1100, 4, ws=ws)) if c is pair[0] else (lambda ws, c=c: c.tree(c.mask, ws=ws))
            assert shared_out(c, c.ws, call)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    graphs = []
    for pair, s in zip(made[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(pair)
            run(pair)  # the next call's parts overwrite those that the last one joined
        graphs.append(g)
    for cut in (0, 333, 70, 0):
        for pair in made:
            for c in pair:
                c.ctxs = [max(n, x - cut) for n, x in zip(c.counts, c.full)]
                c.ctx_dev.copy_(i32(c.ctxs))
                c.out.fill_(7)
                c.lse.fill_(7)
                c.ws.fill_(255)
        torch.cuda.synchronize()
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            run(made[2], streams[2])
        torch.cuda.synchronize()
        idx.idx_device_error()
        for a, b in made:
            a.check(a.window_seen(1100, 4))
            b.check(b.tree_seen(b.mask))
