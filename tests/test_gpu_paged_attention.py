"""Window and tree attention against the fp64 oracle, element by element within the bounds that it derives."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import paged as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def stride_of(bs):
    return -(-bs * 644 // 512) * 512


def random_cache(blocks, bs, g):
    """Every token a quantised random latent, scales that differ from tile to tile."""
    cache = torch.zeros(blocks, stride_of(bs), dtype=torch.uint8, device=DEV)
    lat = torch.randn(blocks * bs, 4, 128, generator=g, device=DEV)
    lat = lat * torch.exp(0.5 * torch.randn(blocks * bs, 4, 1, generator=g, device=DEV))
    code = torch.ceil(torch.log2(lat.abs().amax(dim=2) / 448)).clamp(-127, 7)
    val = (lat / torch.exp2(code)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[:, :512 * bs] = val.view(blocks, bs * 512)
    cache[:, 512 * bs:640 * bs] = torch.randn(blocks, bs * 64, generator=g, device=DEV).bfloat16().view(torch.uint8)
    cache[:, 640 * bs:644 * bs] = (code + 127).to(torch.uint8).view(blocks, bs * 4)
    return cache


class Case:
    """Requests with ``counts`` new rows and ``ctxs`` tokens, their blocks anywhere in the cache; pages beyond a
    context and blocks of nobody hold bytes of any kind."""

    def __init__(self, H, counts, ctxs, bs, seed=0, before=0, behind=0, spread=2.0, extra_pages=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.H, self.counts, self.ctxs, self.bs = H, list(counts), list(ctxs), bs
        need = [-(-max(c, 0) // bs) for c in ctxs]
        blocks = sum(need) + 5
        self.cache = random_cache(blocks, bs, g)
        ids = rng.permutation(blocks)
        pages = max(need + [1]) + extra_pages
        self.table = rng.integers(-2 ** 31, 2 ** 31 - 1, (len(need), pages))  # nothing that may be looked up
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
            if n and ctxs[b] % bs:  # behind the last token: NaN bytes and NaN scales
                blk, off = int(ids[at - 1]), ctxs[b] % bs
                rec = self.cache[blk]
                rec[512 * off:512 * bs] = 255
                rec[512 * bs + 128 * off:640 * bs] = 255
                rec[640 * bs + 4 * off:644 * bs] = 255
        for blk in ids[at:]:
            self.cache[int(blk)] = 255
        self.cu = np.concatenate([[0], np.cumsum(self.counts)]) + before
        self.T = int(self.cu[-1]) + behind
        self.q = (spread * torch.randn(self.T, H, 576, generator=g, device=DEV)).bfloat16()
        self.block_table = i32(self.table)
        self.out = torch.full((self.T, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, H), 7.0, dtype=torch.float32, device=DEV)

    def workspace(self):
        n = idx.idx_paged_attention_workspace_bytes(self.T, len(self.counts), self.H)
        return torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None

    def window(self, window, sinks, ws=None, **kw):
        idx.idx_window_attention(self.q, self.cache, self.bs, self.block_table, i32(self.cu), i32(self.ctxs), self.out, SCALE,
                                 window, sinks=sinks, lse=self.lse, ws=ws, **kw)

    def tree(self, mask, ws=None, **kw):
        idx.idx_tree_attention(self.q, self.cache, self.bs, self.block_table, i32(self.cu), i32(self.ctxs), mask, self.out,
                               SCALE, lse=self.lse, ws=ws, **kw)

    def rows(self):
        return [(b, i) for b, n in enumerate(self.counts) for i in range(n)]

    def want(self, seen):
        """``seen(b, i)``: the tokens that row i of request b sees."""
        cache = self.cache.cpu().numpy()
        tokens = [P.context(cache, self.bs, self.table[b], max(c, 0)) for b, c in enumerate(self.ctxs)]
        rows = self.rows()
        q = self.q.double().cpu().numpy()[self.cu[0]:self.cu[-1]]
        return P.attention(q, lambda t: tokens[rows[t][0]], lambda t: seen(*rows[t]), SCALE)

    def check(self, seen, rows=None):
        out, lse, oerr, lerr = self.want(seen)
        got, glse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        a, z = int(self.cu[0]), int(self.cu[-1])
        assert (got[:a] == 7).all() and (got[z:] == 7).all() and (glse[:a] == 7).all() and (glse[z:] == 7).all()
        got, glse = got[a:z], glse[a:z]
        keep = np.arange(z - a) if rows is None else np.asarray(rows)
        for t in keep:
            empty = np.isneginf(lse[t])
            assert np.array_equal(np.isneginf(glse[t]), empty), t
            assert (np.abs(got[t] - out[t]) <= oerr[t]).all(), (t, np.abs(got[t] - out[t]).max(), oerr[t].max())
            with np.errstate(invalid="ignore"):
                assert (empty | (np.abs(glse[t] - lse[t]) <= lerr[t])).all(), (t, np.abs(glse[t] - lse[t]).max())

    def window_seen(self, window, sinks):
        return lambda b, i: P.window_seen(self.ctxs[b] - self.counts[b] + i, window, sinks)

    def tree_seen(self, mask):
        m = mask.cpu().numpy()
        return lambda b, i: P.tree_seen(self.ctxs[b] - self.counts[b], self.counts[b], m[self.cu[b] + i])


def random_mask(counts, words, rng, before=0, behind=0):
    """Trees of random parents, as words."""
    rows = [np.zeros((before, words), dtype=np.int32)]
    for n in counts:
        rows.append(P.mask_words(P.tree_sets([int(rng.integers(max(-1, i - 5), i)) for i in range(n)]), words))
    rows.append(np.zeros((behind, words), dtype=np.int32))
    return i32(np.concatenate(rows))


WINDOWS = [
    (1, [1], [1], 1, 0, 64), (128, [1], [3000], 1024, 4, 64), (16, [1] * 5, [1, 64, 65, 200, 31], 50, 4, 16),
    (20, [37, 1, 0, 5], [300, 1, 10, 777], 333, 7, 16), (64, [3, 2], [130, 64], 64, 0, 128), (65, [2], [70], 5, 0, 32),
    (3, [130], [130], 17, 2, 16), (200, [2], [100], 1000, 0, 64), (128, [9], [700], 2 ** 40, 0, 64),
    (8, [70, 64], [70, 200], 1, 64, 32), (7, [33], [2000], 128, 130, 128), (33, [5, 5, 5], [1000, 63, 129], 64, 1, 64),
    (128, [4, 3], [64, 67], 3, 2, 64), (48, [11], [400], 130, 0, 16), (1, [300], [900], 100, 3, 64), (1000, [1], [50], 9, 1, 16)]


@pytest.mark.parametrize("with_ws", [False, True])
@pytest.mark.parametrize("H,counts,ctxs,window,sinks,bs", WINDOWS)
def test_window(H, counts, ctxs, window, sinks, bs, with_ws):
    c = Case(H, counts, ctxs, bs, seed=H, before=2, behind=3)
    c.window(window, sinks, ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    c.check(c.window_seen(window, sinks))


TREES = [
    (1, [1], [1], 1, 64), (128, [8], [2100], 1, 64), (20, [13, 1, 0, 7], [150, 1, 10, 900], 1, 16),
    (16, [32, 20], [500, 20], 1, 64), (64, [8, 5], [300, 131], 1, 128), (16, [64, 33], [64, 700], 2, 32),
    (5, [100, 3], [333, 1000], 4, 16), (65, [3], [70], 1, 64), (128, [3, 2], [65, 2], 2, 64), (2, [200], [1400], 7, 64),
    (40, [17], [97], 1, 32)]


@pytest.mark.parametrize("with_ws", [False, True])
@pytest.mark.parametrize("H,counts,ctxs,words,bs", TREES)
def test_tree(H, counts, ctxs, words, bs, with_ws):
    c = Case(H, counts, ctxs, bs, seed=H + 1, before=1, behind=2)
    mask = random_mask(counts, words, np.random.default_rng(H), 1, 2)
    c.tree(mask, ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    c.check(c.tree_seen(mask))


@pytest.mark.parametrize("with_ws", [False, True])
def test_masks_of_any_bits(with_ws):
    """Bits need no tree behind them: rows that see nothing, not themselves, later nodes; nodes beyond the words."""
    c = Case(20, [40, 3, 70], [40, 3, 300], 16, seed=5)
    rng = np.random.default_rng(5)
    words = rng.integers(-2 ** 31, 2 ** 31 - 1, (c.T, 2))
    words[3] = 0
    words[41] = 0
    mask = i32(words)
    ws = c.workspace() if with_ws else None
    c.tree(mask, ws=ws)
    c.check(c.tree_seen(mask))
    assert not c.out[3].any() and torch.isneginf(c.lse[41]).all()
    # no words at all: only the earlier tokens are seen
    none = torch.zeros((c.T, 0), dtype=torch.int32, device=DEV)
    c.tree(none, ws=ws)
    idx.idx_device_error()
    c.check(c.tree_seen(none))
    # words past the nodes hold anything
    more = torch.full((c.T, 32), -1, dtype=torch.int32, device=DEV)
    c.tree(more[:, :31], ws=ws)  # with a row stride
    idx.idx_device_error()
    c.check(c.tree_seen(more[:, :31]))


@pytest.mark.parametrize("op", ["window", "tree"])
@pytest.mark.parametrize("with_ws", [False, True])
def test_contexts_shorter_than_their_rows(op, with_ws):
    """A request that sits out has length 0; rows before a context's first token see nothing."""
    c = Case(16, [1, 1, 5, 2], [0, 9, 3, -4], 16, seed=8)
    ws = c.workspace() if with_ws else None
    if op == "window":
        c.window(4, 1, ws=ws)
        c.check(c.window_seen(4, 1))
    else:
        mask = i32(np.full((c.T, 1), -1))
        c.tree(mask, ws=ws)
        c.check(c.tree_seen(mask))
    idx.idx_device_error()
    assert not c.out[0].any() and torch.isneginf(c.lse[0]).all() and not c.out[7:].any()


@pytest.mark.parametrize("H", [8, 128])
@pytest.mark.parametrize("with_ws", [False, True])
def test_strides(H, with_ws):
    """Rows and heads of q and out that are slices of larger tensors, lse too; what lies between stays."""
    c = Case(H, [5, 9], [200, 77], 64, seed=3)
    qb = torch.full((c.T, H + 2, 600), float("nan"), dtype=torch.bfloat16, device=DEV)
    qb[:, 1:-1, 8:584] = c.q
    ob = torch.full((c.T, H + 3, 528), 5.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((c.T, H + 1), 5.0, dtype=torch.float32, device=DEV)
    tb = torch.full((2, c.block_table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    tb[:, :-3] = c.block_table
    idx.idx_window_attention(qb[:, 1:-1, 8:584], c.cache, 64, tb[:, :-3], i32(c.cu), i32(c.ctxs), ob[:, 2:-1, 8:520], SCALE, 60,
                             sinks=2, lse=lb[:, 1:], ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    c.out, c.lse = ob[:, 2:-1, 8:520].contiguous(), lb[:, 1:].contiguous()
    c.check(c.window_seen(60, 2))
    ob[:, 2:-1, 8:520] = 5.0
    assert (ob == 5).all() and (lb[:, 0] == 5).all()
    # heads outside, rows inside
    qt, ot = c.q.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros(H, c.T, 512, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    idx.idx_window_attention(qt, c.cache, 64, c.block_table, i32(c.cu), i32(c.ctxs), ot, SCALE, 60, sinks=2)
    assert torch.equal(ot, c.out) or with_ws
    c.out = ot.contiguous()
    c.check(c.window_seen(60, 2))


@pytest.mark.parametrize("H,rows", [(128, 6), (16, 24), (3, 50), (64, 70), (128, 50)])
@pytest.mark.parametrize("with_ws", [False, True])
def test_tokens_that_are_not_finite(H, rows, with_ws):
    """A NaN token makes the rows that see it NaN and no other; an infinite position dim likewise."""
    window, ctx, bs = 20, 200, 16
    c = Case(H, [rows], [ctx], bs, seed=4)
    at = {ctx - rows - 3: "latent", ctx - rows // 2: "latent", ctx - rows - 10: "rope nan", ctx - rows - 12: "rope inf", 150 - rows: "unseen"}
    for j, kind in at.items():
        rec = c.cache[int(c.table[0, j // bs])]
        off = j % bs
        if kind.startswith("rope"):
            rec[512 * bs + 128 * off:512 * bs + 128 * off + 2] = torch.tensor(
                [0xC0, 0x7F] if kind == "rope nan" else [0x80, 0x7F], dtype=torch.uint8, device=DEV)
        else:
            rec[640 * bs + 4 * off + 2] = 255
            rec[512 * off + 256:512 * off + 384] = 0
    c.window(window, 2, ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    out, lse = c.out.float(), c.lse
    seen = c.window_seen(window, 2)
    clean = []
    for i in range(rows):
        s = set(seen(0, i))
        nans = [j for j, k in at.items() if j in s and k in ("latent", "rope nan")]
        infs = [j for j, k in at.items() if j in s and k == "rope inf"]
        if nans:
            assert torch.isnan(out[i]).all() and torch.isnan(lse[i]).all(), i
        elif infs:
            # +inf among the logits: NaN weights; -inf: the token does not count
            up = c.q[i, :, 512].float() > 0
            assert torch.isnan(out[i][up]).all() and torch.isnan(lse[i][up]).all() and torch.isfinite(out[i][~up]).all(), i
        else:
            clean.append(i)
    assert clean or rows < 50  # of a few rows, each sees one of them
    c.check(seen, clean)


@pytest.mark.parametrize("H", [16, 128])
def test_queries_that_are_not_finite(H):
    """A head's NaN or infinity stays in that head."""
    c = Case(H, [6], [90], 16, seed=6)
    c.q[2, 3, 100] = float("nan")
    c.q[4, 0, 570] = float("inf")
    c.window(40, 1)
    idx.idx_device_error()
    bad = torch.zeros(6, H, dtype=torch.bool, device=DEV)
    bad[2, 3], bad[4, 0] = True, True
    assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
    c.q[2, 3, 100], c.q[4, 0, 570] = 0, 0
    out, lse, oerr, lerr = c.want(c.window_seen(40, 1))
    ok = ~bad.cpu().numpy()
    assert (np.abs(c.out.double().cpu().numpy() - out) <= oerr)[ok].all() and (np.abs(c.lse.double().cpu().numpy() - lse) <= lerr)[ok].all()


@pytest.mark.parametrize("H,rows", [(16, 1), (128, 1), (16, 40), (128, 5)])
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("with_ws", [False, True])
def test_pages_that_no_row_sees_may_be_gone(H, rows, bs, with_ws):
    """A server that frees blocks behind the window: their entries are -1 or point anywhere."""
    ctx, window, sinks = 1000, 200, 5
    c = Case(H, [rows], [ctx], bs, seed=9)
    first = ctx - rows - window + 1  # the first token that the first row's window has
    dead = [p for p in range(c.table.shape[1]) if p > (sinks - 1) // bs and (p + 1) * bs <= first]
    assert dead
    c.block_table[0, dead] = i32([[-1, 2 ** 31 - 1, -2 ** 31][i % 3] for i in range(len(dead))])
    c.window(window, sinks, ws=c.workspace() if with_ws else None)
    idx.idx_device_error()
    c.check(c.window_seen(window, sinks))


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("with_ws", [False, True])
def test_bad_pages_are_skipped_and_flagged(H, with_ws):
    c = Case(H, [3, 2], [300, 100], 16, seed=10)
    ws = c.workspace() if with_ws else None
    gone = {0: [2, 17], 1: [0]}
    c.block_table[0, 2], c.block_table[0, 17], c.block_table[1, 0] = -1, c.cache.shape[0], 2 ** 31 - 1
    mask = i32(np.full((5, 1), -1))
    c.tree(mask, ws=ws)
    with pytest.raises(idx.IdxError, match="tree attention 0x00000001"):
        idx.idx_device_error()
    full = c.tree_seen(mask)
    c.check(lambda b, i: [j for j in full(b, i) if j // 16 not in gone[b]])
    # a context longer than the table: the pages beyond are missing
    c2 = Case(H, [3], [300], 16, seed=11)
    c2.block_table = c2.block_table[:, :10].contiguous()
    c2.window(10 ** 6, 0, ws=c2.workspace() if with_ws else None)
    with pytest.raises(idx.IdxError, match="tree attention 0x00000001"):
        idx.idx_device_error()
    c2.check(lambda b, i: list(range(160)))
    idx.idx_device_error()


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes, q and out rows beyond 2^31 elements."""
    bs, H, far = 64, 4, 110_000
    c = Case(H, [2], [130], bs, seed=12)
    big = torch.empty((far + 3, stride_of(bs)), dtype=torch.uint8, device=DEV)
    t = c.table.copy()
    for p in range(3):
        big[far + 2 - p] = c.cache[int(c.table[0, p])]
        t[0, p] = far + 2 - p
    step = 2 ** 31 + 64
    qb, ob = torch.empty(step + H * 576, dtype=torch.bfloat16, device=DEV), torch.empty(step + H * 512, dtype=torch.bfloat16, device=DEV)
    q, out = qb.as_strided((2, H, 576), (step, 576, 1)), ob.as_strided((2, H, 512), (step, 512, 1))
    q.copy_(c.q)
    for ws in (None, c.workspace()):
        idx.idx_window_attention(q, big, bs, i32(t), i32(c.cu), i32(c.ctxs), out, SCALE, 100, sinks=3, lse=c.lse, ws=ws)
        idx.idx_device_error()
        c.out = out.contiguous()
        c.check(c.window_seen(100, 3))


@pytest.mark.parametrize("H,counts,ctxs", [(16, [1] * 40, [500] * 40), (128, [2], [3000]), (128, [40, 30], [500, 100])])
def test_two_graphs_and_a_side_stream(H, counts, ctxs):
    """Two captured calls with a workspace each, replayed at once on two streams, beside an eager call."""
    cases = [Case(H, counts, ctxs, 64, seed=s) for s in (20, 21, 22)]
    for c in cases:
        c.ws = c.workspace()
        c.dev = (i32(c.cu), i32(c.ctxs))

    def run(c, stream=None):
        idx.idx_window_attention(c.q, c.cache, c.bs, c.block_table, c.dev[0], c.dev[1], c.out, SCALE, 333, sinks=4, lse=c.lse,
                                 ws=c.ws, stream=stream)

    run(cases[0])
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    for c, s in zip(cases[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(c)
        graphs.append(g)
    for c in cases:
        c.out.fill_(7)
        c.lse.fill_(7)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        run(cases[2], stream=streams[2])
    torch.cuda.synchronize()
    idx.idx_device_error()
    for c in cases:
        c.check(c.window_seen(333, 4))


@pytest.mark.parametrize("op", ["window", "tree"])
@pytest.mark.parametrize("H,counts,ctxs", [(16, [1] * 3, [5000, 100, 1]), (64, [8] * 20, [700] * 20), (128, [70, 9], [300, 1000])])
def test_results_repeat_bit_for_bit(op, H, counts, ctxs):
    c = Case(H, counts, ctxs, 64, seed=30)
    mask = random_mask(counts, 3, np.random.default_rng(1))
    got = []
    for fill in (255, 0):
        ws = c.workspace()
        if ws is not None:
            ws.fill_(fill)
        for _ in range(3):
            c.window(100, 2, ws=ws) if op == "window" else c.tree(mask, ws=ws)
            got.append((c.out.clone(), c.lse.clone()))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_refusals_of_the_bindings():
    c = Case(8, [2], [50], 64)
    with pytest.raises(ValueError, match="cu_rows"):
        idx.idx_window_attention(c.q, c.cache, 64, c.block_table, i32([0, 1, 2]), i32(c.ctxs), c.out, SCALE, 10)
    with pytest.raises(ValueError, match="ctx_lens"):
        idx.idx_window_attention(c.q, c.cache, 64, c.block_table, i32(c.cu), i32([1, 2]), c.out, SCALE, 10)
    with pytest.raises(ValueError, match="out"):
        idx.idx_window_attention(c.q, c.cache, 64, c.block_table, i32(c.cu), i32(c.ctxs), c.out[:1], SCALE, 10)
    with pytest.raises(ValueError, match="mask"):
        idx.idx_tree_attention(c.q, c.cache, 64, c.block_table, i32(c.cu), i32(c.ctxs), torch.zeros(3, 1, dtype=torch.int32, device=DEV),
                               c.out, SCALE)
    with pytest.raises(idx.IdxError, match="window 0"):
        idx.idx_window_attention(c.q, c.cache, 64, c.block_table, i32(c.cu), i32(c.ctxs), c.out, SCALE, 0)
    n = idx.idx_paged_attention_workspace_bytes(2, 1, 8)
    if n:
        with pytest.raises(idx.IdxError, match="workspace has"):
            c.window(10, 0, ws=torch.empty(n - 16, dtype=torch.uint8, device=DEV))


def lengths(n, lo, hi, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(lo, hi + 1, n)]


@pytest.mark.parametrize("H,counts,ctxs", [
    (16, [9, 0, 20, 3] * 11, lengths(44, 20, 900, 1)),          # more units than the GPU has blocks: shares of several units
    (3, [1] * 100, lengths(100, 1, 2500, 2)),                   # fewer, of lengths that no whole number of parts fits
    (64, [2, 1, 3], [3000, 40, 9000]),                          # few: a context cut into many parts
    (2, [1] * 160, lengths(160, 0, 700, 3)), (2, [1] * 161, lengths(161, 0, 700, 4)),  # the most requests that are shared, and more
    (128, [1, 1], [1500, 1500]), (5, [64, 0, 0, 1], [800, 0, 900, 2000]),
    (2, [1] * 160, lengths(160, 0, 1300, 5)), (16, [37, 0, 50, 3] * 11, lengths(44, 60, 1300, 6)),
    (64, [5, 0, 2] * 50, lengths(150, 0, 1300, 7))])
def test_shared_work(H, counts, ctxs):
    """The same results with a workspace, where blocks take equal shares of ragged work, as the oracle has."""
    ctxs = [max(c, n) for c, n in zip(ctxs, counts)]
    c = Case(H, counts, ctxs, 64, seed=H, before=1, behind=1, extra_pages=20)
    mask = random_mask(counts, 2, np.random.default_rng(H), 1, 1)
    c.tree(mask, ws=c.workspace())
    idx.idx_device_error()
    c.check(c.tree_seen(mask))
    c.tree(mask)
    c.check(c.tree_seen(mask))


@pytest.mark.parametrize("bs", [16, 64])
def test_long_context(bs):
    """One row over 70 000 tokens, whole and cut: every token counts once, first and last among them."""
    ctx, H = 70_001, 2
    c = Case(H, [1], [ctx], bs, seed=2)
    # all weights alike, values 1 at one dim each
    c.q.zero_()
    codes = torch.zeros(c.cache.shape[0], bs, 512, dtype=torch.uint8, device=DEV)
    order = {int(blk): p for p, blk in enumerate(c.table[0])}
    dims = np.random.default_rng(3).integers(0, 512, ctx)
    host = np.zeros((c.cache.shape[0], bs, 512), dtype=np.uint8)
    for blk, p in order.items():
        n = min(bs, ctx - p * bs)
        host[blk, np.arange(n), dims[p * bs:p * bs + n]] = 0x38  # 1.0
    codes.copy_(torch.from_numpy(host))
    c.cache[:, :512 * bs] = codes.view(-1, 512 * bs)
    c.cache[:, 512 * bs:640 * bs] = 0
    c.cache[:, 640 * bs:644 * bs] = 127
    want = np.bincount(dims, minlength=512) / ctx
    for ws in (None, c.workspace()):
        c.out.fill_(7)
        c.window(10 ** 9, 0, ws=ws)
        idx.idx_device_error()
        got = c.out.double().cpu().numpy()
        # counts up to 200 of 70001 are exact in the accumulator; 1 / n, one product and the bf16 store round
        assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -21) * want).all()
        assert np.abs(c.lse.double().cpu().numpy() - np.log(ctx)).max() <= 2.0 ** -20 * np.log(ctx)


@pytest.mark.parametrize("bs,pages", [(128, 2 ** 24 + 3), (64, 2 ** 21)])
def test_wide_table(bs, pages):
    """Tables for more tokens than 31 bits count, and for so many that the call's work is not shared out."""
    c = Case(3, [2, 1], [900, 2000], bs, seed=7)
    have = c.block_table.shape[1]
    c.block_table = torch.cat([c.block_table, torch.full((2, pages - have), -1, dtype=torch.int32, device=DEV)], dim=1)
    mask = random_mask(c.counts, 1, np.random.default_rng(7))
    c.tree(mask, ws=c.workspace())
    idx.idx_device_error()
    c.check(c.tree_seen(mask))
    c.window(2 ** 31 - 1, 2 ** 31 - 1, ws=c.workspace())
    idx.idx_device_error()
    c.check(c.window_seen(2 ** 31 - 1, 2 ** 31 - 1))


def test_two_streams():
    """Calls on two streams at once, each with its own workspace, give what they give alone."""
    cases = [Case(64, [5, 0, 2, 8] * 4, lengths(16, 100, 4000, 8), 64, seed=8), Case(128, [1, 3], [9000, 40], 16, seed=9)]
    masks = [random_mask(c.counts, 1, np.random.default_rng(1)) for c in cases]
    ws = [c.workspace() for c in cases]
    want = []
    for c, m, w in zip(cases, masks, ws):
        c.tree(m, ws=w)
        want.append((c.out.clone(), c.lse.clone()))
        c.out.fill_(7)
    lens = [(i32(c.cu), i32(c.ctxs)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, m, w, st, (cu, ctx) in zip(cases, masks, ws, streams, lens):
            idx.idx_tree_attention(c.q, c.cache, c.bs, c.block_table, cu, ctx, m, c.out, SCALE, lse=c.lse, ws=w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cases, want):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    idx.idx_device_error()


def test_extents_of_one():
    """One row, one head, one block: their strides are never used, whatever they are."""
    c = Case(1, [1], [50], 64, seed=10)
    block = int(c.table[0, 0])
    c.cache, c.table = c.cache[block:block + 1], c.table * 0
    c.block_table = i32(c.table)
    q, out = c.q.as_strided((1, 1, 576), (24, 40, 1)), c.out.as_strided((1, 1, 512), (8, 16, 1))
    cache = c.cache.as_strided((1, c.cache.shape[1]), (3, 1))
    idx.idx_window_attention(q, cache, 64, c.block_table.as_strided((1, 1), (5, 1)), i32(c.cu), i32(c.ctxs), out, SCALE, 30,
                             lse=c.lse.as_strided((1, 1), (9, 7)))
    idx.idx_device_error()
    c.check(c.window_seen(30, 0))
