"""Step tables and tree masks against the host's: every integer equal."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import paged as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def outputs(B, rows, fill=-77):
    return {"ctx_lens": torch.full((B,), fill, dtype=torch.int32, device=DEV),
            "cu_rows": torch.full((B + 1,), fill, dtype=torch.int32, device=DEV),
            "cu_ctx": torch.full((B + 1,), fill, dtype=torch.int32, device=DEV),
            "held": torch.full((B,), fill, dtype=torch.int32, device=DEV),
            "free_end": torch.full((1,), fill, dtype=torch.int32, device=DEV),
            "positions": torch.full((rows,), fill, dtype=torch.int32, device=DEV),
            "slots": torch.full((rows,), fill, dtype=torch.int64, device=DEV),
            "row_to_req": torch.full((rows,), fill, dtype=torch.int32, device=DEV),
            "row_ke": torch.full((rows,), fill, dtype=torch.int32, device=DEV)}


def call(o, cached, new, free, table, bs, held=None, start=None, stream=None):
    idx.idx_build_tables(cached, new, free, table, bs, o["ctx_lens"], o["cu_rows"], o["positions"], o["slots"],
                         held_pages=held, held_out=o["held"], free_start=start, free_end=o["free_end"],
                         cu_ctx=o["cu_ctx"], row_to_req=o["row_to_req"], row_ke=o["row_ke"], stream=stream)


def same(o, table, want):
    for k, v in want.items():
        got = table if k == "table" else o[k]
        assert np.array_equal(got.cpu().numpy().astype(np.int64).reshape(-1), np.asarray(v).reshape(-1)), k


@pytest.mark.parametrize("B,new,ctx,bs,pad,with_held", [
    (0, 0, 0, 64, 5, False), (1, 1, 0, 16, 0, False), (1, 1, 100, 64, 0, True), (1, 5000, 63, 64, 7, False),
    (3, 40, 200, 16, 3, True), (128, 1, 5000, 64, 0, False), (129, 3, 999, 128, 40, True), (1023, 2, 300, 32, 1, True),
    (1024, 1, 300, 32, 0, False), (1025, 2, 300, 16, 600, True), (2500, 3, 70, 16, 11, True), (8192, 1, 40, 16, 3, True),
    (40, 700, 4000, 64, 100, True)])
def test_tables(B, new, ctx, bs, pad, with_held):
    rng = np.random.default_rng(B + new)
    cached = rng.integers(0, ctx + 1, B)
    add = rng.integers(0, new + 1, B) if B > 2 else np.full(B, new)
    held = -(-cached // bs) + (rng.random(B) < 0.3) if with_held else None
    pages = max(1, -(-(ctx + new) // bs) + 1)
    total = int(B * pages + 9)
    ids = rng.permutation(total)
    table = np.where(rng.random((B, pages)) < 0.5, -1, rng.integers(0, total, (B, pages)))
    for b in range(B):
        n = -(-cached[b] // bs) if held is None else held[b]
        table[b, :n] = ids[:n] + b  # any blocks will do
    rows = int(add.sum()) + pad
    start = 3 if with_held else 0
    want = P.build_tables(cached, add, ids, table, bs, rows, held, start)
    wide = torch.full((B, pages + 5), -9, dtype=torch.int32, device=DEV)  # a table with a row stride
    wide[:, :pages] = i32(table).view(B, pages)
    o = outputs(B, rows)
    call(o, i32(cached), i32(add), i32(ids), wide[:, :pages], bs, None if held is None else i32(held),
         i32([start]) if with_held else None)
    idx.idx_device_error()
    same(o, wide[:, :pages], want)
    assert (wide[:, pages:] == -9).all()


def test_blocks_run_out_and_a_later_call_serves_the_rest():
    cached, add, bs = [0, 30, 5], [40, 10, 20], 16
    table = np.full((3, 4), -1)
    table[1, :2], table[2, :1] = [50, 51], [52]
    o, t = outputs(3, 80), i32(table)
    call(o, i32(cached), i32(add), i32([1, 2, 3, 4]), t, bs)
    with pytest.raises(idx.IdxError, match="tables 0x00000002"):
        idx.idx_device_error()
    want = P.build_tables(cached, add, [1, 2, 3, 4], table, bs, 80)
    assert want["held"].tolist() == [3, 3, 1] and want["free_end"] == 4
    same(o, t, want)
    # with more blocks the same lengths and the pages that are held complete the table
    o2 = outputs(3, 80)
    call(o2, i32(cached), i32(add), i32([1, 2, 3, 4, 5, 6]), t, bs, held=o["held"], start=o["free_end"])
    idx.idx_device_error()
    assert o2["held"].tolist() == [3, 3, 2] and o2["free_end"].item() == 5 and t[2].tolist() == [52, 5, -1, -1]
    assert (o2["slots"][:70] >= 0).all() and (o2["slots"][70:] == -1).all()


@pytest.mark.parametrize("B", [3, 3000])
def test_what_is_out_of_range(B):
    def run(cached, add, held=None, start=None, pages=2, rows=8, flag=0):
        c, a = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
        c[-3:], a[-3:] = cached, add
        h = None
        if held is not None:
            h = np.zeros(B, dtype=np.int64)
            h[-3:] = held
        o, t = outputs(B, rows), torch.full((B, pages), 7, dtype=torch.int32, device=DEV)
        call(o, i32(c), i32(a), torch.arange(100, 200, dtype=torch.int32, device=DEV), t, 16, None if h is None else i32(h),
             None if start is None else i32([start]))
        with pytest.raises(idx.IdxError, match=f"tables 0x{flag:08x}"):
            idx.idx_device_error()
        idx.idx_device_error()
        return o, t

    # a negative length, and one beyond 32 bits: the request is empty, the others are served
    o, _ = run([4, -1, 2 ** 31 - 1], [2, 5, 1], flag=1)
    assert o["ctx_lens"][-3:].tolist() == [6, 0, 0] and o["cu_rows"][-3:].tolist() == [2, 2, 2]
    assert o["slots"].tolist() == [7 * 16 + 4, 7 * 16 + 5] + [-1] * 6
    # a context beyond the table: its tokens there have no slot
    o, t = run([30, 0, 0], [4, 0, 1], flag=4)
    assert o["slots"].tolist() == [7 * 16 + 14, 7 * 16 + 15, -1, -1, 100 * 16, -1, -1, -1] and o["ctx_lens"][-3].item() == 34
    # page counts and free_start
    o, t = run([0, 0, 0], [1, 0, 1], held=[-2, 0, 9], flag=1)
    assert o["held"][-3:].tolist() == [1, 0, 2] and t[-3].tolist() == [100, 7] and t[-1].tolist() == [7, 7]
    o, t = run([0, 0, 0], [1, 0, 1], start=-5, flag=1)
    assert t[-3:, 0].tolist() == [100, 7, 101] and o["free_end"].item() == 2
    # blocks that start beyond the list, and more tokens than rows
    o, t = run([0, 0, 0], [1, 0, 1], start=2 ** 31 - 1, flag=2)
    assert t[-3:, 0].tolist() == [-1, 7, -1] and o["free_end"].item() == 2 ** 31 - 1 and (o["slots"] == -1).all()
    o, t = run([0, 0, 0], [5, 0, 6], flag=8)
    assert o["positions"].tolist() == [0, 1, 2, 3, 4, 0, 1, 2] and o["cu_rows"][-1].item() == 11


def test_sums_beyond_32_bits():
    B = 3
    cached, add = i32([2 ** 30, 2 ** 30, 2 ** 30]), i32([1, 1, 1])
    o, t = outputs(B, 3), torch.full((B, 1), 5, dtype=torch.int32, device=DEV)
    call(o, cached, add, i32([1]), t, 128)
    with pytest.raises(idx.IdxError, match="tables 0x00000005"):
        idx.idx_device_error()
    assert o["cu_ctx"].tolist() == [0, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31 - 1] and o["positions"].tolist() == [2 ** 30] * 3


@pytest.mark.parametrize("B,n", [(5, 1), (5, 3), (1500, 2)])
def test_captured_steps_advance_their_own_lengths(B, n):
    """Lengths, pages and the start of the free blocks updated in place by every replay, on a side stream."""
    rng = np.random.default_rng(B)
    bs, pages, steps = 16, 8, 12
    cached = rng.integers(0, 60, B)
    add = rng.integers(0, n + 1, B)
    ids = rng.permutation(B * pages)
    table = np.full((B, pages), -1)
    at = 0
    for b in range(B):
        k = -(-cached[b] // bs)
        table[b, :k] = ids[at:at + k]
        at += k
    lens, held = i32(cached), i32(-(-cached // bs))
    t, a, free, start = i32(table), i32(add), i32(ids), i32([at])
    o = outputs(B, int(add.sum()) + 2)
    o["ctx_lens"], o["held"], o["free_end"] = lens, held, start
    before = (lens.clone(), held.clone(), start.clone(), t.clone())
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(o, lens, a, free, t, bs, held, start)  # loads the kernel before the capture
    side.synchronize()
    for x, y in zip((lens, held, start, t), before):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        call(o, lens, a, free, t, bs, held, start)
    c, h, s = cached.copy(), -(-cached // bs), at
    for _ in range(steps):
        g.replay()
        torch.cuda.synchronize()
        want = P.build_tables(c, add, ids, table, bs, int(add.sum()) + 2, h, s)
        same(o, t, want)
        c, h, s, table = want["ctx_lens"], want["held"], want["free_end"], want["table"]
    idx.idx_device_error()


# ------------------------------------------------------------------ tree masks

@pytest.mark.parametrize("counts,words", [
    ([1], 1), ([16] * 8, 1), ([0, 5, 0, 31, 32], 1), ([33, 64, 1, 63], 2), ([128, 3], 4), ([300, 1000, 129], 32), ([7], 32)])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_tree_mask(counts, words, kind):
    rng = np.random.default_rng(len(counts) + words)
    parents, want, depth = [], [], []
    for n in counts:
        up = [i - 1 if kind == "chain" else -1 if kind == "star" else int(rng.integers(max(-1, i - 9), i)) for i in range(n)]
        sets = P.tree_sets(up)
        parents += up
        want.append(P.mask_words(sets, words))
        depth += [len(s) - 1 for s in sets]
    first = 2  # rows before the first request and behind the last stay as they are
    cu = np.concatenate([[0], np.cumsum(counts)]) + first
    n = int(cu[-1]) + 3
    base = rng.integers(0, 1000, len(counts))
    wide = torch.full((n, words + 3), -9, dtype=torch.int32, device=DEV)
    pos = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    par = i32([5, 5] + parents + [9, 9, 9])
    idx.idx_tree_mask(par, i32(cu), wide[:, :words], base_lens=i32(base), positions=pos)
    idx.idx_device_error()
    full = np.full((n, words + 3), -9)
    full[first:-3, :words] = np.concatenate(want)
    assert np.array_equal(wide.cpu().numpy(), full)
    assert pos[:first].tolist() == [-9] * 2 and pos[-3:].tolist() == [-9] * 3
    assert pos[first:-3].tolist() == [d + int(base[b]) for d, b in zip(depth, np.repeat(np.arange(len(counts)), counts))]
    idx.idx_tree_mask(par, i32(cu), wide[:, :words])  # without positions
    assert np.array_equal(wide.cpu().numpy(), full)


def test_tree_mask_of_bad_parents_and_too_many_nodes():
    mask, pos = torch.zeros(40, 1, dtype=torch.int32, device=DEV), torch.zeros(40, dtype=torch.int32, device=DEV)
    par = np.arange(-1, 39)
    par[3], par[5], par[7] = 3, 30, -2  # itself, a later node, below -1: all roots
    idx.idx_tree_mask(i32(par), i32([0, 40]), mask, base_lens=i32([100]), positions=pos)
    with pytest.raises(idx.IdxError, match="tables 0x00000010"):
        idx.idx_device_error()
    good = par.copy()
    good[[3, 5, 7]] = -1
    sets = P.tree_sets(good)
    want = P.mask_words(sets[:32], 1)[:, 0].tolist() + [0] * 8
    assert mask[:, 0].tolist() == want
    assert pos.tolist() == [100 + len(s) - 1 for s in sets[:32]] + [100] * 8
    idx.idx_device_error()


def test_tree_mask_rows_end_at_the_tensors():
    """cu_rows beyond the rows that there are: nothing behind them is touched."""
    mask = torch.full((6, 1), -9, dtype=torch.int32, device=DEV)
    idx.idx_tree_mask(i32([-1, 0, 1, 2]), i32([0, 9]), mask[:4])
    assert mask[:, 0].tolist() == [1, 3, 7, 15, -9, -9]
    idx.idx_device_error()
