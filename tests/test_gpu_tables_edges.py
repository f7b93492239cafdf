"""Step tables and tree masks at the edges: sums beyond 32 bits, request counts around what a block holds, calls at once."""

import threading

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import paged as P
from test_gpu_tables import call, i32, outputs, same

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


@pytest.mark.parametrize("B", [3023, 3024, 3050, 3071, 4500])
@pytest.mark.parametrize("new", [1, 2])
def test_request_counts_around_what_a_block_holds_without_asking(B, new):
    """Sums of about 3000 requests reach the 48 KB of shared memory that a block has by default."""
    rng = np.random.default_rng(B)
    cached, bs = rng.integers(0, 50, B), 16
    add = rng.integers(0, new + 1, B)
    pages = 5
    ids, table = rng.permutation(B * pages), rng.integers(0, B * pages, (B, pages))
    rows = int(add.sum()) + 2
    want = P.build_tables(cached, add, ids, table, bs, rows)
    o, t = outputs(B, rows), i32(table)
    call(o, i32(cached), i32(add), i32(ids), t, bs)
    idx.idx_device_error()
    same(o, t, want)


def test_calls_of_two_threads():
    """Calls of different sizes from two threads at once, each on its own stream: each is launched and right."""
    failed = []

    def work(B, seed):
        try:
            rng = np.random.default_rng(seed)
            cached, add, bs, pages = rng.integers(0, 50, B), np.ones(B, dtype=np.int64), 16, 4
            ids, table = rng.permutation(B * pages), rng.integers(0, B * pages, (B, pages))
            want = P.build_tables(cached, add, ids, table, bs, B)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                o, t = outputs(B, B), i32(table)
                args = i32(cached), i32(add), i32(ids), t, bs
                for _ in range(500):
                    call(o, *args)
                stream.synchronize()
                same(o, t, want)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(B, s)) for s, B in enumerate((8192, 3500))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed
    idx.idx_device_error()


@pytest.mark.parametrize("aliased", [False, True])
def test_lengths_are_whole_where_the_sum_of_rows_is_held(aliased):
    """Only sums are held to 2^31 - 1: every request's own length is its cached and its new tokens."""
    cached, add = [1, 2, 3, 4], [2 ** 30, 2 ** 30, 2 ** 30, 5]
    o, t = outputs(4, 3), torch.full((4, 1), 6, dtype=torch.int32, device=DEV)
    lens = i32(cached)
    if aliased:
        o["ctx_lens"] = lens
    call(o, lens, i32(add), i32([9]), t, 64, held=i32([1] * 4))
    with pytest.raises(idx.IdxError, match="tables 0x0000000d"):
        idx.idx_device_error()
    assert o["ctx_lens"].tolist() == [c + a for c, a in zip(cached, add)]
    assert o["cu_rows"].tolist() == [0, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert o["cu_ctx"].tolist() == [0, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert o["positions"].tolist() == [1, 2, 3] and o["slots"].tolist() == [6 * 64 + 1, 6 * 64 + 2, 6 * 64 + 3]


def test_positions_near_the_end_of_32_bits():
    """A late request's rows: neither its length nor the row's number alone is near 2^31, their sum is."""
    B, n = 3, 40
    cached, add = [0, 2 ** 31 - 41, 2 ** 31 - 21], [n, n, 20]
    o, t = outputs(B, 2 * n + 25), torch.full((B, 3), 5, dtype=torch.int32, device=DEV)
    call(o, i32(cached), i32(add), i32([1]), t, 128, held=i32([3] * B))
    with pytest.raises(idx.IdxError, match="tables 0x00000005"):
        idx.idx_device_error()
    want = list(range(n)) + [2 ** 31 - 41 + i for i in range(n)] + [2 ** 31 - 21 + i for i in range(20)]
    assert o["positions"].tolist() == want + [0] * 5
    assert o["row_ke"].tolist() == [p + 1 for p in want] + [0] * 5
    assert o["ctx_lens"].tolist() == [n, 2 ** 31 - 1, 2 ** 31 - 1]


@pytest.mark.parametrize("cu,written", [
    ([2 ** 31 - 1, -2 ** 31], []), ([-2 ** 31, 2 ** 31 - 1], list(range(6))), ([4, 1], []), ([7, 9], []), ([-5, -2], []), ([5, 5], []),
    ([3, 2 ** 31 - 1], [3, 4, 5])])
def test_tree_mask_rows_of_any_bounds(cu, written):
    """Whatever cu_rows holds, only rows that there are are read and written."""
    mask = torch.full((6, 1), -9, dtype=torch.int32, device=DEV)
    pos = torch.full((6,), -9, dtype=torch.int32, device=DEV)
    idx.idx_tree_mask(i32([-1] * 6), i32(cu), mask, positions=pos, base_lens=i32([3]))
    idx.idx_device_error()
    want = [-9] * 6
    for i, r in enumerate(written):
        want[r] = 1 << i
    assert mask[:, 0].tolist() == want and pos.tolist() == [3 if r in written else -9 for r in range(6)]


def test_the_most_rows():
    """As many rows as 32 bits count, nearly all of them padding."""
    rows = 2 ** 31 - 1
    pos, slots = torch.full((rows,), 7, dtype=torch.int32, device=DEV), torch.full((rows,), 7, dtype=torch.int64, device=DEV)
    t, ctx, cu = i32([[3]]), i32([0]), i32([0, 0])
    idx.idx_build_tables(i32([10]), i32([4]), i32([5]), t, 16, ctx, cu, pos, slots)
    idx.idx_device_error()
    assert pos[:5].tolist() == [10, 11, 12, 13, 0] and slots[:5].tolist() == [58, 59, 60, 61, -1]
    assert not pos[5:].any() and slots[5:].max().item() == -1 and slots[5:].min().item() == -1
