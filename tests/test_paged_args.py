"""Refusals of the step tables, the tree masks and the attention over contexts (CPU only).

Every call fails its validation before anything is enqueued, so the fake pointers are never used.
"""

import ctypes
import math

import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)
BIG = (1 << 31)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_fp8_gb300 import _lib
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    return _lib.load()


def _args(base, changes):
    d = dict(base)
    assert set(changes) <= set(d)
    d.update(changes)
    return list(d.values())


TABLES = dict(cached=P, new=P, held=None, B=4, free=P, n_free=9, start=None, bt=P, ld_bt=8, pages=8, bs=64, ctx=P, cu=P,
              cu_ctx=None, held_out=None, free_end=None, pos=P, slots=P, req=None, ke=None, rows=5, stream=None)
MASK = dict(parents=P, cu=P, B=2, rows=9, base=None, mask=P, ld=1, words=1, pos=None, stream=None)
HEAD = dict(q=P, ld_q=576 * 8, ld_qh=576, cache=P, blocks=8, bs=64, stride=41472, bt=P, ld_bt=4, pages=4, cu=P, ctx=P, B=2)
TAIL = dict(T=4, H=8, scale=0.07, out=P, ld_out=512 * 8, ld_oh=512, lse=None, ld_lse=0, ws=None, wsb=0, stream=None)
WINDOW = {**HEAD, "window": 128, "sinks": 4, **TAIL}
TREE = {**HEAD, "mask": P, "ld_mask": 2, "words": 2, **TAIL}


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, INVALID), ({"n_free": -1}, INVALID), ({"pages": -1}, INVALID), ({"rows": -1}, INVALID),
    ({"B": 8193}, UNSUPPORTED), ({"bs": 48}, UNSUPPORTED), ({"bs": 0}, UNSUPPORTED), ({"ld_bt": 7}, INVALID),
    ({"cached": None}, INVALID), ({"new": None}, INVALID), ({"free": None}, INVALID), ({"bt": None}, INVALID),
    ({"ctx": None}, INVALID), ({"cu": None}, INVALID), ({"pos": None}, INVALID), ({"slots": None}, INVALID)])
def test_tables_refusals(lib, change, status):
    assert lib.idx_build_tables(*_args(TABLES, change)) == status


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, INVALID), ({"rows": -1}, INVALID), ({"words": 0}, INVALID), ({"words": 33, "ld": 33}, UNSUPPORTED),
    ({"words": 2}, INVALID), ({"parents": None}, INVALID), ({"cu": None}, INVALID), ({"mask": None}, INVALID),
    ({"B": 0, "cu": None}, OK), ({"rows": 0, "mask": None}, OK)])
def test_tree_mask_refusals(lib, change, status):
    assert lib.idx_tree_mask(*_args(MASK, change)) == status


@pytest.mark.parametrize("which", ["window", "tree"])
@pytest.mark.parametrize("change,status", [
    ({"T": -1}, INVALID), ({"H": -1}, INVALID), ({"B": -1}, INVALID), ({"pages": -1}, INVALID), ({"H": 1025}, UNSUPPORTED),
    ({"ld_bt": 3}, INVALID), ({"ld_q": 575}, INVALID), ({"ld_qh": 575}, INVALID), ({"ld_out": 511}, INVALID),
    ({"ld_oh": 511}, INVALID), ({"lse": P, "ld_lse": 7}, INVALID), ({"scale": math.inf}, INVALID),
    ({"scale": math.nan}, INVALID), ({"scale": 3e38}, INVALID), ({"q": None}, INVALID), ({"cache": None}, INVALID),
    ({"out": None}, INVALID), ({"bt": None}, INVALID), ({"cu": None}, INVALID), ({"ctx": None}, INVALID),
    ({"bs": 24}, UNSUPPORTED), ({"stride": 41200}, INVALID), ({"stride": 41480}, UNSUPPORTED), ({"blocks": -1}, INVALID),
    ({"cache": MIS}, UNSUPPORTED), ({"q": MIS}, UNSUPPORTED), ({"out": MIS}, UNSUPPORTED),
    ({"ld_q": 576 * 8 + 4}, UNSUPPORTED), ({"ld_qh": 580}, UNSUPPORTED), ({"ld_out": 512 * 8 + 4}, UNSUPPORTED),
    ({"ld_oh": 516}, UNSUPPORTED), ({"ws": MIS, "wsb": 1 << 40}, UNSUPPORTED), ({"T": 0, "q": None}, OK),
    ({"H": 0, "q": None}, OK), ({"B": 0, "cu": None}, OK)])
def test_attention_refusals(lib, which, change, status):
    call, base = (lib.idx_window_attention, WINDOW) if which == "window" else (lib.idx_tree_attention, TREE)
    assert call(*_args(base, change)) == status


@pytest.mark.parametrize("which", ["window", "tree"])
@pytest.mark.parametrize("change", [{"ld_q": 1 << 39}, {"ld_qh": 1 << 39}, {"stride": 1 << 40}])
def test_strides_beyond_a_tensor_map(lib, which, change):
    call, base = (lib.idx_window_attention, WINDOW) if which == "window" else (lib.idx_tree_attention, TREE)
    assert call(*_args(base, change)) == UNSUPPORTED


@pytest.mark.parametrize("change,status", [({"window": 0}, INVALID), ({"window": -5}, INVALID), ({"sinks": -1}, INVALID)])
def test_window_refusals(lib, change, status):
    assert lib.idx_window_attention(*_args(WINDOW, change)) == status


@pytest.mark.parametrize("change,status", [({"words": -1}, INVALID), ({"words": 33, "ld_mask": 33}, UNSUPPORTED),
                                           ({"ld_mask": 1}, INVALID), ({"mask": None}, INVALID)])
def test_tree_refusals(lib, change, status):
    assert lib.idx_tree_attention(*_args(TREE, change)) == status


def test_workspace_bytes_of_nothing(lib):
    for sizes in ((0, 1, 8), (4, 0, 8), (4, 2, 0), (-1, 2, 8)):
        assert lib.idx_paged_attention_workspace_bytes(*sizes) == 0
    with pytest.raises(ValueError, match="32 bits"):
        idx.idx_paged_attention_workspace_bytes(BIG, 1, 8)


def test_bindings_refuse_host_tensors():
    f, i32, i64, u8, bf = torch.zeros, torch.int32, torch.int64, torch.uint8, torch.bfloat16
    q, cache, bt, cu, ctx = f(4, 8, 576, dtype=bf), f(8, 41472, dtype=u8), f(2, 4, dtype=i32), f(3, dtype=i32), f(2, dtype=i32)
    out = f(4, 8, 512, dtype=bf)
    with pytest.raises(ValueError, match="cached_lens must be a CUDA tensor"):
        idx.idx_build_tables(ctx, ctx, f(5, dtype=i32), bt, 64, ctx, cu, f(4, dtype=i32), f(4, dtype=i64))
    with pytest.raises(ValueError, match="parents must be a CUDA tensor"):
        idx.idx_tree_mask(f(4, dtype=i32), cu, f(4, 1, dtype=i32))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        idx.idx_window_attention(q, cache, 64, bt, cu, ctx, out, 0.07, 128)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        idx.idx_tree_attention(q, cache, 64, bt, cu, ctx, f(4, 1, dtype=i32), out, 0.07)
