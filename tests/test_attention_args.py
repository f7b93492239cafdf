"""Refusals of the normalised inserts, the read-back and the sparse attention (CPU only).

Every call fails its validation before anything is enqueued, so the fake pointers are never used.
"""

import ctypes
import math

import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_fp8_gb300 import _lib
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    return _lib.load()


def _args(base, changes):
    d = dict(base)
    d.update(changes)
    return list(d.values())


K_INSERT = dict(k=P, dtype=1, ld_k=128, n=4, weight=P, bias=None, eps=1e-6, pos=P, cs=P, ld_cs=64, max_pos=10,
                style=0, slots=P, cache=P, blocks=8, bs=64, stride=8704, fmt=0, stream=None)
KV_INSERT = dict(c=P, ld_c=576, pe=P, ld_pe=576, dtype=1, n=4, weight=P, eps=1e-6, pos=P, cs=P, ld_cs=64,
                 max_pos=10, style=0, slots=P, cache=P, blocks=8, bs=64, stride=41472, stream=None)
GATHER = dict(cache=P, blocks=8, bs=64, stride=41472, bt=P, ld_bt=4, pages=4, starts=None, cu=P, B=2, out=P, dtype=1,
              ld_out=576, n_out=10, stream=None)
ATTN = dict(q=P, ld_q=576 * 8, ld_qh=576, cache=P, blocks=8, bs=64, stride=41472, span=64, slots=P, ld_slots=32, k=32,
            n_sel=None, T=4, H=8, scale=0.04, out=P, ld_out=512 * 8, ld_oh=512, lse=None, ld_lse=0, ws=None, wsb=0,
            stream=None)
MIS = ctypes.c_void_p(0x10008)


@pytest.mark.parametrize("change,status", [
    ({"n": -1}, INVALID), ({"dtype": 3}, UNSUPPORTED), ({"ld_k": 127}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": math.nan}, INVALID), ({"k": None}, INVALID), ({"weight": None}, INVALID), ({"pos": None}, INVALID),
    ({"cs": None}, INVALID), ({"slots": None}, INVALID), ({"cache": None}, INVALID), ({"ld_cs": 63}, INVALID),
    ({"max_pos": 0}, INVALID), ({"style": 2}, UNSUPPORTED), ({"bs": 48}, UNSUPPORTED), ({"stride": 8432}, INVALID),
    ({"stride": 8712}, UNSUPPORTED), ({"cache": MIS}, UNSUPPORTED), ({"fmt": 2}, UNSUPPORTED), ({"blocks": -1}, INVALID),
    ({"n": 0, "k": None}, OK)])
def test_k_insert_refusals(lib, change, status):
    assert lib.idx_k_norm_rope_quant_and_cache(*_args(K_INSERT, change)) == status


@pytest.mark.parametrize("change,status", [
    ({"n": -1}, INVALID), ({"dtype": 3}, UNSUPPORTED), ({"ld_c": 511}, INVALID), ({"ld_pe": 63}, INVALID),
    ({"eps": -1.0}, INVALID), ({"c": None}, INVALID), ({"pe": None}, INVALID), ({"pos": None}, INVALID),
    ({"cs": None}, INVALID), ({"slots": None}, INVALID), ({"cache": None}, INVALID), ({"ld_cs": 63}, INVALID),
    ({"max_pos": 0}, INVALID), ({"style": 2}, UNSUPPORTED), ({"bs": 48}, UNSUPPORTED), ({"stride": 41200}, INVALID),
    ({"stride": 41480}, UNSUPPORTED), ({"cache": MIS}, UNSUPPORTED), ({"blocks": -1}, INVALID),
    ({"n": 0, "c": None}, OK)])
def test_kv_insert_refusals(lib, change, status):
    assert lib.idx_kv_norm_rope_quant_and_cache(*_args(KV_INSERT, change)) == status


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, INVALID), ({"n_out": -1}, INVALID), ({"pages": -1}, INVALID), ({"ld_bt": 3}, INVALID),
    ({"ld_out": 575}, INVALID), ({"ld_out": 580}, UNSUPPORTED), ({"dtype": 2}, UNSUPPORTED), ({"out": MIS}, UNSUPPORTED),
    ({"cache": None}, INVALID), ({"bt": None}, INVALID), ({"cu": None}, INVALID), ({"out": None}, INVALID),
    ({"bs": 8}, UNSUPPORTED), ({"stride": 41200}, INVALID), ({"stride": 41480}, UNSUPPORTED),
    ({"cache": MIS}, UNSUPPORTED), ({"B": 0, "bt": None}, OK), ({"n_out": 0, "out": None}, OK)])
def test_gather_refusals(lib, change, status):
    assert lib.idx_gather_kv(*_args(GATHER, change)) == status


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, INVALID), ({"H": -1}, INVALID), ({"k": -1}, INVALID), ({"H": 1025}, UNSUPPORTED),
    ({"ld_slots": 31}, INVALID), ({"ld_q": 575}, INVALID), ({"ld_qh": 575}, INVALID), ({"ld_out": 511}, INVALID),
    ({"ld_oh": 511}, INVALID), ({"lse": P, "ld_lse": 7}, INVALID), ({"scale": math.inf}, INVALID),
    ({"scale": math.nan}, INVALID), ({"scale": 3e38}, INVALID), ({"q": None}, INVALID), ({"cache": None}, INVALID), ({"out": None}, INVALID),
    ({"slots": None}, INVALID), ({"bs": 24}, UNSUPPORTED), ({"stride": 41200}, INVALID), ({"stride": 41480}, UNSUPPORTED),
    ({"cache": MIS}, UNSUPPORTED), ({"span": 63}, UNSUPPORTED), ({"q": MIS}, UNSUPPORTED), ({"out": MIS}, UNSUPPORTED),
    ({"ld_q": 576 * 8 + 4}, UNSUPPORTED), ({"ld_qh": 580}, UNSUPPORTED), ({"ld_out": 512 * 8 + 4}, UNSUPPORTED),
    ({"ld_oh": 516}, UNSUPPORTED), ({"ws": MIS, "wsb": 1 << 40}, UNSUPPORTED), ({"T": 0, "q": None}, OK),
    ({"H": 0, "q": None}, OK)])
def test_attention_refusals(lib, change, status):
    assert lib.idx_sparse_attention(*_args(ATTN, change)) == status


def test_workspace_bytes_of_nothing(lib):
    for sizes in ((0, 8, 2048), (4, 0, 2048), (4, 8, 0), (-1, 8, 8)):
        assert lib.idx_sparse_attention_workspace_bytes(*sizes) == 0


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    f = torch.zeros
    i32, i64, u8, bf = torch.int32, torch.int64, torch.uint8, torch.bfloat16
    with pytest.raises(ValueError, match="CUDA tensor"):
        idx.idx_k_norm_rope_quant_and_cache(f(4, 128), f(128), None, 1e-6, f(4, dtype=i32), f(8, 64),
                                            f(4, dtype=i64), f(8, 8704, dtype=u8), 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        idx.idx_kv_norm_rope_quant_and_cache(f(4, 512), f(4, 64), None, 1e-6, None, None, f(4, dtype=i64),
                                             f(8, 41472, dtype=u8), 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        idx.idx_gather_kv(f(8, 41472, dtype=u8), 64, f(1, 8, dtype=i32), f(2, dtype=i32), f(4, 576))
    with pytest.raises(ValueError, match="CUDA tensor"):
        idx.idx_sparse_attention(f(4, 8, 576, dtype=bf), f(8, 41472, dtype=u8), 64, f(4, 32, dtype=i32),
                                 f(4, 8, 512, dtype=bf), 0.04)
    # the checks behind the device check, on what they see of a tensor
    with pytest.raises(ValueError, match="must be torch.int32"):
        idx._vec("f", "x", f(4), -1, i32, 4)
    with pytest.raises(ValueError, match="dimensions"):
        idx._mat("f", "x", f(4), -1, torch.float32, 4, 1)
    with pytest.raises(ValueError, match="shape"):
        idx._mat("f", "x", f(4, 3), -1, torch.float32, None, 4)
    with pytest.raises(ValueError, match="shape"):
        idx._vec("f", "x", f(5), -1, torch.float32, 4)
    with pytest.raises(ValueError, match="unit stride"):
        idx._mat("f", "x", f(4, 6)[:, ::2], -1, torch.float32, 4, 3)
    with pytest.raises(ValueError, match="unit stride"):
        idx._vec("f", "x", f(8)[::2], -1, torch.float32, 4)
    with pytest.raises(ValueError, match="unit stride"):
        idx._heads("f", "x", f(2, 3, 1152, dtype=bf)[:, :, ::2], -1, 2, 3, 576)
    with pytest.raises(ValueError, match="shape"):
        idx._heads("f", "x", f(2, 3, 576, dtype=bf), -1, 2, 4, 576)
    with pytest.raises(ValueError, match="go together"):
        idx._rope_args("f", None, f(8, 64), 4, -1)
    with pytest.raises(ValueError, match="go together"):
        idx._rope_args("f", f(4, dtype=i32), None, 4, -1)
    with pytest.raises(ValueError, match="64 columns"):
        idx._rope_args("f", f(4, dtype=i32), f(8, 63), 4, -1)
    with pytest.raises(ValueError, match="fewer than"):
        idx._cache_args("f", f(8, 41215, dtype=u8), -1, 64, 644)
    # strides of what has one row or one head only do not matter
    assert idx._mat("f", "x", f(1, 576)[:, :512], -1, torch.float32, 1, 512)[1] >= 512
    assert idx._heads("f", "x", f(1, 1, 576, dtype=bf), -1, 1, 1, 576)[1:] == (576, 576)
