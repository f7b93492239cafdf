"""GB300-native FP8 lightning indexer: Python binding over the C ABI of ``libidx.so``.

Every function here only marshals arguments (torch tensors -> device pointers,
row strides, the current CUDA stream) and calls the entry point of the same
name declared in ``include/idx.h``; every step of the computation runs in the
library's CUDA kernels. A non-OK status raises :class:`IdxError` with the
library's message. The library must have been built (``build.build_library``);
importing the binding without it works, calling it raises.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib

__all__ = [
    "IdxError", "idx_k_quant_and_cache", "idx_k_quant_and_cache_mxfp4", "idx_gather_k", "idx_gather_k_mxfp4",
    "idx_mqa_logits_prefill", "idx_mqa_logits_prefill_mxfp4", "idx_paged_mqa_logits_decode", "idx_paged_mqa_logits_decode_mxfp4", "idx_topk", "idx_expand_candidates", "idx_sparse_topk_remap",
    "idx_req_to_global_slots", "idx_dcp_topk_merge", "idx_q_rope_quant", "idx_block_span",
    "idx_workspace_bytes", "idx_device_error", "library",
    "idx_k_norm_rope_quant_and_cache", "idx_kv_norm_rope_quant_and_cache", "idx_gather_kv", "idx_sparse_attention",
    "idx_sparse_attention_workspace_bytes",
]


class IdxError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: status {status}: {message}")
        self.status = status


def library() -> ctypes.CDLL:
    return _lib.load()


def _check(fn: str, status: int) -> None:
    if status != _lib.IDX_OK:
        msg = library().idx_last_error().decode(errors="replace")
        raise IdxError(fn, status, msg)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _lib.IDX_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return _lib.IDX_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _rows(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("2-D tensor with unit column stride expected")
    return t.stride(0)


def idx_k_quant_and_cache(k, slot_mapping, cache, block_size, ue8m0=False, stream=None):
    """k [n, 128] bf16/f32, slot_mapping int64 [n], cache uint8 [num_blocks, block_stride].

    ``ue8m0``: power-of-two scales (the UE8M0 scale format) instead of amax / 448.
    """
    ld_k = _rows(k)
    _check("idx_k_quant_and_cache", library().idx_k_quant_and_cache(
        _ptr(k), _dtype_code(k), ld_k, k.shape[0], _ptr(slot_mapping), _ptr(cache),
        cache.shape[0], block_size, cache.stride(0),
        _lib.IDX_SCALE_UE8M0 if ue8m0 else _lib.IDX_SCALE_FP32, _stream(stream)))


def idx_k_quant_and_cache_mxfp4(k, slot_mapping, cache, block_size, stream=None):
    """k [n, 128] bf16/f32 -> MXFP4 cache uint8 [num_blocks, block_stride] (68 bytes per token)."""
    _check("idx_k_quant_and_cache_mxfp4", library().idx_k_quant_and_cache_mxfp4(
        _ptr(k), _dtype_code(k), _rows(k), k.shape[0], _ptr(slot_mapping), _ptr(cache),
        cache.shape[0], block_size, cache.stride(0), _stream(stream)))


def idx_gather_k(cache, block_size, block_table_row, n_tok, k8_out, kscale_out, stream=None):
    """Copy n_tok tokens of one request (block_table_row int32) into k8_out [n, 128] / kscale_out [n]."""
    _check("idx_gather_k", library().idx_gather_k(
        _ptr(cache), block_size, cache.stride(0), _ptr(block_table_row), n_tok, _ptr(k8_out),
        _ptr(kscale_out), _stream(stream)))


def idx_gather_k_mxfp4(cache, block_size, block_table_row, n_tok, codes_out, scales_out, stream=None):
    """Copy n_tok tokens of one request out of an MXFP4 cache into codes_out uint8 [n, 64] /
    scales_out int32 [n] (the words of four E8M0 codes)."""
    _check("idx_gather_k_mxfp4", library().idx_gather_k_mxfp4(
        _ptr(cache), block_size, cache.stride(0), _ptr(block_table_row), n_tok, _ptr(codes_out),
        _ptr(scales_out), _stream(stream)))


def _q_stride(q: torch.Tensor) -> int:
    if q.dim() != 3 or q.shape[1:] != (64, 128) or q.stride(2) != 1 or q.stride(1) != 128:
        raise ValueError("q must be uint8 [rows, 64, 128] with contiguous heads")
    return q.stride(0)


def idx_mqa_logits_prefill(q, w, k8, kscale, row_ks, row_ke, logits, sparse_idx=None, end=None,
                           sbk=0, n_si=None, ws=None, stream=None):
    """Dense (sparse_idx None) or sparse prefill logits; see include/idx.h."""
    ld_si = sparse_idx.stride(0) if sparse_idx is not None else 0
    if n_si is None:
        n_si = sparse_idx.shape[1] if sparse_idx is not None else 0
    _check("idx_mqa_logits_prefill", library().idx_mqa_logits_prefill(
        _ptr(q), _q_stride(q), _ptr(w), _dtype_code(w), _rows(w), _ptr(k8), _ptr(kscale),
        k8.shape[0], _ptr(row_ks), _ptr(row_ke), q.shape[0], _ptr(sparse_idx), ld_si, n_si,
        _ptr(end), sbk, _ptr(logits), _dtype_code(logits), _rows(logits), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def idx_mqa_logits_prefill_mxfp4(q, w, k_codes, k_scales, logits, sparse_idx, end, sbk, n_si=None, ws=None,
                                 stream=None):
    """Sparse prefill logits over gathered MXFP4 k (k_codes uint8 [S, 64], k_scales int32 [S])."""
    n_si = sparse_idx.shape[1] if n_si is None else n_si
    _check("idx_mqa_logits_prefill_mxfp4", library().idx_mqa_logits_prefill_mxfp4(
        _ptr(q), _q_stride(q), _ptr(w), _dtype_code(w), _rows(w), _ptr(k_codes), _ptr(k_scales),
        k_codes.shape[0], None, None, q.shape[0], _ptr(sparse_idx), sparse_idx.stride(0), n_si,
        _ptr(end), sbk, _ptr(logits), _dtype_code(logits), _rows(logits), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def idx_paged_mqa_logits_decode(q, w, cache, block_size, block_table, ctx_lens, logits, next_n=1,
                                sparse_idx=None, end=None, sbk=0, n_si=None, ws=None, stream=None):
    """Dense (sparse_idx None) or sparse decode logits read through the block table."""
    ld_si = sparse_idx.stride(0) if sparse_idx is not None else 0
    if n_si is None:
        n_si = sparse_idx.shape[1] if sparse_idx is not None else 0
    _check("idx_paged_mqa_logits_decode", library().idx_paged_mqa_logits_decode(
        _ptr(q), _q_stride(q), _ptr(w), _dtype_code(w), _rows(w), _ptr(cache), cache.shape[0],
        block_size, cache.stride(0), _ptr(block_table), _rows(block_table), _ptr(ctx_lens),
        ctx_lens.shape[0], next_n, _ptr(sparse_idx), ld_si, n_si, _ptr(end), sbk, _ptr(logits),
        _dtype_code(logits), _rows(logits), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def idx_paged_mqa_logits_decode_mxfp4(q, w, cache, block_size, block_table, ctx_lens, logits, next_n=1,
                                      sparse_idx=None, end=None, sbk=0, n_si=None, ws=None, stream=None):
    """idx_paged_mqa_logits_decode over an MXFP4 cache (dense next_n 1, or sparse)."""
    ld_si = sparse_idx.stride(0) if sparse_idx is not None else 0
    if n_si is None:
        n_si = sparse_idx.shape[1] if sparse_idx is not None else 0
    _check("idx_paged_mqa_logits_decode_mxfp4", library().idx_paged_mqa_logits_decode_mxfp4(
        _ptr(q), _q_stride(q), _ptr(w), _dtype_code(w), _rows(w), _ptr(cache), cache.shape[0],
        block_size, cache.stride(0), _ptr(block_table), _rows(block_table), _ptr(ctx_lens),
        ctx_lens.shape[0], next_n, _ptr(sparse_idx), ld_si, n_si, _ptr(end), sbk, _ptr(logits),
        _dtype_code(logits), _rows(logits), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def idx_topk(logits, row_ks, row_ke, k, out, vals=None, ws=None, stream=None, slots=None,
             block_table=None, block_size=None, block_span=None, row_to_req=None):
    """Per-row top-k indices (request-local), -1 filled; out int32 [rows, >= k]; optional scores.

    With ``slots`` (int32 [rows, >= k]) the slot conversion of idx_req_to_global_slots
    (``block_table``, ``block_size``, ``block_span``, ``row_to_req``) is fused into the
    selection's output pass (idx_topk_slots; no ``vals`` then)."""
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    if slots is None:
        _check("idx_topk", library().idx_topk(
            _ptr(logits), _dtype_code(logits), _rows(logits), _ptr(row_ks), _ptr(row_ke), logits.shape[0],
            k, _ptr(out), _rows(out), _ptr(vals), 0 if vals is None else _rows(vals), _ptr(ws), wsb,
            _stream(stream)))
        return
    if vals is not None:
        raise ValueError("idx_topk: the fused slot conversion has no score output")
    _check("idx_topk_slots", library().idx_topk_slots(
        _ptr(logits), _dtype_code(logits), _rows(logits), _ptr(row_ks), _ptr(row_ke), logits.shape[0],
        k, _ptr(out), _rows(out), _ptr(row_to_req), _ptr(block_table), _rows(block_table), block_size,
        block_span, _ptr(slots), _rows(slots), _ptr(ws), wsb, _stream(stream)))


def idx_q_rope_quant(q, positions, cos_sin, w, q8, w_out, softmax_scale, n_head_scale,
                     interleaved=False, stream=None):
    """Partial RoPE (dims 0-63), per-head e4m3 quantisation and folded weights.

    q [T, 64, 128] (or [T, 8192]) bf16/fp32, positions int32 [T], cos_sin fp32
    [max_pos, >= 64] (cos of the 32 pair angles, then sin), w [T, 64] bf16/fp32;
    writes q8 uint8 [T, 64, 128] and w_out [T, 64] (fp32 or bf16).
    """
    T = q.shape[0]
    q2 = q.reshape(T, -1) if q.dim() == 3 else q
    q8_2 = q8.reshape(T, -1) if q8.dim() == 3 else q8
    _check("idx_q_rope_quant", library().idx_q_rope_quant(
        _ptr(q2), _dtype_code(q2), _rows(q2) if T else 64 * 128, _ptr(positions), _ptr(cos_sin),
        _rows(cos_sin), cos_sin.shape[0], _lib.IDX_ROPE_INTERLEAVED if interleaved else _lib.IDX_ROPE_NEOX,
        _ptr(w), _dtype_code(w), _rows(w), float(softmax_scale), float(n_head_scale), T, _ptr(q8_2),
        _rows(q8_2) if T else 64 * 128, _ptr(w_out), _dtype_code(w_out), _rows(w_out), _stream(stream)))


def idx_dcp_topk_merge(cand_vals, cand_idx, shard_offset, k_local, k, out, vals=None, pos_stride=1,
                       stream=None):
    """Merge shard-local top-k candidates [rows, n_shards * k_local] into global top-k positions.

    ``shard_offset``: int32 [n_shards] shared by every row, int32 [rows, n_shards]
    per row, or None (offsets 0). Candidate index i of shard s maps to
    ``shard_offset[s] + i * pos_stride``.
    """
    if shard_offset is None:
        n_shards, ld_off = cand_vals.shape[1] // k_local, 0
    elif shard_offset.dim() == 1:
        n_shards, ld_off = shard_offset.shape[0], 0
    else:
        n_shards, ld_off = shard_offset.shape[1], _rows(shard_offset)
    _check("idx_dcp_topk_merge", library().idx_dcp_topk_merge(
        _ptr(cand_vals), _rows(cand_vals), _ptr(cand_idx), _rows(cand_idx), _ptr(shard_offset), ld_off,
        n_shards, pos_stride, k_local, cand_vals.shape[0], k, _ptr(out), _rows(out), _ptr(vals),
        0 if vals is None else _rows(vals), _stream(stream)))


def idx_expand_candidates(cand, row_ks, row_ke, cand_block_size, sbk, sparse_idx, end, stream=None):
    """cand int32 [rows, n_cand] -> sparse_idx int32 [rows, n_cand * R], end int32 [rows]."""
    _check("idx_expand_candidates", library().idx_expand_candidates(
        _ptr(cand), _rows(cand), cand.shape[0], cand.shape[1], _ptr(row_ks), _ptr(row_ke),
        cand_block_size, sbk, _ptr(sparse_idx), _rows(sparse_idx), _ptr(end), _stream(stream)))


def idx_sparse_topk_remap(sparse_logits, end, sparse_idx, row_ks, sbk, k, positions, col_scratch=None,
                          ws=None, stream=None, slots=None, block_table=None, block_size=None,
                          block_span=None, row_to_req=None):
    """Top-k over sparse columns [0, end) then column -> request-local position.

    With ``slots`` the slot conversion is fused into the output pass
    (idx_sparse_topk_remap_slots), as for idx_topk."""
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    if slots is None:
        _check("idx_sparse_topk_remap", library().idx_sparse_topk_remap(
            _ptr(sparse_logits), _dtype_code(sparse_logits), _rows(sparse_logits), _ptr(end),
            _ptr(sparse_idx), _rows(sparse_idx), _ptr(row_ks), sbk, sparse_logits.shape[0], k,
            _ptr(col_scratch), 0 if col_scratch is None else _rows(col_scratch), _ptr(positions),
            _rows(positions), _ptr(ws), wsb, _stream(stream)))
        return
    _check("idx_sparse_topk_remap_slots", library().idx_sparse_topk_remap_slots(
        _ptr(sparse_logits), _dtype_code(sparse_logits), _rows(sparse_logits), _ptr(end),
        _ptr(sparse_idx), _rows(sparse_idx), _ptr(row_ks), sbk, sparse_logits.shape[0], k,
        _ptr(col_scratch), 0 if col_scratch is None else _rows(col_scratch), _ptr(positions),
        _rows(positions), _ptr(row_to_req), _ptr(block_table), _rows(block_table), block_size,
        block_span, _ptr(slots), _rows(slots), _ptr(ws), wsb, _stream(stream)))


def idx_req_to_global_slots(local, row_to_req, block_table, block_size, block_span, slots, k=None,
                            stream=None):
    """Request-local positions int32 [rows, k] -> physical slots (block * block_span + offset)."""
    kk = local.shape[1] if k is None else k
    _check("idx_req_to_global_slots", library().idx_req_to_global_slots(
        _ptr(local), _rows(local), local.shape[0], kk, _ptr(row_to_req), _ptr(block_table),
        _rows(block_table), block_size, block_span, _ptr(slots), _rows(slots), _stream(stream)))


def _refuse(fn: str, name: str, t, dev: int, dtype, shape) -> None:
    """Say what is wrong with ``t`` as argument ``name`` (shape entries None: any extent)."""
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} must be a tensor on cuda:{dev}, got one on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    have = tuple(t.shape)
    if len(have) != len(shape):
        raise ValueError(f"{fn}: {name} must have {len(shape)} dimensions, got {len(have)}")
    if any(w is not None and h != w for h, w in zip(have, shape)):
        raise ValueError(f"{fn}: {name} has shape {have}, expected {shape}")
    if max(have) > _MAX_EXTENT:
        raise ValueError(f"{fn}: {name} has shape {have}: extents of 2**31 and more are not taken")
    raise ValueError(f"{fn}: {name} must have a unit stride in its last dimension")


_MAX_EXTENT = (1 << 31) - 1  # the entry points take extents in 32 bits, and ctypes would cut what exceeds them


def _int32(fn: str, name: str, v: int) -> int:
    if not -_MAX_EXTENT - 1 <= v <= _MAX_EXTENT:
        raise ValueError(f"{fn}: {name} {v} does not fit in 32 bits")
    return v


def _vec(fn: str, name: str, t, dev: int, dtype, n: int) -> int:
    """Device pointer of the contiguous vector ``t`` [n]. These checks run on every call of a decode step, so the
    common case is one expression."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == (n,) and (n < 2 or t.stride(0) == 1):
        return t.data_ptr()
    _refuse(fn, name, t, dev, dtype, (n,))


def _mat(fn: str, name: str, t, dev: int, dtype, rows, cols):
    """(device pointer, row stride) of ``t`` [rows, cols] with contiguous rows (None: any extent). Of one row or
    none, any stride serves."""
    if t.get_device() == dev and t.dtype is dtype and t.dim() == 2:
        r, c = t.shape
        if (rows is None or r == rows) and (cols is None or c == cols):
            ld, step = t.stride()
            if (step == 1 or c < 2) and r <= _MAX_EXTENT and c <= _MAX_EXTENT:
                return t.data_ptr(), ld if r > 1 or ld > c else c
    _refuse(fn, name, t, dev, dtype, (rows, cols))


def _heads(fn: str, name: str, t, dev: int, rows, heads, dims: int):
    """(device pointer, row stride, head stride) of the bf16 ``t`` [rows, heads, dims]."""
    if t.get_device() == dev and t.dtype is torch.bfloat16 and t.dim() == 3:
        r, h, d = t.shape
        if d == dims and (rows is None or r == rows) and (heads is None or h == heads):
            ld, ldh, step = t.stride()
            if step == 1 and r <= _MAX_EXTENT and h <= _MAX_EXTENT:
                return t.data_ptr(), ld if r > 1 else dims, ldh if h > 1 else dims
    _refuse(fn, name, t, dev, torch.bfloat16, (rows, heads, dims))


def _cuda_device(fn: str, name: str, t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    return dev


_ENTRY = {}  # entry points by name


def _call(fn: str, dev: int, stream, *args) -> None:
    """Call entry point ``fn`` with ``stream`` (None: torch's current one of the tensors' device) on that device."""
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        if stream.device_index != dev:
            raise ValueError(f"{fn}: the stream belongs to cuda:{stream.device_index}, the tensors to cuda:{dev}")
        st = stream.cuda_stream
    else:
        st = int(stream)
    f = _ENTRY.get(fn)
    if f is None:
        f = _ENTRY[fn] = getattr(library(), fn)
    if dev == torch._C._cuda_getDevice():
        status = f(*args, st)
    else:
        with torch.cuda.device(dev):
            status = f(*args, st)
    if status:
        _check(fn, status)


def _rope_args(fn: str, positions, cos_sin, n: int, dev: int):
    if positions is None or cos_sin is None:
        if positions is not cos_sin:
            raise ValueError(f"{fn}: positions and cos_sin go together")
        return None, None, 64, 1
    c, ld = _mat(fn, "cos_sin", cos_sin, dev, torch.float32, None, None)
    max_pos, cols = cos_sin.shape
    if cols < 64:
        raise ValueError(f"{fn}: cos_sin needs 64 columns, got {cols}")
    return _vec(fn, "positions", positions, dev, torch.int32, n), c, ld, max_pos


def _cache_args(fn: str, cache, dev: int, block_size: int, token_bytes: int):
    p, ld = _mat(fn, "cache", cache, dev, torch.uint8, None, None)
    blocks, size = cache.shape
    if size < block_size * token_bytes:
        raise ValueError(f"{fn}: cache blocks of {size} bytes hold fewer than {block_size} tokens")
    return p, blocks, block_size, ld


def idx_k_norm_rope_quant_and_cache(k, weight, bias, eps, positions, cos_sin, slot_mapping, cache, block_size,
                                    ue8m0=False, interleaved=False, stream=None):
    """LayerNorm, partial RoPE, e4m3 quantisation and insert of the indexer's k, in one pass.

    k [n, 128] bf16/fp32 (the raw projection), weight / bias fp32 [128] (bias may be None), positions int32
    [n], cos_sin fp32 [max_pos, >= 64], slot_mapping int64 [n], cache uint8 [num_blocks, block_stride] (the
    indexer cache of idx_k_quant_and_cache).
    """
    fn = "idx_k_norm_rope_quant_and_cache"
    dev = _cuda_device(fn, "k", k)
    bf16 = k.dtype is torch.bfloat16
    kp, ld_k = _mat(fn, "k", k, dev, torch.bfloat16 if bf16 else torch.float32, None, 128)
    n = k.shape[0]
    if positions is None:
        raise ValueError(f"{fn}: positions and cos_sin are required")
    _call(fn, dev, stream, kp, _lib.IDX_BF16 if bf16 else _lib.IDX_F32, ld_k, n,
          _vec(fn, "weight", weight, dev, torch.float32, 128),
          None if bias is None else _vec(fn, "bias", bias, dev, torch.float32, 128), eps,
          *_rope_args(fn, positions, cos_sin, n, dev),
          _lib.IDX_ROPE_INTERLEAVED if interleaved else _lib.IDX_ROPE_NEOX,
          _vec(fn, "slot_mapping", slot_mapping, dev, torch.int64, n), *_cache_args(fn, cache, dev, block_size, 132),
          _lib.IDX_SCALE_UE8M0 if ue8m0 else _lib.IDX_SCALE_FP32)


def idx_kv_norm_rope_quant_and_cache(c, pe, weight, eps, positions, cos_sin, slot_mapping, cache, block_size,
                                     interleaved=False, stream=None):
    """RMSNorm, RoPE, e4m3 quantisation and insert of the attention latent, in one pass.

    c [n, 512] and pe [n, 64] bf16/fp32 (column slices of one projection will do), weight fp32 [512] or None
    (no norm), positions int32 [n] and cos_sin fp32 [max_pos, >= 64] or both None (already rotated),
    slot_mapping int64 [n], cache uint8 [num_blocks, block_stride] (644 bytes per token).
    """
    fn = "idx_kv_norm_rope_quant_and_cache"
    dev = _cuda_device(fn, "c", c)
    bf16 = c.dtype is torch.bfloat16
    dt = torch.bfloat16 if bf16 else torch.float32
    cp, ld_c = _mat(fn, "c", c, dev, dt, None, 512)
    n = c.shape[0]
    _call(fn, dev, stream, cp, ld_c, *_mat(fn, "pe", pe, dev, dt, n, 64), _lib.IDX_BF16 if bf16 else _lib.IDX_F32, n,
          None if weight is None else _vec(fn, "weight", weight, dev, torch.float32, 512), eps,
          *_rope_args(fn, positions, cos_sin, n, dev),
          _lib.IDX_ROPE_INTERLEAVED if interleaved else _lib.IDX_ROPE_NEOX,
          _vec(fn, "slot_mapping", slot_mapping, dev, torch.int64, n), *_cache_args(fn, cache, dev, block_size, 644))


def idx_gather_kv(cache, block_size, block_table, cu_lens, out, starts=None, stream=None):
    """Read the tokens of a batch of requests back, dequantised and packed.

    block_table int32 [B, pages], cu_lens int32 [B + 1] (first output row of each request, ascending), starts
    int32 [B] or None (first token of each request), out [n_out, 576] bf16/fp32; rows past cu_lens[B] are left
    as they were.
    """
    fn = "idx_gather_kv"
    dev = _cuda_device(fn, "out", out)
    bf16 = out.dtype is torch.bfloat16
    op, ld_out = _mat(fn, "out", out, dev, torch.bfloat16 if bf16 else torch.float32, None, 576)
    bt, ld_bt = _mat(fn, "block_table", block_table, dev, torch.int32, None, None)
    B, pages = block_table.shape
    # pages beyond the table's own columns do not exist, whatever its row stride
    _call(fn, dev, stream, *_cache_args(fn, cache, dev, block_size, 644), bt, ld_bt, pages,
          None if starts is None else _vec(fn, "starts", starts, dev, torch.int32, B),
          _vec(fn, "cu_lens", cu_lens, dev, torch.int32, B + 1), B, op, _lib.IDX_BF16 if bf16 else _lib.IDX_F32,
          ld_out, out.shape[0])


def idx_sparse_attention_workspace_bytes(rows: int, heads: int, topk: int) -> int:
    """Bytes of the workspace with which idx_sparse_attention splits these rows' lists (0: it would not)."""
    fn = "idx_sparse_attention_workspace_bytes"
    return library().idx_sparse_attention_workspace_bytes(
        _int32(fn, "rows", rows), _int32(fn, "heads", heads), _int32(fn, "topk", topk))


def idx_sparse_attention(q, cache, block_size, slots, out, softmax_scale, lse=None, n_sel=None, block_span=None,
                         ws=None, stream=None):
    """Attention of each query row over the tokens selected for it.

    q bf16 [T, H, 576], cache uint8 [num_blocks, block_stride] (644 bytes per token), slots int32 [T, k] (block *
    block_span + offset, -1 = empty), out bf16 [T, H, 512], lse fp32 [T, H] or None, n_sel int32 [T] or None (the
    list entries used), ws: a contiguous tensor of idx_sparse_attention_workspace_bytes(T, H, k) bytes, or None.
    """
    fn = "idx_sparse_attention"
    dev = _cuda_device(fn, "q", q)
    qp, ld_q, ld_qh = _heads(fn, "q", q, dev, None, None, 576)
    T, H, _ = q.shape
    op, ld_out, ld_oh = _heads(fn, "out", out, dev, T, H, 512)
    sp, ld_slots = _mat(fn, "slots", slots, dev, torch.int32, T, None)
    wp, wb = None, 0
    if ws is not None:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"{fn}: ws must be a contiguous tensor on cuda:{dev}")
        wp, wb = ws.data_ptr(), ws.numel() * ws.element_size()
    lp, ld_lse = (None, 0) if lse is None else _mat(fn, "lse", lse, dev, torch.float32, T, H)
    cp, blocks, bs, stride = _cache_args(fn, cache, dev, block_size, 644)
    _call(fn, dev, stream, qp, ld_q, ld_qh, cp, blocks, bs, stride,
          bs if block_span is None else _int32(fn, "block_span", block_span), sp,
          ld_slots, slots.shape[1], None if n_sel is None else _vec(fn, "n_sel", n_sel, dev, torch.int32, T), T, H,
          softmax_scale, op, ld_out, ld_oh, lp, ld_lse, wp, wb)


def idx_block_span(block_stride: int, token_stride: int) -> int:
    span = ctypes.c_int32(0)
    _check("idx_block_span", library().idx_block_span(block_stride, token_stride, ctypes.byref(span)))
    return span.value


def idx_workspace_bytes(op: str, rows: int, max_cols: int, k: int) -> int:
    return library().idx_workspace_bytes(_lib.OPS[op], rows, max_cols, k)


def idx_device_error(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a device-side failure."""
    _check("idx_device_error", library().idx_device_error(_stream(stream)))
