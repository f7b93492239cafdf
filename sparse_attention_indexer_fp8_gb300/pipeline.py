"""Orchestration of whole indexer steps over the C ABI (no arithmetic of its own).

``fill_paged_cache`` inserts a workload's k into a device cache through
``idx_k_quant_and_cache``; ``DecodeStep`` owns the device buffers of one dense
decode step (k insert of the new tokens, paged logits, top-k, slot conversion)
``HierarchicalStep`` those of one V4.1 consumer-layer step (candidate
expansion, sparse logits, sparse top-k with remap, slot conversion), and
``DcpDecodeStep`` those of one rank of a context-parallel decode step (scoring
of the rank's own shard, local top-k with scores, one exchange, merge).
``AttentionDecodeStep`` goes from a layer's projections to its attention output
(both normalised inserts, q preparation, ``DecodeStep``, sparse attention).
``TreeStep`` verifies trees of drafted tokens: tables and masks once a step, then a
layer's insert and its attention over whole contexts. Buffers are allocated once
at construction; ``run`` allocates nothing but the exchange's
receive lists. ``kv="mxfp4"`` selects the MXFP4 indexer cache (the V4.1 format)
for the cache fill and the decode and hierarchical steps.
"""

from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import (idx_build_tables, idx_dcp_topk_merge, idx_expand_candidates, idx_k_norm_rope_quant_and_cache,
               idx_k_quant_and_cache, idx_k_quant_and_cache_mxfp4, idx_kv_norm_rope_quant_and_cache,
               idx_paged_attention_workspace_bytes, idx_paged_mqa_logits_decode, idx_paged_mqa_logits_decode_mxfp4,
               idx_q_rope_quant, idx_req_to_global_slots, idx_sparse_attention, idx_sparse_attention_workspace_bytes,
               idx_sparse_topk_remap, idx_topk, idx_tree_attention, idx_tree_mask, idx_workspace_bytes, _heads, _mat, _vec)
from . import workloads as W


def _workspace(op: str, rows: int, ld: int, k: int, device) -> torch.Tensor | None:
    """The selection workspace (first-digit histograms, zero between steps), or None
    where the selection of these rows would not read it."""
    with torch.cuda.device(torch.device(device)):
        nbytes = idx_workspace_bytes(op, rows, ld, k)
    return torch.zeros((nbytes // 4,), dtype=torch.int32, device=device).view(rows, 1024) if nbytes else None


def _stream_context(stream, device):
    """Torch's operations on the stream that a call was given (None: they stay on the device's current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device))


def _insert(kv: str):
    return idx_k_quant_and_cache_mxfp4 if kv == "mxfp4" else idx_k_quant_and_cache


def _decode_logits(kv: str):
    return idx_paged_mqa_logits_decode_mxfp4 if kv == "mxfp4" else idx_paged_mqa_logits_decode


def cache_block_stride(kv: str = "fp8", block_size: int = W.BLOCK_SIZE) -> int:
    """Bytes per block of the cache format (512-byte aligned): 8704 (e4m3) or 4608 (MXFP4) for 64 tokens."""
    return W.mxfp4_block_stride_bytes(block_size) if kv == "mxfp4" else W.block_stride_bytes(block_size)


def fill_paged_cache(pool: W.PagedPool, seed: int, cache: torch.Tensor, device_k: bool = False,
                     chunk_tokens: int = 1 << 21, stream=None, kv: str = "fp8") -> None:
    """Quantise and insert every request's k into ``cache`` through the cache format's insert.

    k comes from ``workloads.make_k`` (host generator) or, with ``device_k``,
    from ``workloads.make_k_device`` (for pools too large to draw on the host).
    """
    idx_k_quant_and_cache = _insert(kv)
    dev = cache.device
    if device_k:
        for b in range(len(pool.ctx_lens)):
            L = int(pool.ctx_lens[b])
            k = W.make_k_device(seed, b, L, dev)
            s = torch.from_numpy(pool.slot_mapping(b)).to(dev)
            idx_k_quant_and_cache(k, s, cache, pool.block_size, stream=stream)
        torch.cuda.current_stream(dev).synchronize()
        return
    pend_k, pend_s, n = [], [], 0

    def flush():
        nonlocal pend_k, pend_s, n
        if not pend_k:
            return
        k = torch.from_numpy(np.concatenate(pend_k).view(np.int16)).to(dev)
        s = torch.from_numpy(np.concatenate(pend_s)).to(dev)
        idx_k_quant_and_cache(k.view(torch.bfloat16), s, cache, pool.block_size, stream=stream)
        torch.cuda.current_stream(dev).synchronize()
        pend_k, pend_s, n = [], [], 0

    for b in range(len(pool.ctx_lens)):
        L = int(pool.ctx_lens[b])
        pend_k.append(W.make_k(seed, b, L))
        pend_s.append(pool.slot_mapping(b))
        n += L
        if n >= chunk_tokens:
            flush()
    flush()


class DecodeStep:
    """One dense decode step of the indexer for a fixed batch shape."""

    def __init__(self, batch: int, max_ctx: int, topk: int = W.TOPK, next_n: int = 1,
                 block_size: int = W.BLOCK_SIZE, block_span: int | None = None, device="cuda",
                 kv: str = "fp8"):
        rows = batch * next_n
        self.batch, self.next_n, self.topk = batch, next_n, topk
        self.insert, self.logits_call = _insert(kv), _decode_logits(kv)
        self.block_size = block_size
        self.block_span = block_size if block_span is None else block_span
        ld = (max_ctx + 63) // 64 * 64   # 256-byte aligned rows: vector loads in the selection
        self.logits = torch.empty((rows, ld), dtype=torch.float32, device=device)
        self.local = torch.empty((rows, topk), dtype=torch.int32, device=device)
        self.slots = torch.empty((rows, topk), dtype=torch.int32, device=device)
        self.row_ke = torch.empty(rows, dtype=torch.int32, device=device)
        # No selection workspace: without the first-digit histogram the scoring
        # kernel keeps five k stages in flight instead of four, which saves more
        # than the selection's own first-digit sweep costs (128K decode step
        # 282.3 -> 281.3 us, 64 x U[8K,32K] 49.9 -> 49.4 us on a GB300).
        self.ws = None

    def run(self, q, w, cache, block_table, ctx_lens, new_k=None, new_slots=None, row_ke=None,
            stream=None):
        """Insert new k (optional), score, select, convert; returns the slot table."""
        if new_k is not None:
            self.insert(new_k, new_slots, cache, self.block_size, stream=stream)
        self.logits_call(q, w, cache, self.block_size, block_table, ctx_lens, self.logits,
                         next_n=self.next_n, ws=self.ws, stream=stream)
        ke = ctx_lens if (row_ke is None and self.next_n == 1) else row_ke
        # selection with the slot conversion fused into its output pass
        idx_topk(self.logits, None, ke, self.topk, self.local, ws=self.ws, stream=stream,
                 slots=self.slots, block_table=block_table, block_size=self.block_size,
                 block_span=self.block_span,
                 row_to_req=None if self.next_n == 1 else self._row_to_req(ctx_lens))
        return self.slots

    def _row_to_req(self, ctx_lens):
        if not hasattr(self, "_r2r"):
            self._r2r = torch.arange(self.batch, dtype=torch.int32, device=ctx_lens.device)
            self._r2r = self._r2r.repeat_interleave(self.next_n)
        return self._r2r


class HierarchicalStep:
    """One V4.1 decode step for the consumer layers: expand once, then score, select + remap, slots.

    [V41] 功能与动机 / 实现拆解 item 2: the candidate expansion (and the schedule)
    is done once per step and shared by every consumer layer of that step;
    ``expand`` fills ``sparse_idx`` / ``end`` and ``score`` runs one layer on
    them (any number of times, the expansion buffers are only read). With
    ``next_n > 1`` (multi-token prediction) every request has ``next_n`` query
    rows, row ``r`` belonging to request ``r // next_n``, each with its own
    causal limit (``row_ke``) and candidates.
    """

    def __init__(self, rows: int, n_cand: int, cand_block_size: int = 64, sbk: int = 64,
                 topk: int = W.TOPK, block_size: int = W.BLOCK_SIZE, device="cuda", next_n: int = 1,
                 kv: str = "fp8"):
        R = cand_block_size // sbk
        self.logits_call = _decode_logits(kv)
        self.cand_block_size, self.sbk, self.topk, self.block_size = cand_block_size, sbk, topk, block_size
        self.next_n = next_n
        self.sparse_idx = torch.empty((rows, n_cand * R), dtype=torch.int32, device=device)
        self.end = torch.empty(rows, dtype=torch.int32, device=device)
        self.logits = torch.empty((rows, n_cand * R * sbk), dtype=torch.bfloat16, device=device)
        self.cols = torch.empty((rows, topk), dtype=torch.int32, device=device)
        self.positions = torch.empty((rows, topk), dtype=torch.int32, device=device)
        self.slots = torch.empty((rows, topk), dtype=torch.int32, device=device)
        self.ws = _workspace("sparse_topk_remap", rows, n_cand * R * sbk, topk, device)
        self.row_to_req = (None if next_n == 1 else
                           torch.arange(rows // next_n, dtype=torch.int32, device=device).repeat_interleave(next_n))

    def expand(self, cand, ctx_lens, row_ke=None, stream=None):
        """Once per step. ``row_ke`` (int32 [rows]) is required when ``next_n > 1``."""
        ke = ctx_lens if row_ke is None else row_ke
        idx_expand_candidates(cand, None, ke, self.cand_block_size, self.sbk, self.sparse_idx, self.end,
                              stream=stream)

    def score(self, q, w, cache, block_table, ctx_lens, stream=None):
        """One consumer layer on the current expansion; returns the slot table."""
        self.logits_call(q, w, cache, self.block_size, block_table, ctx_lens, self.logits,
                         next_n=self.next_n, sparse_idx=self.sparse_idx, end=self.end,
                         sbk=self.sbk, ws=self.ws, stream=stream)
        idx_sparse_topk_remap(self.logits, self.end, self.sparse_idx, None, self.sbk, self.topk,
                              self.positions, col_scratch=self.cols, ws=self.ws, stream=stream,
                              slots=self.slots, block_table=block_table, block_size=self.block_size,
                              block_span=self.block_size, row_to_req=self.row_to_req)
        return self.slots

    def run(self, q, w, cache, block_table, ctx_lens, cand, row_ke=None, stream=None):
        self.expand(cand, ctx_lens, row_ke, stream=stream)
        return self.score(q, w, cache, block_table, ctx_lens, stream=stream)


class AttentionDecodeStep:
    """One layer's dense decode step from its projections to the attention output, one query row per request.

    [DSA] data-flow items 1-3: the new token's indexer k and attention latent are
    normalised, rotated and inserted into their caches, the indexer's q is
    prepared, ``DecodeStep`` scores and selects, and every head attends to the selected
    slots. Both caches share block tables and slots. ``run`` allocates nothing.
    ``softmax_scale`` is that of the heads before absorption, which keeps their dot products:
    by default 192 ** -0.5 (128 dims without position, 64 with); a model whose context was
    extended with a factor on the logits passes the product of the two.
    """

    def __init__(self, batch: int, max_ctx: int, heads: int, topk: int = W.TOPK, block_size: int = W.BLOCK_SIZE,
                 device="cuda", softmax_scale: float = W.ATTN_HEAD_DIM ** -0.5, eps: float = 1e-6,
                 interleaved: bool = False, index_interleaved: bool = False):
        self.block_size, self.softmax_scale, self.eps = block_size, softmax_scale, eps
        # pairing of the rotary dims of the attention latent and of the indexer's q and k
        self.interleaved, self.index_interleaved = interleaved, index_interleaved
        self.indexer = DecodeStep(batch, max_ctx, topk=topk, block_size=block_size, device=device)
        self.q8 = torch.empty((batch, 64, 128), dtype=torch.uint8, device=device)
        self.w = torch.empty((batch, 64), dtype=torch.float32, device=device)
        self.out = torch.empty((batch, heads, 512), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((batch, heads), dtype=torch.float32, device=device)
        with torch.cuda.device(self.out.device):
            nbytes = idx_sparse_attention_workspace_bytes(batch, heads, topk)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None

    def make_caches(self, num_blocks: int):
        """Zeroed (indexer, attention) caches of ``num_blocks`` blocks."""
        return tuple(torch.zeros((num_blocks, stride), dtype=torch.uint8, device=self.out.device)
                     for stride in (W.block_stride_bytes(self.block_size), W.kv_block_stride_bytes(self.block_size)))

    def _check_batch(self, new_k, q_index, w_index, q, block_table, ctx_lens):
        """Refuse what is not of the step's batch before anything is enqueued: the q preparation, the scoring and the
        selection take the step's own buffers and read as many rows of these."""
        fn, dev, (batch, heads, _) = "AttentionDecodeStep", self.out.get_device(), self.out.shape
        _vec(fn, "ctx_lens", ctx_lens, dev, torch.int32, batch)
        _mat(fn, "block_table", block_table, dev, torch.int32, None, None)
        _heads(fn, "q", q, dev, batch, heads, W.ATTN_DIM)
        for name, t in (("new_k", new_k), ("block_table", block_table), ("w_index", w_index)):
            if t.shape[0] < batch:
                raise ValueError(f"{fn}: {name} has {t.shape[0]} rows, the batch {batch}")
        if not (q_index.shape == self.q8.shape or (q_index.dim() == 2 and q_index.shape[0] == batch
                                                   and q_index.shape[1] >= 64 * 128)):
            raise ValueError(f"{fn}: q_index has shape {tuple(q_index.shape)}, expected {tuple(self.q8.shape)}")
        if w_index.dim() != 2 or w_index.shape[1] < 64:
            raise ValueError(f"{fn}: w_index has shape {tuple(w_index.shape)}, expected {(batch, 64)}")
        if q_index.get_device() != dev or w_index.get_device() != dev:
            raise ValueError(f"{fn}: q_index and w_index must be on {self.out.device}")

    def insert(self, k, kv, k_weight, k_bias, kv_weight, positions, cos_sin, slots, k_cache, kv_cache, stream=None):
        """Any number of tokens: indexer k [n, 128] and attention projection [n, 576] into both caches."""
        idx_k_norm_rope_quant_and_cache(k, k_weight, k_bias, self.eps, positions, cos_sin, slots, k_cache,
                                        self.block_size, interleaved=self.index_interleaved, stream=stream)
        idx_kv_norm_rope_quant_and_cache(kv[:, :512], kv[:, 512:], kv_weight, self.eps, positions, cos_sin, slots,
                                         kv_cache, self.block_size, interleaved=self.interleaved, stream=stream)

    def run(self, new_k, new_kv, k_weight, k_bias, kv_weight, positions, cos_sin, new_slots, q_index, w_index, q,
            k_cache, kv_cache, block_table, ctx_lens, stream=None):
        """``ctx_lens`` (int32 [batch], at most ``max_ctx``) count the new token; ``q`` [batch, heads, 576] is the
        absorbed and rotated query. A request that sits a step out has length 0 and a negative slot."""
        self._check_batch(new_k, q_index, w_index, q, block_table, ctx_lens)
        # the q preparation, the scoring and the selection run on the current device and its current stream
        with torch.cuda.device(self.out.device):
            self.insert(new_k, new_kv, k_weight, k_bias, kv_weight, positions, cos_sin, new_slots, k_cache, kv_cache,
                        stream=stream)
            idx_q_rope_quant(q_index, positions, cos_sin, w_index, self.q8, self.w, 128 ** -0.5, 64 ** -0.5,
                             interleaved=self.index_interleaved, stream=stream)
            slots = self.indexer.run(self.q8, self.w, k_cache, block_table, ctx_lens, stream=stream)
            # the lists of contexts shorter than topk end with -1: nothing past a context's length is looked at
            idx_sparse_attention(q, kv_cache, self.block_size, slots, self.out, self.softmax_scale, lse=self.lse,
                                 n_sel=ctx_lens, ws=self.ws, stream=stream)
        return self.out


class TreeStep:
    """Verification of drafted trees over the attention cache, for up to ``requests`` requests and ``rows`` new tokens.

    ``plan`` prepares a step from the requests' lengths and the nodes' parents, once for all layers: blocks and slots
    of the new tokens, their positions (the request's length and the node's depth) and who sees whom. ``layer`` inserts
    a layer's new tokens and attends to every request's earlier tokens and each node's ancestors. A prompt is nodes whose
    parent is the one before (32 ``words`` nodes a request at most; longer prompts go through ``idx_window_attention``).

    Records lie in the order of the tree. Accepted nodes that are its first, each the child of the one before, are where the
    sequence wants them: the next step's ``cached_lens`` count them. Any other accepted path is brought again by the next
    step, as a chain before its tree, and costs as many rows once more. The records of dropped nodes are overwritten, and
    their blocks used again, by the next step over the same ``cached_lens``. Rows behind the last node are padding.

    Up to 160 ``requests``, those that sit a step out among them, the attention shares its work out evenly over the GPU;
    with more, a step of few live requests with long contexts takes several times as long. Neither call allocates anything.
    """

    def __init__(self, requests: int, rows: int, heads: int, words: int = 2, block_size: int = W.BLOCK_SIZE,
                 device="cuda", softmax_scale: float = W.ATTN_HEAD_DIM ** -0.5, eps: float = 1e-6,
                 interleaved: bool = False):
        # what the second call of ``plan`` or ``layer`` would refuse, when the first is enqueued already
        for name, value, most in (("requests", requests, 8192), ("heads", heads, 1024), ("words", words, 32)):
            if not (name == "words") <= value <= most:
                raise ValueError(f"TreeStep: {name} {value}, at most {most} are taken")
        if block_size not in (16, 32, 64, 128):
            raise ValueError(f"TreeStep: block_size {block_size} is not one of 16, 32, 64, 128")
        if not abs(softmax_scale) < 2.358e38:  # times log2(e) it is a binary32 number
            raise ValueError(f"TreeStep: softmax_scale {softmax_scale}")
        self.block_size, self.softmax_scale, self.eps, self.interleaved = block_size, softmax_scale, eps, interleaved

        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=device)

        self.ctx_lens, self.cu_rows = ints(requests), ints(requests + 1)
        self.base_lens = ints(requests)
        self.held_pages, self.free_end = ints(requests), ints(1)
        self.row_positions, self.slots = ints(rows), ints(rows, dtype=torch.int64)
        self.positions, self.mask = ints(rows), ints(rows, words)
        self.out = torch.zeros((rows, heads, 512), dtype=torch.bfloat16, device=device)
        self.lse = torch.zeros((rows, heads), dtype=torch.float32, device=device)
        with torch.cuda.device(self.out.device):
            nbytes = idx_paged_attention_workspace_bytes(rows, requests, heads)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None

    def plan(self, cached_lens, new_lens, parents, free_blocks, block_table, held_pages=None, free_start=None,
             stream=None):
        """Lengths and ``held_pages`` int32 [requests], ``parents`` int32 [rows] (within the request, -1: none);
        ``block_table`` is updated. ``cached_lens``, ``held_pages`` and ``free_start`` may be the step's own ``ctx_lens``,
        ``held_pages`` and ``free_end``, which go on from step to step then. See ``idx_build_tables`` and ``idx_tree_mask``."""
        # the masks' arguments, before the tables count a block: after a refusal the same plan may be tried again
        fn, dev = "TreeStep", self.out.get_device()
        _vec(fn, "cached_lens", cached_lens, dev, torch.int32, self.ctx_lens.shape[0])
        _vec(fn, "parents", parents, dev, torch.int32, self.positions.shape[0])
        base = cached_lens
        if cached_lens.data_ptr() == self.ctx_lens.data_ptr():
            # the tables advance it, and the nodes' positions count from what it was before
            base = self.base_lens
            with _stream_context(stream, self.ctx_lens.device):
                base.copy_(cached_lens)
        idx_build_tables(cached_lens, new_lens, free_blocks, block_table, self.block_size, self.ctx_lens, self.cu_rows,
                         self.row_positions, self.slots, held_pages=held_pages, held_out=self.held_pages,
                         free_start=free_start, free_end=self.free_end, stream=stream)
        idx_tree_mask(parents, self.cu_rows, self.mask, base_lens=base, positions=self.positions, stream=stream)

    def layer(self, kv, kv_weight, cos_sin, q, kv_cache, block_table, stream=None):
        """``kv`` [rows, 576] is the attention projection, ``q`` [rows, heads, 576] the absorbed and rotated query."""
        # the attention's arguments, before the insert
        fn, dev, (rows, heads, _) = "TreeStep", self.out.get_device(), self.out.shape
        _mat(fn, "block_table", block_table, dev, torch.int32, self.ctx_lens.shape[0], None)
        ptr, ld, ld_head = _heads(fn, "q", q, dev, rows, heads, W.ATTN_DIM)
        if ptr % 16 or ld % 8 or ld_head % 8 or min(ld, ld_head) < W.ATTN_DIM:
            raise ValueError(f"{fn}: q's rows and heads must begin at 16-byte boundaries and not overlap, "
                             f"its strides are {q.stride()}")
        idx_kv_norm_rope_quant_and_cache(kv[:, :512], kv[:, 512:], kv_weight, self.eps, self.positions, cos_sin, self.slots,
                                         kv_cache, self.block_size, interleaved=self.interleaved, stream=stream)
        idx_tree_attention(q, kv_cache, self.block_size, block_table, self.cu_rows, self.ctx_lens, self.mask, self.out,
                           self.softmax_scale, lse=self.lse, ws=self.ws, stream=stream)
        return self.out


def exchange_candidates(vals: torch.Tensor, idx: torch.Tensor, group=None):
    """The one exchange of context-parallel decode: every rank's local top-k.

    [DSA] 几个容易踩的点: ranks that each hold a shard of a long context send
    each other only their local (score, index) lists, never the score matrix.
    ``vals`` float32 / ``idx`` int32 ``[rows, k_local]`` on each rank become
    ``[rows, world * k_local]`` on every rank, rank after rank along the row, the
    candidate layout ``idx_dcp_topk_merge`` reads. Any backend whose tensors
    these are will do (gloo with host tensors, NCCL with device tensors).
    """
    import torch.distributed as dist

    world = dist.get_world_size(group)
    gv = [torch.empty_like(vals) for _ in range(world)]
    gi = [torch.empty_like(idx) for _ in range(world)]
    dist.all_gather(gv, vals.contiguous(), group=group)
    dist.all_gather(gi, idx.contiguous(), group=group)
    return torch.cat(gv, dim=1), torch.cat(gi, dim=1)


class DcpDecodeStep:
    """One rank of a context-parallel decode step.

    The rank's paged cache holds only its shard of every request's context
    (``ctx_lens`` are shard lengths). ``select_local`` scores that shard and keeps
    its top-k with scores; ``merge`` turns every rank's lists, gathered rank after
    rank, into global top-k positions; ``run`` chains the two around
    ``exchange_candidates``. ``shard_offset`` / ``pos_stride`` give each rank's
    global positions (see ``idx_dcp_topk_merge``): per-request first positions of
    contiguous shards ([rows, world], stride 1), or ``arange(world)`` with stride
    ``world`` when tokens are dealt round-robin.
    """

    def __init__(self, batch: int, max_shard_ctx: int, world: int, topk: int = W.TOPK,
                 block_size: int = W.BLOCK_SIZE, device="cuda"):
        self.topk, self.block_size, self.world = topk, block_size, world
        ld = (max_shard_ctx + 63) // 64 * 64
        self.logits = torch.empty((batch, ld), dtype=torch.float32, device=device)
        self.cand_vals = torch.empty((batch, topk), dtype=torch.float32, device=device)
        self.cand_idx = torch.empty((batch, topk), dtype=torch.int32, device=device)
        self.positions = torch.empty((batch, topk), dtype=torch.int32, device=device)
        self.scores = torch.empty((batch, topk), dtype=torch.float32, device=device)
        self.ws = _workspace("topk", batch, ld, topk, device)

    def select_local(self, q, w, cache, block_table, ctx_lens, stream=None):
        idx_paged_mqa_logits_decode(q, w, cache, self.block_size, block_table, ctx_lens, self.logits,
                                    ws=self.ws, stream=stream)
        idx_topk(self.logits, None, ctx_lens, self.topk, self.cand_idx, vals=self.cand_vals, ws=self.ws,
                 stream=stream)
        return self.cand_vals, self.cand_idx

    def merge(self, all_vals, all_idx, shard_offset, pos_stride: int = 1, stream=None):
        idx_dcp_topk_merge(all_vals, all_idx, shard_offset, self.topk, self.topk, self.positions,
                           vals=self.scores, pos_stride=pos_stride, stream=stream)
        return self.positions

    def run(self, q, w, cache, block_table, ctx_lens, shard_offset, pos_stride: int = 1, group=None):
        """All three stages on torch's current stream, which the exchange also orders on."""
        self.select_local(q, w, cache, block_table, ctx_lens)
        all_vals, all_idx = exchange_candidates(self.cand_vals, self.cand_idx, group)
        return self.merge(all_vals, all_idx, shard_offset, pos_stride)
