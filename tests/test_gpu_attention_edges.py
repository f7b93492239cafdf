"""Edges of the inserts, the read-back and the sparse attention: values that are not finite, lists whose every entry
shows in the result, and every way in which a list is split and joined.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import attention as A
from oracle.codecs import bf16_decode, bf16_encode, e4m3_decode, e4m3_encode
from tests.checks import assert_attention_counts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def as_bf16(bits):
    return dev(np.asarray(bits).view(np.int16)).view(torch.bfloat16)


# ------------------------------------------------------------------ latents that are not finite

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_latent_that_is_not_finite_reads_back_as_nan(bad, dtype):
    # one value each in tokens 1, 2 and 5, in different tiles of 128 dims; no norm, so the other tiles stay what they are
    rng = np.random.default_rng(1)
    n, bs = 7, 16
    x = rng.normal(size=(n, 576)).astype(np.float32)
    clean = x.copy()
    at = {1: 0, 2: 255, 5: 511}
    for t, d in at.items():
        x[t, d] = bad

    def run(a):
        cache = torch.full((2, bs * 644), 77, dtype=torch.uint8, device=DEV)
        y = dev(a).to(dtype)
        idx.idx_kv_norm_rope_quant_and_cache(y[:, :512], y[:, 512:], None, 1e-6, None, None,
                                             dev(np.arange(n, dtype=np.int64) + 3), cache, bs)
        return cache

    got, want = run(x), run(clean)
    reads = []
    for out_dtype in (torch.float32, torch.bfloat16):
        out = torch.zeros((n, 576), dtype=out_dtype, device=DEV)
        idx.idx_gather_kv(got, bs, dev(np.array([[0]], np.int32)), dev(np.array([0, n], np.int32)), out,
                          starts=dev(np.array([3], np.int32)))
        reads.append(out.double().cpu().numpy())
    idx.idx_device_error()
    clean_bytes = want.cpu().numpy()
    for t in range(n):
        tok = A.kv_token(clean_bytes, bs, t + 3)
        tile = slice(at[t] // 128 * 128, at[t] // 128 * 128 + 128) if t in at else slice(0, 0)
        keep = np.ones(576, bool)
        keep[tile] = False
        for r in reads:
            assert np.isnan(r[t][tile]).all() and (r[t][keep] == tok[keep]).all()
        mine = A.kv_token(got.cpu().numpy(), bs, t + 3)
        assert np.isnan(mine[tile]).all() and (mine[keep] == tok[keep]).all()


def test_a_norm_that_meets_a_nan_spoils_its_token_only():
    rng = np.random.default_rng(2)
    n, bs = 9, 16
    x = rng.normal(size=(n, 576)).astype(np.float32)
    x[4, 100] = np.nan
    w = dev(rng.normal(size=512).astype(np.float32))
    y = dev(x).bfloat16()
    cache = torch.zeros((1, bs * 644), dtype=torch.uint8, device=DEV)
    idx.idx_kv_norm_rope_quant_and_cache(y[:, :512], y[:, 512:], w, 1e-6, None, None, dev(np.arange(n, dtype=np.int64)),
                                         cache, bs)
    out = torch.zeros((n, 576), dtype=torch.float32, device=DEV)
    idx.idx_gather_kv(cache, bs, dev(np.array([[0]], np.int32)), dev(np.array([0, n], np.int32)), out)
    nan = torch.isnan(out).cpu().numpy()
    assert nan[4, :512].all() and not nan[4, 512:].any() and not np.delete(nan, 4, axis=0).any()


@pytest.mark.parametrize("K", [130, 640])
def test_a_token_that_is_nan_spoils_the_rows_that_list_it(K):
    rng = np.random.default_rng(3)
    T, H, bs, n = 3, 20, 64, 256
    x = rng.normal(size=(n, 576)).astype(np.float32)
    clean = dev(x).bfloat16()
    x[77, 300] = np.nan
    bad = dev(x).bfloat16()
    slots = rng.integers(0, n, (T, K)).astype(np.int32)
    slots[slots == 77] = 78
    slots[1, K - 2] = 77
    q = as_bf16(bf16_encode(rng.normal(size=(T, H, 576)).astype(np.float32)))
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    assert (nbytes > 0) == (K == 640)
    res = []
    for y in (clean, bad):
        cache = torch.zeros((n // bs, bs * 644), dtype=torch.uint8, device=DEV)
        idx.idx_kv_norm_rope_quant_and_cache(y[:, :512], y[:, 512:], None, 1e-6, None, None,
                                             dev(np.arange(n, dtype=np.int64)), cache, bs)
        out, lse = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((T, H), device=DEV)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
        idx.idx_sparse_attention(q, cache, bs, dev(slots), out, 0.04, lse=lse, ws=ws)
        res.append((out, lse))
    idx.idx_device_error()
    (o, l), (ob, lb) = res
    assert torch.isnan(ob[1]).all() and torch.isnan(lb[1]).all()
    for t in (0, 2):
        assert torch.equal(o[t], ob[t]) and torch.equal(l[t], lb[t]) and torch.isfinite(o[t]).all()


# ------------------------------------------------------------------ q and cache bytes that nothing may pick up

def normal_cache(rng, blocks, bs, codes=(120, 131)):
    """Tokens of random latents under scales 2^(codes - 127), normal position dims."""
    cache = np.zeros((blocks, bs * 644), dtype=np.uint8)
    n = blocks * bs
    lat, pe = e4m3_encode(rng.normal(size=(n, 512)) * 3), bf16_encode(rng.normal(size=(n, 64)).astype(np.float32))
    sc = rng.integers(codes[0], codes[1], (n, 4)).astype(np.uint8)
    for s in range(n):
        A.kv_put(cache, bs, s, lat[s], pe[s], sc[s])
    return cache


@pytest.mark.parametrize("K", [100, 600])
def test_tokens_that_are_not_listed_may_hold_anything(K):
    # every record but the listed ones all ones (NaN position dims, NaN scales), holes and an offset past the block
    # in the lists: the result is that of a cache whose other records are zero, to the bit
    rng = np.random.default_rng(5)
    T, H, bs, blocks = 2, 70, 32, 40
    base = normal_cache(rng, blocks, bs)
    slots = rng.choice(blocks * bs, (T, K)).astype(np.int32)
    slots[:, ::7] = -1
    listed = np.unique(slots[slots >= 0])
    caches = []
    for fill in (0, 255):
        c = np.full_like(base, fill)
        for s in listed:
            A.kv_put(c, bs, s, *A.kv_record(base, bs, s))
        caches.append(dev(c))
    q = as_bf16(bf16_encode(rng.normal(size=(T, H, 576)).astype(np.float32)))
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    res = []
    for c in caches:
        out, lse = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((T, H), device=DEV)
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV) if nbytes else None
        idx.idx_sparse_attention(q, c, bs, dev(slots), out, 0.04, lse=lse, ws=ws)
        res.append((out, lse))
    idx.idx_device_error()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert torch.isfinite(res[0][0]).all() and torch.isfinite(res[0][1]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("K", [90, 700])
def test_a_head_whose_query_is_not_finite_spoils_itself_only(K, bad):
    rng = np.random.default_rng(7)
    T, H, bs = 2, 66, 64
    cache = dev(normal_cache(rng, 12, bs))
    slots = rng.integers(0, 12 * bs, (T, K)).astype(np.int32)
    slots[0, 5:30] = -1
    slots = dev(slots)
    x = rng.normal(size=(T, H, 576)).astype(np.float32)
    clean = dev(x).bfloat16()
    x[0, 3, 17] = x[1, 64, 575] = bad
    dirty = dev(x).bfloat16()
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    assert (nbytes > 0) == (K == 700)
    res = []
    for q in (clean, dirty):
        out, lse = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((T, H), device=DEV)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
        idx.idx_sparse_attention(q, cache, bs, slots, out, 0.04, lse=lse, ws=ws)
        res.append((out.cpu(), lse.cpu()))
    idx.idx_device_error()
    hit = torch.zeros((T, H), dtype=torch.bool)
    hit[0, 3] = hit[1, 64] = True
    (o, l), (ob, lb) = res
    assert torch.isnan(ob[hit]).all() and torch.isnan(lb[hit]).all()
    assert torch.equal(o[~hit], ob[~hit]) and torch.equal(l[~hit], lb[~hit])


def test_scales_from_the_lowest_to_the_highest():
    # latents between 2^-12 and 2^7 of one another in one token: the products and the value are held element by element
    rng = np.random.default_rng(9)
    T, H, K, bs = 2, 24, 200, 64
    cache = normal_cache(rng, 6, bs, codes=(115, 135))
    slots = rng.integers(0, 6 * bs, (T, K)).astype(np.int32)
    q = bf16_encode((rng.normal(size=(T, H, 576)) * 2.0 ** -9).astype(np.float32))
    out, lse = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((T, H), device=DEV)
    idx.idx_sparse_attention(as_bf16(q), dev(cache), bs, dev(slots), out, 0.04, lse=lse)
    idx.idx_device_error()
    o, l, oe, le = A.sparse_attention(bf16_decode(q), cache, bs, slots, 0.04)
    assert (np.abs(out.double().cpu().numpy() - o) <= oe).all() and (np.abs(lse.double().cpu().numpy() - l) <= le).all()


# ------------------------------------------------------------------ every entry counts once

def parts_of(T, H, K):
    """Parts that the workspace of these rows has room for (64 heads of 512 sums, a maximum and a sum each)."""
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    per_part = T * -(-H // 64) * 64 * (512 * 4 + 8)
    assert nbytes % per_part == 0
    return nbytes // per_part


def counting_cache(blocks, bs):
    """Token s is 1 at dim s % 512 and 0 elsewhere, under scales of 2^-4 .. 2^4; its position dims are noise."""
    cache = np.zeros((blocks, bs * 644), dtype=np.uint8)
    rng = np.random.default_rng(0)
    n = blocks * bs
    pe = bf16_encode(rng.normal(size=(n, 64)).astype(np.float32))
    for s in range(n):
        shift = s // 512 % 9 - 4
        codes = np.zeros(512, np.uint8)
        codes[s % 512] = (7 - shift) << 3                          # 2^-shift under the scale 2^shift
        A.kv_put(cache, bs, s, codes, pe[s], np.full(4, 127 + shift, np.uint8))
    return cache


def check_counts(slots, n_sel, out, lse, K, span, bs, blocks):
    got, g = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t in range(len(slots)):
        lst = slots[t][:max(0, min(K, int(n_sel[t])))]
        blk, off = lst // span, lst % span
        lst = (blk * bs + off)[(lst >= 0) & (blk < blocks) & (off < bs)]
        assert_attention_counts(got[t], g[t], lst % 512, (t, len(lst)))


@pytest.mark.parametrize("T,H,K,parts", [
    (1, 64, 8192, 128), (1, 17, 5000, 79), (2, 128, 2048, 32), (3, 33, 1500, 24), (4, 24, 640, 10), (4, 24, 512, 8), (16, 64, 2048, 8),
    (24, 40, 2500, 6), (28, 16, 1100, 5), (37, 8, 900, 4), (48, 64, 1800, 3), (70, 20, 2048, 2), (80, 64, 2048, 0), (5, 3, 300, 0)])
def test_every_entry_of_whole_and_split_lists_counts_once(T, H, K, parts):
    rng = np.random.default_rng(T + K)
    bs, span, blocks = 32, 40, 64
    assert parts_of(T, H, K) == parts
    tiles = -(-K // 64)
    per = -(-tiles // max(parts, 1)) * 64                          # entries of a part
    cache = dev(counting_cache(blocks, bs))
    slots = rng.integers(0, blocks * bs, (T, K)).astype(np.int32)
    slots = slots // bs * span + slots % bs
    slots[rng.random((T, K)) < 0.1] = -1
    slots[rng.random((T, K)) < 0.02] = blocks * span + 3           # past the cache
    slots[rng.random((T, K)) < 0.02] = 3 * span + bs               # an offset past its block
    if T > 1:
        slots[1, K // 3:K // 3 + 50] = 7                           # one token fifty times
    if parts:
        slots[0, per // 2:per // 2 + per] = -1                     # holes across a border; a part half empty on each side
    # the list ends at, before and behind the borders of tiles and parts, in turn
    ends = [K, K - 1, 1, 63, 64, 65, 127, 128, 129, per - 1, per, per + 1, 2 * per - 1, 2 * per, 2 * per + 1, 0, -3, K + 9,
            K // 2, K // 64 * 64, K // 64 * 64 - 1, 2]
    qd = as_bf16(bf16_encode(rng.normal(size=(T, H, 576)).astype(np.float32)))
    sb = torch.zeros((T, K + 5), dtype=torch.int32, device=DEV)
    sb[:, :K] = dev(slots)
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    buf = torch.full((nbytes + 256,), 0x7B, dtype=torch.uint8, device=DEV)
    for first in range(0, len(ends), T):
        n_sel = np.array([ends[(first + t) % len(ends)] for t in range(T)], np.int32)
        for split in ((False, True) if parts else (False,)):
            ob = torch.full((H, T, 520), 9.0, dtype=torch.bfloat16, device=DEV)
            lb = torch.full((T, H + 3), 9.0, device=DEV)
            idx.idx_sparse_attention(qd, cache, bs, sb[:, :K], ob[:, :, :512].transpose(0, 1), 0.0, lse=lb[:, :H],
                                     n_sel=dev(n_sel), block_span=span, ws=buf[:nbytes] if split else None)
            check_counts(slots, n_sel, ob[:, :, :512].transpose(0, 1), lb[:, :H], K, span, bs, blocks)
            assert (ob[:, :, 512:] == 9).all() and (lb[:, H:] == 9).all()
            assert (buf[nbytes:] == 0x7B).all()                    # nothing behind the workspace is written
    with pytest.raises(idx.IdxError, match="attention 0x00000001"):
        idx.idx_device_error()
    idx.idx_device_error()


@pytest.mark.parametrize("T,H,K,bs", [(4, 24, 700, 16), (16, 65, 2048, 64), (2, 20, 513, 32)])
def test_split_lists_with_spans_strides_and_bad_slots(T, H, K, bs):
    rng = np.random.default_rng(T * K)
    span, blocks = bs + 8, 50
    assert parts_of(T, H, K) > 1
    cache = normal_cache(rng, blocks, bs)
    slots = rng.integers(0, blocks * bs, (T, K)).astype(np.int32)
    slots = np.where(rng.random((T, K)) < 0.1, -1, slots // bs * span + slots % bs).astype(np.int32)
    slots[0, 7], slots[0, K - 3], slots[1, 3] = bs, blocks * span, np.iinfo(np.int32).max
    n_sel = rng.integers(1, K + 1, T).astype(np.int32)
    n_sel[0], n_sel[-1] = K, 0
    q = bf16_encode((rng.normal(size=(T, H, 576)) * 0.05).astype(np.float32))
    qb = torch.zeros((T, 2, H, 592), dtype=torch.bfloat16, device=DEV)
    qb[:, 1, :, :576] = as_bf16(q)
    ob = torch.full((H, T, 520), 9.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((T, H + 3), 9.0, device=DEV)
    sb = torch.zeros((T, K + 5), dtype=torch.int32, device=DEV)
    sb[:, :K] = dev(slots)
    out = ob[:, :, :512].transpose(0, 1)
    ws = torch.full((idx.idx_sparse_attention_workspace_bytes(T, H, K),), 255, dtype=torch.uint8, device=DEV)
    idx.idx_sparse_attention(qb[:, 1, :, :576], dev(cache), bs, sb[:, :K], out, 0.05, lse=lb[:, :H], n_sel=dev(n_sel),
                             block_span=span, ws=ws)
    with pytest.raises(idx.IdxError, match="attention 0x00000001"):
        idx.idx_device_error()
    idx.idx_device_error()
    o, l, oe, le = A.sparse_attention(bf16_decode(q), cache, bs, slots, 0.05, n_sel, span)
    got, g = out.double().cpu().numpy(), lb[:, :H].double().cpu().numpy()
    assert (np.abs(got - o) <= oe + 1e-30).all()
    empty = np.isneginf(l)
    assert (np.isneginf(g) == empty).all() and (np.abs(g[~empty] - l[~empty]) <= le[~empty]).all()
    assert (ob[:, :, 512:] == 9).all() and (lb[:, H:] == 9).all()


def test_two_graphs_replayed_in_turn_may_share_a_workspace():
    rng = np.random.default_rng(15)
    T, H, K, bs = 2, 40, 900, 64
    cache = dev(normal_cache(rng, 20, bs))
    nbytes = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    sets = []
    for _ in range(2):
        q = as_bf16(bf16_encode(rng.normal(size=(T, H, 576)).astype(np.float32)))
        slots = dev(rng.integers(0, 20 * bs, (T, K)).astype(np.int32))
        ref, out = (torch.empty((T, H, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        idx.idx_sparse_attention(q, cache, bs, slots, ref, 0.04, ws=torch.empty_like(ws))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            idx.idx_sparse_attention(q, cache, bs, slots, out, 0.04, ws=ws)
        sets.append((g, out, ref, q, slots))
    for _ in range(3):
        for g, out, _, _, _ in sets:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, ref) for _, out, ref, _, _ in sets)


# ------------------------------------------------------------------ paths of the inserts that no aligned buffer takes

def test_misaligned_weights_and_wide_angle_rows():
    # weights that start 4 bytes past a 16-byte border and angle rows of 70 floats write the same bytes
    rng = np.random.default_rng(11)
    n, bs = 40, 64
    x = dev(rng.normal(size=(n, 576)).astype(np.float32)).bfloat16()
    k = dev(rng.normal(size=(n, 128)).astype(np.float32)).bfloat16()
    pos, slots = dev(rng.integers(0, 30, n).astype(np.int32)), dev(rng.permutation(64)[:n].astype(np.int64))
    cs = dev(rng.normal(size=(30, 64)).astype(np.float32))
    wide = torch.full((30, 70), 7.0, device=DEV)
    wide[:, :64] = cs
    base = dev(rng.normal(size=520).astype(np.float32))
    w = base[:512]
    shifted = torch.empty(521, device=DEV)
    shifted[1:] = base
    assert shifted[1:].data_ptr() % 16 == 4
    res = []
    for buf, table in ((base, cs), (shifted[1:], wide), (shifted[1:], wide[:, :66])):
        kc = torch.full((1, bs * 132), 3, dtype=torch.uint8, device=DEV)
        vc = torch.full((1, bs * 644), 3, dtype=torch.uint8, device=DEV)
        idx.idx_kv_norm_rope_quant_and_cache(x[:, :512], x[:, 512:], buf[:512], 1e-6, pos, table, slots, vc, bs)
        idx.idx_k_norm_rope_quant_and_cache(k, buf[:128], buf[100:228], 1e-6, pos, table, slots, kc, bs, interleaved=True)
        res.append((vc, kc))
    idx.idx_device_error()
    assert w.data_ptr() % 16 == 0
    for vc, kc in res[1:]:
        assert torch.equal(vc, res[0][0]) and torch.equal(kc, res[0][1])
    # against the oracle: the latents within the record's own rounding and the norm's error
    y, err = A.kv_norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), float(np.float32(1e-6)))
    got = res[0][0].cpu().numpy()
    for i, s in enumerate(slots.cpu().numpy()):
        codes, _, sc = A.kv_record(got, bs, s)
        scale = np.repeat(np.exp2(sc.astype(np.float64) - 127), 128)
        v = e4m3_decode(codes) * scale
        assert (np.abs(v - y[i]) <= np.maximum(2.0 ** -4 * np.abs(y[i]), 2.0 ** -10 * scale) * (1 + 2.0 ** -20) + err[i]).all()


# ------------------------------------------------------------------ the layer's step

def test_a_step_with_split_lists_and_requests_that_sit_out():
    """Lists long enough to be split, more tokens than topk in some contexts, two requests of length 0."""
    from sparse_attention_indexer_fp8_gb300.pipeline import AttentionDecodeStep

    rng = np.random.default_rng(13)
    B, L, H, K, bs = 6, 1500, 24, 512, 64
    lens = np.array([0, 1400, 600, 0, 512, 65], np.int32)
    pages = -(-L // bs)
    bt = rng.permutation(B * pages).reshape(B, pages).astype(np.int32)
    ang = rng.uniform(0, 2 * np.pi, (L, 32))
    cs = dev(np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32))
    step = AttentionDecodeStep(B, L, heads=H, topk=K, device=DEV)
    assert step.ws is not None and parts_of(B, H, K) == 8
    kc, vc = step.make_caches(B * pages)
    w, bias, rw = (dev(rng.normal(size=n).astype(np.float32)) for n in (128, 128, 512))
    slot = lambda b, p: bt[b, p // bs].astype(np.int64) * bs + p % bs  # noqa: E731
    for b in range(B):
        p = np.arange(max(lens[b] - 1, 0))
        if len(p):
            step.insert(dev(rng.normal(size=(len(p), 128)).astype(np.float32)).bfloat16(),
                        dev(rng.normal(size=(len(p), 576)).astype(np.float32)).bfloat16(), w, bias, rw,
                        dev(p.astype(np.int32)), cs, dev(slot(b, p)), kc, vc)
    last = np.maximum(lens - 1, 0)
    new_slots = np.array([slot(b, last[b]) if lens[b] else -1 for b in range(B)], np.int64)
    q = bf16_encode(rng.normal(size=(B, H, 576)).astype(np.float32))
    before = kc.clone(), vc.clone()
    out = step.run(dev(rng.normal(size=(B, 128)).astype(np.float32)).bfloat16(),
                   dev(rng.normal(size=(B, 576)).astype(np.float32)).bfloat16(), w, bias, rw, dev(last.astype(np.int32)), cs,
                   dev(new_slots), dev(rng.normal(size=(B, 64, 128)).astype(np.float32)).bfloat16(),
                   dev(rng.normal(size=(B, 64)).astype(np.float32) / 64), as_bf16(q), kc, vc, dev(bt), dev(lens))
    idx.idx_device_error()
    sl = step.indexer.slots.cpu().numpy()
    for b in range(B):
        own = {int(slot(b, p)) for p in range(lens[b])}
        kept = sl[b][sl[b] >= 0]
        assert len(set(kept.tolist())) == len(kept) == min(K, lens[b]) and set(kept.tolist()) <= own
        assert (sl[b][:len(kept)] >= 0).all()                      # what counts stands first: lists may end at the length
        if lens[b] == 0:                                           # its blocks are as they were
            own_blocks = dev(bt[b].astype(np.int64))
            assert torch.equal(kc[own_blocks], before[0][own_blocks]) and torch.equal(vc[own_blocks], before[1][own_blocks])
    o, l, oe, le = A.sparse_attention(bf16_decode(q), vc.cpu().numpy(), bs, sl, step.softmax_scale)
    got, g = out.double().cpu().numpy(), step.lse.double().cpu().numpy()
    assert (np.abs(got - o) <= oe + 1e-30).all()
    empty = np.isneginf(l)
    assert empty[0].all() and empty[3].all() and (np.isneginf(g) == empty).all()
    assert (np.abs(g[~empty] - l[~empty]) <= le[~empty]).all()
