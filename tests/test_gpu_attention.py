"""Normalised inserts, read-back of the attention cache and sparse attention, against the fp64 oracle.

Quantised values are held to the codes that some value within binary32's error of the fp64 one rounds to;
the read-back is exact; attention is held element by element to the bounds that ``oracle.attention`` derives.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import attention as A
from oracle.codecs import bf16_decode, bf16_encode, e4m3_decode, e4m3_encode
from oracle.indexer import ue8m0_ceil

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def cos_sin(n, seed=0):
    ang = np.random.default_rng(seed).uniform(0, 2 * np.pi, (n, 32))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def half_step(v, scale):
    """Half the distance between the e4m3 values next to ``v`` times ``scale``: the largest rounding error."""
    _, e = np.frexp(np.abs(v))
    return np.ldexp(1.0, np.maximum(e - 1, -6) - 4) * scale


def typed(x, dtype):
    t = torch.from_numpy(x).to(DEV)
    return t.bfloat16() if dtype == "bf16" else t.float()


# ------------------------------------------------------------------ indexer k

@pytest.mark.parametrize("n,bs,dtype,inter,ue8m0,pad", [
    (1, 64, "bf16", False, False, 0), (7, 16, "bf16", True, False, 8), (33, 32, "fp32", False, False, 0),
    (65, 128, "fp32", True, True, 3), (200, 64, "bf16", False, True, 5)])
def test_k_insert(n, bs, dtype, inter, ue8m0, pad):
    rng = np.random.default_rng(n)
    x = (rng.normal(size=(n, 128 + pad)) * np.exp(rng.normal(size=(n, 1))) + rng.normal()).astype(np.float32)
    k = typed(x, dtype)[:, pad:]                                   # strided, and misaligned for odd pads
    xs = k.double().cpu().numpy()
    w, b = rng.normal(size=128).astype(np.float32), rng.normal(size=128).astype(np.float32)
    if n == 7:
        b = None
    cs = cos_sin(50)
    pos = rng.integers(0, 50, n).astype(np.int32)
    blocks = -(-n // bs) + 1
    stride = -(-bs * 132 // 512) * 512
    slots = rng.permutation(blocks * bs)[:n].astype(np.int64)
    if n > 30:
        slots[3], slots[5] = -1, blocks * bs                       # skipped
        pos[4], pos[6] = -1, 50                                    # written as zeros, flagged
    cache = torch.full((blocks, stride), 77, dtype=torch.uint8, device=DEV)
    idx.idx_k_norm_rope_quant_and_cache(k, dev(w), None if b is None else dev(b), 1e-6, dev(pos), dev(cs), dev(slots),
                                        cache, bs, ue8m0=ue8m0, interleaved=inter)
    if n > 30:
        with pytest.raises(idx.IdxError, match="inserts and read-back 0x00000001"):
            idx.idx_device_error()
    idx.idx_device_error()
    y, err = A.k_norm_rope(xs, w, b, float(np.float32(1e-6)), pos, cs, inter)
    got = cache.cpu().numpy()
    touched = np.zeros_like(got, dtype=bool)
    for i in range(n):
        s = int(slots[i])
        if s < 0 or s >= blocks * bs:
            continue
        blk, off = divmod(s, bs)
        at = bs * 128 + 4 * off
        touched[blk, off * 128:off * 128 + 128] = True
        touched[blk, at:at + 4] = True
        scale = got[blk, at:at + 4].copy().view(np.float32)[0]
        codes = got[blk, off * 128:off * 128 + 128]
        lo = (np.abs(y[i]) - err[i]).max() / 448 * (1 - 2 * U)
        hi = (np.abs(y[i]) + err[i]).max() / 448 * (1 + 2 * U)
        if ue8m0:
            assert ue8m0_ceil(max(lo, 0)) <= scale <= ue8m0_ceil(hi)
        else:
            assert lo <= scale <= hi
        if scale == 0:
            assert not codes.any() and not y[i].any()
            continue
        v = e4m3_decode(codes)
        # the largest code stands for everything up to the scale's own rounding
        assert (np.abs(v * scale - y[i]) <= half_step(v, scale) * (1 + 2.0 ** -20) + err[i] + 2 * U * np.abs(y[i])).all()
    assert (got[~touched] == 77).all()


# ------------------------------------------------------------------ attention latent

@pytest.mark.parametrize("n,bs,dtype,inter,norm,rope,pad", [
    (1, 64, "bf16", True, True, True, 0), (5, 16, "bf16", False, True, True, 3), (40, 32, "fp32", True, True, False, 0),
    (67, 128, "fp32", False, False, True, 1), (130, 64, "bf16", True, False, False, 8)])
def test_kv_insert(n, bs, dtype, inter, norm, rope, pad):
    rng = np.random.default_rng(n)
    x = (rng.normal(size=(n, 576 + pad)) * np.exp(2 * rng.normal(size=(n, 1)))).astype(np.float32)
    if n > 30:
        x[2] = 0.0                                                 # an all-zero token
        x[7, pad:pad + 128] *= 1e-30                               # a tile far below the others
        if not norm:
            x[8, pad + 130] = 1e8                                  # beyond the largest scale: saturates
    t = typed(x, dtype)
    c, pe = t[:, pad:pad + 512], t[:, pad + 512:]
    w = rng.normal(size=512).astype(np.float32) if norm else None
    cs = cos_sin(50)
    pos = rng.integers(0, 50, n).astype(np.int32)
    blocks = -(-n // bs) + 1
    stride = bs * 644 + 16
    slots = rng.permutation(blocks * bs)[:n].astype(np.int64)
    flagged = rope and n > 30
    if n > 30:
        slots[3], slots[5] = -1, blocks * bs
        if rope:
            pos[4], pos[6] = -1, 50
    cache = torch.full((blocks, stride), 77, dtype=torch.uint8, device=DEV)
    idx.idx_kv_norm_rope_quant_and_cache(c, pe, None if w is None else dev(w), 1e-5, dev(pos) if rope else None,
                                         dev(cs) if rope else None, dev(slots), cache, bs, interleaved=inter)
    if flagged:
        with pytest.raises(idx.IdxError, match="inserts and read-back 0x00000001"):
            idx.idx_device_error()
    idx.idx_device_error()
    y, err = A.kv_norm(c.double().cpu().numpy(), w, float(np.float32(1e-5)))
    p64 = pe.double().cpu().numpy()
    z, perr = p64, np.zeros_like(p64)
    if rope:
        z, ok = A.rotate(p64, pos, cs, inter)
        a, b = A.rope_pairs(inter)
        perr = np.zeros_like(p64)
        perr[:, a] = perr[:, b] = 3 * U * (np.abs(p64[:, a]) + np.abs(p64[:, b]))
        y[~ok], err[~ok] = 0, 0
    got = cache.cpu().numpy()
    want = np.full_like(got, 77)
    for i in range(n):
        s = int(slots[i])
        if s < 0 or s >= blocks * bs:
            continue
        codes, pbits, sc = A.kv_record(got, bs, s)
        tile, te = y[i].reshape(4, 128), err[i].reshape(4, 128)
        lo = A.kv_scale_exponent((np.abs(tile) - te).max(axis=1) * (1 - 2 * U)) + 127
        hi = A.kv_scale_exponent((np.abs(tile) + te).max(axis=1) * (1 + 2 * U)) + 127
        assert (lo <= sc).all() and (sc <= hi).all()
        scale = np.repeat(np.exp2(sc.astype(np.float64) - 127), 128)
        v = e4m3_decode(codes)
        held = np.clip(y[i], -448 * scale, 448 * scale)
        assert (np.abs(v * scale - held) <= half_step(v, scale) + err[i]).all()
        g = bf16_decode(pbits).astype(np.float64)
        assert (np.abs(g - z[i]) <= 2.0 ** -8 * np.abs(z[i]) + 2 * perr[i] + 2.0 ** -134).all()
        A.kv_put(want, bs, s, codes, pbits, sc)
    assert (got == want).all()                                     # nothing else was written


# ------------------------------------------------------------------ read-back

def random_cache(rng, blocks, bs, extra=0):
    """A cache of random e4m3 latents (no NaN codes), scales 2^-7 .. 2^3, normal position dims."""
    cache = np.zeros((blocks, bs * 644 + extra), dtype=np.uint8)
    n = blocks * bs
    codes = e4m3_encode(rng.normal(size=(n, 512)) * 3)
    pe = bf16_encode(rng.normal(size=(n, 64)).astype(np.float32))
    sc = rng.integers(124, 129, (n, 4)).astype(np.uint8)
    for s in range(n):
        A.kv_put(cache, bs, s, codes[s], pe[s], sc[s])
    return cache


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_reads_back_exactly(dtype):
    # every e4m3 code but the two NaNs under every scale code 0 .. 134, in both halves of every pair
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    row = np.concatenate([codes, codes[::-1], [0, 0, 0, 0]]).astype(np.uint8)      # 254 + 254 + 4 = 512
    n, bs = 135, 16
    blocks = -(-n // bs)
    cache = np.zeros((blocks, bs * 644), dtype=np.uint8)
    for s in range(n):
        A.kv_put(cache, bs, s, row, np.arange(64) * 257, np.full(4, s, np.uint8))
    out = torch.zeros((n, 576), dtype=dtype, device=DEV)
    idx.idx_gather_kv(dev(cache), bs, dev(np.arange(blocks, dtype=np.int32)[None]), dev(np.array([0, n], np.int32)), out)
    want = e4m3_decode(row)[None] * np.exp2(np.arange(n) - 127.0)[:, None]
    big = np.abs(want) >= 2.0 ** -126                                              # below: bf16's own subnormals
    got = out.double().cpu().numpy()
    assert (got[:, :512][big] == want[big]).all()
    assert (np.abs(got[:, :512] - want)[~big] <= 2.0 ** -134).all()
    assert (out[:, 512:].bfloat16().view(torch.int16).cpu().numpy().view(np.uint16) == np.arange(64) * 257).all()


@pytest.mark.parametrize("bs,lens,starts,dtype,pad", [
    (64, [1], None, torch.bfloat16, 0), (16, [5, 0, 17, 0, 0, 40], None, torch.float32, 4),
    (32, [33, 64, 1, 95], [0, 31, 32, 1], torch.bfloat16, 8), (128, [0, 300], [5, 127], torch.bfloat16, 0)])
def test_gather(bs, lens, starts, dtype, pad):
    rng = np.random.default_rng(bs)
    B = len(lens)
    pages = max(-(-(n + (starts[b] if starts else 0)) // bs) for b, n in enumerate(lens))
    cache = random_cache(rng, B * pages, bs, 32)
    bt = rng.permutation(B * pages).reshape(B, pages).astype(np.int32)
    wide = np.full((B, pages + 3), 1 << 30, dtype=np.int32)                        # row stride beyond the pages
    wide[:, :pages] = bt
    cu = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int32)               # two rows before the first request
    n = int(cu[-1]) + 5                                                            # and five behind the last
    buf = torch.full((n, 576 + pad), 7.0, dtype=dtype, device=DEV)
    idx.idx_gather_kv(dev(cache), bs, dev(wide)[:, :pages], dev(cu), buf[:, :576],
                      starts=None if starts is None else dev(np.array(starts, np.int32)))
    idx.idx_device_error()
    got = buf.double().cpu().numpy()
    want = A.gather_kv(cache, bs, bt, cu, starts)
    assert (got[2:cu[-1], :576] == want[2:]).all()
    assert (got[:2] == 7).all() and (got[cu[-1]:] == 7).all() and (got[:, 576:] == 7).all()
    cut = torch.full((n - 8, 576), 7.0, dtype=dtype, device=DEV)                   # an output shorter than the ranges
    idx.idx_gather_kv(dev(cache), bs, dev(wide)[:, :pages], dev(cu), cut,
                      starts=None if starts is None else dev(np.array(starts, np.int32)))
    m = max(n - 8, 0)
    assert torch.equal(cut[2:], buf[2:m, :576])


def test_gather_bad_pages():
    rng = np.random.default_rng(3)
    cache = random_cache(rng, 4, 16)
    bt = np.array([[0, 4, 1], [-1, 2, 3]], np.int32)
    cu = np.array([0, 48, 80], np.int32)
    out = torch.full((90, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    idx.idx_gather_kv(dev(cache), 16, dev(bt), dev(cu), out, starts=dev(np.array([0, 20], np.int32)))
    with pytest.raises(idx.IdxError, match="inserts and read-back 0x00000002"):
        idx.idx_device_error()
    got = out.double().cpu().numpy()
    tok = lambda s: A.kv_token(cache, 16, s)  # noqa: E731
    assert (got[15] == tok(15)).all() and not got[16:32].any() and (got[32] == tok(16)).all()
    # request 1 starts at token 20: pages 1, 2 and then past its three pages
    assert (got[48] == tok(32 + 4)).all() and (got[48 + 27] == tok(48 + 15)).all()
    assert not got[48 + 28:80].any() and (got[80:] == 7).all()
    out.fill_(7.0)
    idx.idx_gather_kv(dev(cache), 16, dev(bt), dev(cu), out, starts=dev(np.array([-3, 0], np.int32)))
    with pytest.raises(idx.IdxError):
        idx.idx_device_error()
    got = out.double().cpu().numpy()
    assert not got[:3].any() and (got[3] == tok(0)).all() and not got[48:64].any()


# ------------------------------------------------------------------ attention

def attention_case(seed, T, H, K, bs, amp=1.0, holes=0.1, blocks=None):
    rng = np.random.default_rng(seed)
    blocks = blocks or max(2, -(-2 * max(K, 1) // bs))
    cache = random_cache(rng, blocks, bs, 16)
    slots = rng.integers(0, blocks * bs, (T, K)).astype(np.int32)
    slots[rng.random((T, K)) < holes] = -1
    q = bf16_encode((rng.normal(size=(T, H, 576)) * amp).astype(np.float32))
    return cache, slots, q


def check_attention(cache, slots, q, bs, scale, out, lse, n_sel=None, span=None):
    """Element by element against the oracle's value and error bound."""
    o, l, oe, le = A.sparse_attention(bf16_decode(q), cache, bs, slots, scale, n_sel, span)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - o) > oe + 1e-30
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], float(np.abs(got - o).max()), float(oe.min()))
    if lse is not None:
        g = lse.double().cpu().numpy()
        empty = np.isneginf(l)
        assert (np.isneginf(g) == empty).all()
        assert (np.abs(g[~empty] - l[~empty]) <= le[~empty]).all()


def workspace(T, H, K):
    n = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    # sentinels behind it, and garbage inside: its contents mean nothing
    return torch.full((n + 64,), 0x7B, dtype=torch.uint8, device=DEV)[:n] if n else None


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("T,H,K,bs,amp", [
    (1, 1, 1, 64, 1.0), (1, 128, 64, 64, 1.0), (2, 64, 63, 16, 2.0), (3, 20, 65, 32, 1.0), (2, 7, 128, 128, 4.0),
    (1, 64, 129, 64, 0.0), (5, 65, 191, 16, 1.0), (1, 130, 300, 64, 2.0), (2, 16, 777, 64, 8.0), (1, 128, 2048, 64, 3.0),
    (3, 33, 2048, 128, 1.0)])
def test_attention(T, H, K, bs, amp, ws):
    cache, slots, q = attention_case(T * 1000 + H + K, T, H, K, bs, amp)
    if T > 2:
        slots[1] = -1                                              # a row with no token
    out = torch.full((T, H, 512), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 9.0, device=DEV)
    w = workspace(T, H, K) if ws else None
    if ws and K >= 512 and T == 1:
        assert w is not None                                       # a single long row is split
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), bs, dev(slots), out, 576 ** -0.5,
                             lse=lse, ws=w)
    idx.idx_device_error()
    check_attention(cache, slots, q, bs, 576 ** -0.5, out, lse)


def test_attention_without_lists():
    cache, _, q = attention_case(1, 3, 70, 8, 64)
    out = torch.full((3, 70, 512), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((3, 70), 9.0, device=DEV)
    qd = dev(q.view(np.int16)).view(torch.bfloat16)
    idx.idx_sparse_attention(qd, dev(cache), 64, torch.zeros((3, 0), dtype=torch.int32, device=DEV), out, 0.04, lse=lse)
    idx.idx_device_error()
    assert not out.any() and torch.isneginf(lse).all()
    out.fill_(9.0)
    idx.idx_sparse_attention(qd, dev(cache), 64, torch.full((3, 200), -1, dtype=torch.int32, device=DEV), out, 0.04)
    assert not out.any()


@pytest.mark.parametrize("ws", [False, True])
def test_attention_counts_spans_strides_and_bad_slots(ws):
    T, H, K, bs, span = 4, 24, 300, 16, 40
    cache, slots, q = attention_case(11, T, H, K, bs, 2.0, blocks=50)
    slots = np.where(slots >= 0, slots // bs * span + slots % bs, -1).astype(np.int32)
    slots[0, 7], slots[0, 200] = 16, 50 * span                     # an offset past the block; a block past the cache
    slots[2, 3] = np.iinfo(np.int32).max
    slots[1, :40] = slots[1, 0] if slots[1, 0] >= 0 else 3         # one token forty times
    n_sel = np.array([300, 250, 0, 1], np.int32)
    # rows and heads strided, slots and lse columns of wider buffers
    qb = torch.zeros((T, 2, H, 592), dtype=torch.bfloat16, device=DEV)
    qb[:, 1, :, :576] = dev(q.view(np.int16)).view(torch.bfloat16)
    ob = torch.full((H, T, 520), 9.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((T, H + 3), 9.0, device=DEV)
    sb = torch.full((T, K + 5), 0, dtype=torch.int32, device=DEV)
    sb[:, :K] = dev(slots)
    out = ob[:, :, :512].transpose(0, 1)
    idx.idx_sparse_attention(qb[:, 1, :, :576], dev(cache), bs, sb[:, :K], out, 0.05, lse=lb[:, :H], n_sel=dev(n_sel),
                             block_span=span, ws=workspace(T, H, K) if ws else None)
    with pytest.raises(idx.IdxError, match="attention 0x00000001"):
        idx.idx_device_error()
    idx.idx_device_error()
    check_attention(cache, slots, q, bs, 0.05, out, lb[:, :H], n_sel, span)
    assert (ob[:, :, 512:] == 9).all() and (lb[:, H:] == 9).all()


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_attention_scales(scale):
    cache, slots, q = attention_case(13, 2, 40, 150, 32, 1.0)
    out = torch.empty((2, 40, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2, 40), device=DEV)
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), 32, dev(slots), out, scale, lse=lse)
    check_attention(cache, slots, q, 32, scale, out, lse)


@pytest.mark.parametrize("ws", [False, True])
def test_attention_rising_logits(ws):
    # logits that climb by tens from tile to tile: every tile moves the running maximum, late tokens
    # outweigh all earlier ones, and the other order must give the same row
    rng = np.random.default_rng(17)
    K, bs = 640, 64
    cache = np.zeros((10, bs * 644), dtype=np.uint8)
    codes = e4m3_encode(rng.normal(size=(K, 512)))
    pe = np.zeros((K, 64), np.float32)
    pe[:, 0] = np.arange(K) // 40                                  # the last dims rank the tokens
    for s in range(K):
        A.kv_put(cache, bs, s, codes[s], bf16_encode(pe[s]), [127] * 4)
    q = rng.normal(size=(2, 66, 576)).astype(np.float32) * 0.05
    q[:, :, 512] = 30.0
    q = bf16_encode(q)
    up = np.arange(K, dtype=np.int32)
    slots = np.stack([up, up[::-1]])
    out = torch.empty((2, 66, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2, 66), device=DEV)
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), bs, dev(slots), out, 1.0, lse=lse,
                             ws=workspace(2, 66, K) if ws else None)
    check_attention(cache, slots, q, bs, 1.0, out, lse)


def test_attention_many_rows_equal_rows_alone():
    # more rows than SMs, lists of every length: each row's result does not depend on the others
    cache, slots, q = attention_case(19, 400, 16, 100, 64, 2.0, blocks=8)
    n_sel = (np.arange(400) % 101).astype(np.int32)
    qd, cd, sd, nd = dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), dev(slots), dev(n_sel)
    out = torch.empty((400, 16, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((400, 16), device=DEV)
    idx.idx_sparse_attention(qd, cd, 64, sd, out, 0.05, lse=lse, n_sel=nd)
    for t in (0, 1, 64, 65, 100, 303, 399):
        o1, l1 = torch.empty_like(out[:1]), torch.empty_like(lse[:1])
        idx.idx_sparse_attention(qd[t:t + 1], cd, 64, sd[t:t + 1], o1, 0.05, lse=l1, n_sel=nd[t:t + 1])
        assert torch.equal(o1[0], out[t]) and torch.equal(l1[0], lse[t])
    pick = [0, 1, 64, 65, 100, 303, 399]
    check_attention(cache, slots[pick], q[pick], 64, 0.05, out[pick], lse[pick], n_sel[pick])


def test_attention_repeats_bit_for_bit_on_streams_and_in_graphs():
    T, H, K = 2, 128, 1024
    cache, slots, q = attention_case(23, T, H, K, 64, 2.0)
    qd, cd, sd = dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), dev(slots)
    out, lse = torch.empty((T, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), device=DEV)
    idx.idx_sparse_attention(qd, cd, 64, sd, out, 0.05, lse=lse, ws=workspace(T, H, K))
    torch.cuda.synchronize()
    # two calls at once on two streams, a workspace each
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(out) for _ in side]
    wss = [workspace(T, H, K) for _ in side]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(side, outs, wss):
            idx.idx_sparse_attention(qd, cd, 64, sd, o, 0.05, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    # captured, then replayed on new queries
    g = torch.cuda.CUDAGraph()
    o2, w2, qg = torch.empty_like(out), workspace(T, H, K), qd.clone()
    with torch.cuda.graph(g):
        idx.idx_sparse_attention(qg, cd, 64, sd, o2, 0.05, ws=w2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, out)
    q2 = bf16_encode(np.random.default_rng(29).normal(size=(T, H, 576)).astype(np.float32))
    qg.copy_(dev(q2.view(np.int16)).view(torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    check_attention(cache, slots, q2, 64, 0.05, o2, None)
    idx.idx_device_error()


def test_small_workspace_and_wrong_tensors_are_refused():
    T, H, K = 1, 64, 2048
    cache, slots, q = attention_case(31, T, H, K, 64)
    qd, cd, sd = dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), dev(slots)
    out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=DEV)
    n = idx.idx_sparse_attention_workspace_bytes(T, H, K)
    assert n > 0
    with pytest.raises(idx.IdxError, match="workspace"):
        idx.idx_sparse_attention(qd, cd, 64, sd, out, 0.05, ws=torch.empty(n - 16, dtype=torch.uint8, device=DEV))
    for bad in (dict(out=out.float()), dict(out=out[:, :32]), dict(slots=sd.long()), dict(q=qd.float()),
                dict(lse=torch.empty((T, H + 1), device=DEV)), dict(n_sel=torch.zeros(T + 1, dtype=torch.int32, device=DEV)),
                dict(cache=cd.cpu())):
        a = dict(q=qd, cache=cd, block_size=64, slots=sd, out=out, softmax_scale=0.05)
        a.update(bad)
        with pytest.raises(ValueError):
            idx.idx_sparse_attention(**a)
    idx.idx_device_error()


def test_offsets_past_32_bits():
    # blocks that start past 2^32 bytes and past 2^31 token bytes, written, read back and attended to
    bs, stride = 128, 128 * 644
    blocks = (1 << 32) // stride + 300
    cache = torch.zeros((blocks, stride), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(41)
    high = np.arange(blocks - 3, blocks)
    slots = (high[:, None] * bs + np.arange(bs)).reshape(-1).astype(np.int64)
    n = len(slots)
    x = dev(rng.normal(size=(n, 576)).astype(np.float32)).bfloat16()
    idx.idx_kv_norm_rope_quant_and_cache(x[:, :512], x[:, 512:], None, 1e-6, None, None, dev(slots), cache, bs)
    out = torch.empty((n, 576), dtype=torch.float32, device=DEV)
    idx.idx_gather_kv(cache, bs, dev(high.astype(np.int32)[None]), dev(np.array([0, n], np.int32)), out)
    small = cache[blocks - 3:].cpu().numpy()
    assert (out.double().cpu().numpy() == A.gather_kv(small, bs, [[0, 1, 2]], [0, n])).all() and bool(out.any())
    q = bf16_encode(rng.normal(size=(1, 16, 576)).astype(np.float32))
    lst = rng.permutation(n)[:200]
    o, l = torch.empty((1, 16, 512), dtype=torch.bfloat16, device=DEV), torch.empty((1, 16), device=DEV)
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), cache, bs, dev(slots[lst].astype(np.int32)[None]),
                             o, 576 ** -0.5, lse=l)
    idx.idx_device_error()
    check_attention(small, lst.astype(np.int32)[None], q, bs, 576 ** -0.5, o, l)


@pytest.mark.parametrize("T,H,K,bs", [(1, 17, 4096, 64), (9, 64, 5000, 32), (40, 48, 640, 16)])
def test_attention_long_and_split_lists(T, H, K, bs):
    # every number of parts' join: a part without a token, rows of fewer entries than parts, ragged ends
    cache, slots, q = attention_case(T + K, T, H, K, bs, 2.0, holes=0.3, blocks=40)
    n_sel = np.random.default_rng(T).integers(0, K + 1, T).astype(np.int32)
    slots[0, : K // 2] = -1
    n_sel[0] = K
    if T > 2:
        n_sel[1], n_sel[2] = 0, 1
    out = torch.full((T, H, 512), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 9.0, device=DEV)
    w = workspace(T, H, K)
    assert w is not None or T == 40
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), bs, dev(slots), out, 576 ** -0.5,
                             lse=lse, n_sel=dev(n_sel), ws=w)
    idx.idx_device_error()
    pick = [t for t in range(T) if t < 4 or t % 9 == 0]
    check_attention(cache, slots[pick], q[pick], bs, 576 ** -0.5, out[pick], lse[pick], n_sel[pick])
    # the same row whole and in parts: the same tokens, other roundings only
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    idx.idx_sparse_attention(dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), bs, dev(slots), o2, 576 ** -0.5,
                             lse=l2, n_sel=dev(n_sel))
    check_attention(cache, slots[pick], q[pick], bs, 576 ** -0.5, o2[pick], l2[pick], n_sel[pick])


def test_calls_on_a_side_stream_follow_their_inputs():
    # inputs made on a side stream, the call given that stream: no other synchronisation
    cache, slots, q = attention_case(43, 3, 64, 500, 64, 2.0)
    ref = torch.empty((3, 64, 512), dtype=torch.bfloat16, device=DEV)
    qd, cd, sd = dev(q.view(np.int16)).view(torch.bfloat16), dev(cache), dev(slots)
    idx.idx_sparse_attention(qd, cd, 64, sd, ref, 0.05)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(5_000_000)
        c2 = torch.zeros_like(cd)
        c2.copy_(cd)
        out = torch.empty_like(ref)
        idx.idx_sparse_attention(qd, c2, 64, sd, out, 0.05)                 # torch's current stream
        packed = torch.empty((100, 576), dtype=torch.bfloat16, device=DEV)
        idx.idx_gather_kv(c2, 64, torch.zeros((1, 2), dtype=torch.int32, device=DEV),
                          torch.tensor([0, 64], dtype=torch.int32, device=DEV), packed)
    st.synchronize()
    assert torch.equal(out, ref)
    assert (packed[:64].double().cpu().numpy() == A.gather_kv(cache, 64, [[0]], [0, 64])).all()


# ------------------------------------------------------------------ together

def test_one_layer_step_together():
    """Both inserts, the query preparation, scoring, selection with slots and attention, as one layer's decode
    step calls them; the attention's list is the kernel's own selection, its cache the kernel's own bytes."""
    from sparse_attention_indexer_fp8_gb300.pipeline import AttentionDecodeStep

    rng = np.random.default_rng(37)
    B, L, H, K, bs = 5, 700, 24, 256, 64
    lens = np.array([1, 63, 257, 700, 512], np.int32)
    pages = -(-L // bs)
    bt = rng.permutation(B * pages).reshape(B, pages).astype(np.int32)
    cs = dev(cos_sin(L))
    step = AttentionDecodeStep(B, L, heads=H, topk=K, device=DEV, interleaved=True)
    kc, vc = step.make_caches(B * pages)
    w, bias, rw = (dev(rng.normal(size=n).astype(np.float32)) for n in (128, 128, 512))
    # contexts inserted by the same calls, the last token of each by the step itself
    hist_k = [rng.normal(size=(int(n), 128)).astype(np.float32) for n in lens]
    hist_v = [rng.normal(size=(int(n), 576)).astype(np.float32) for n in lens]
    slot = lambda b, p: (bt[b, p // bs].astype(np.int64) * bs + p % bs)  # noqa: E731
    for b in range(B):
        p = np.arange(lens[b] - 1)
        if len(p):
            step.insert(dev(hist_k[b][:-1]).bfloat16(), dev(hist_v[b][:-1]).bfloat16(), w, bias, rw,
                        dev(p.astype(np.int32)), cs, dev(slot(b, p)), kc, vc)
    last = lens - 1
    new_k = dev(np.stack([h[-1] for h in hist_k])).bfloat16()
    new_v = dev(np.stack([h[-1] for h in hist_v])).bfloat16()
    qi = dev(rng.normal(size=(B, 64, 128)).astype(np.float32)).bfloat16()
    wi = dev(rng.normal(size=(B, 64)).astype(np.float32) / 64)
    q = bf16_encode(rng.normal(size=(B, H, 576)).astype(np.float32))
    slots_new = dev(np.array([slot(b, last[b]) for b in range(B)]))
    args = dict(new_k=new_k, new_kv=new_v, k_weight=w, k_bias=bias, kv_weight=rw, positions=dev(last), cos_sin=cs,
                new_slots=slots_new, q_index=qi, w_index=wi, q=dev(q.view(np.int16)).view(torch.bfloat16),
                k_cache=kc, kv_cache=vc, block_table=dev(bt), ctx_lens=dev(lens))
    out = step.run(**args).clone()
    idx.idx_device_error()
    sl = step.indexer.slots.cpu().numpy()
    for b in range(B):
        own = {int(slot(b, p)) for p in range(lens[b])}
        kept = sl[b][sl[b] >= 0]
        assert len(set(kept.tolist())) == len(kept) == min(K, lens[b]) and set(kept.tolist()) <= own
    check_attention(vc.cpu().numpy(), sl, q, bs, step.softmax_scale, out, step.lse)
    # read-back of the contexts: the bytes the inserts wrote
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    packed = torch.empty((int(cu[-1]), 576), dtype=torch.bfloat16, device=DEV)
    idx.idx_gather_kv(vc, bs, dev(bt), dev(cu), packed)
    assert (packed.double().cpu().numpy() == A.gather_kv(vc.cpu().numpy(), bs, bt, cu)).all()
    # the whole step captured and replayed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run(**args)
    step.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    sl2 = step.indexer.slots.cpu().numpy()
    assert all(set(a.tolist()) == set(b.tolist()) for a, b in zip(sl, sl2))
    check_attention(vc.cpu().numpy(), sl2, q, bs, step.softmax_scale, step.out, step.lse)
    idx.idx_device_error()
