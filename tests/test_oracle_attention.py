"""Pins of the attention oracle (CPU): formats by hand, closed forms, library routines on special cases."""

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle.codecs import bf16_encode, e4m3_encode


def _cos_sin(n, seed=0):
    ang = np.random.default_rng(seed).uniform(0, 2 * np.pi, (n, 32))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def _random_cache(rng, blocks, bs, stride=None):
    cache = np.zeros((blocks, stride or bs * 644), dtype=np.uint8)
    vals = rng.normal(size=(blocks * bs, 512))
    for s in range(blocks * bs):
        A.kv_put(cache, bs, s, e4m3_encode(vals[s]), bf16_encode(rng.normal(size=64).astype(np.float32)),
                 rng.integers(120, 131, 4).astype(np.uint8))
    return cache


def test_layer_norm_matches_torch_and_zero_angle_is_identity():
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(5, 128)) * 3 + 1, rng.normal(size=128), rng.normal(size=128)
    cs = np.concatenate([np.ones((4, 32)), np.zeros((4, 32))], axis=1)
    y, err = A.k_norm_rope(x, w, b, 1e-5, np.zeros(5, int), cs, False)
    t = torch.nn.functional.layer_norm(torch.tensor(x), (128,), torch.tensor(w), torch.tensor(b), 1e-5)
    assert np.allclose(y, t.numpy(), rtol=1e-12, atol=1e-12)
    assert (err > 0).all() and err.max() < 1e-4


@pytest.mark.parametrize("interleaved", [False, True])
def test_binary32_evaluation_stays_within_the_stated_errors(interleaved):
    rng = np.random.default_rng(2)
    for off, spread in ((0, 1), (5, 0.1), (-3, 4)):
        x = (rng.normal(size=(64, 128)) * spread + off).astype(np.float32)
        w, b = rng.normal(size=128).astype(np.float32), rng.normal(size=128).astype(np.float32)
        cs = _cos_sin(16)
        pos = rng.integers(0, 16, 64)
        y, err = A.k_norm_rope(x, w, b, 1e-6, pos, cs, interleaved)
        d = x - x.mean(axis=1, keepdims=True, dtype=np.float32)
        f = d / np.sqrt((d * d).mean(axis=1, keepdims=True, dtype=np.float32) + np.float32(1e-6)) * w + b
        a, c = A.rope_pairs(interleaved)
        g = f.copy()
        g[:, a] = f[:, a] * cs[pos, :32] - f[:, c] * cs[pos, 32:]
        g[:, c] = f[:, c] * cs[pos, :32] + f[:, a] * cs[pos, 32:]
        assert (np.abs(g - y) <= err).all()


def test_rotation_is_a_complex_product_and_outside_the_table_is_zero():
    rng = np.random.default_rng(3)
    x, cs = rng.normal(size=(4, 64)), _cos_sin(3)
    pos = np.array([0, 2, 3, -1])
    y, ok = A.rotate(x, pos, cs, True)
    z = (x[:2, 0::2] + 1j * x[:2, 1::2]) * (cs[pos[:2], :32] + 1j * cs[pos[:2], 32:])
    assert np.allclose(y[:2, 0::2], z.real) and np.allclose(y[:2, 1::2], z.imag)
    assert ok.tolist() == [True, True, False, False] and (y[2:] == 0).all()
    # the half layout is the interleaved one with its dims permuted
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    h, _ = A.rotate(x[:, perm], pos, cs, False)
    assert np.allclose(h, y[:, perm])


def test_scale_exponents_by_hand():
    #        448 -> 1; just above -> 2; 224 -> 1/2; 0 -> lowest; tiny -> lowest; 57344 -> 2^7; beyond: held
    amax = [448.0, 448.5, 224.0, 0.0, 1e-44, 57344.0, 1e9, 1.0]
    assert A.kv_scale_exponent(amax).tolist() == [0, 1, -1, -127, -127, 7, 7, -8]


def test_record_layout_by_hand():
    cache = np.zeros((2, 16 * 644 + 32), dtype=np.uint8)
    A.kv_put(cache, 16, 16 + 3, np.arange(512) % 126, np.arange(64), [127, 128, 126, 134])
    row = cache[1]
    assert row[3 * 512 + 5] == 5 and row[512 * 16 + 3 * 128 + 2] == 1 and row[640 * 16 + 12:640 * 16 + 16].tolist() == [127, 128, 126, 134]
    assert cache[0].sum() == 0
    t = A.kv_token(cache, 16, 19)
    assert t[0] == 0 and t[56] == 1.0 and t[126 + 56] == 2.0      # code 0x38 is 1.0; dims 128.. have scale 2
    codes, pe, sc = A.kv_record(cache, 16, 19)
    assert (codes == np.arange(512) % 126).all() and (pe == np.arange(64)).all() and sc.tolist() == [127, 128, 126, 134]


def test_gather_follows_the_block_table():
    rng = np.random.default_rng(4)
    cache = _random_cache(rng, 4, 16)
    out = A.gather_kv(cache, 16, [[2, 0], [1, 3]], [0, 20, 23], [0, 14])
    assert (out[17] == A.kv_token(cache, 16, 1)).all() and (out[0] == A.kv_token(cache, 16, 32)).all()
    assert (out[20] == A.kv_token(cache, 16, 16 + 14)).all() and (out[22] == A.kv_token(cache, 16, 48)).all()


def test_attention_matches_torch_and_closed_forms():
    rng = np.random.default_rng(5)
    cache = _random_cache(rng, 2, 16)
    q = rng.normal(size=(3, 4, 576))
    slots = np.array([[0, 5, 31, -1, 7], [9, -1, -1, -1, -1], [-1, -1, -1, -1, -1]])
    out, lse, oerr, lerr = A.sparse_attention(q, cache, 16, slots, 0.05)
    k = np.stack([A.kv_token(cache, 16, s) for s in (0, 5, 31, 7)])
    w = torch.softmax(torch.tensor(q[0] @ k.T * 0.05), dim=1)
    assert np.allclose(out[0], w.numpy() @ k[:, :512])
    assert np.allclose(lse[0], torch.logsumexp(torch.tensor(q[0] @ k.T * 0.05), dim=1).numpy())
    # one token: its own value, whatever the query
    one = A.kv_token(cache, 16, 9)
    assert np.allclose(out[1], one[:512]) and np.allclose(lse[1], q[1] @ one * 0.05)
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all() and (oerr[2] == 0).all()
    # a token listed twice counts twice: the same output, ln 2 more
    o2, l2, _, _ = A.sparse_attention(q[1:2], cache, 16, np.array([[9, 9]]), 0.05)
    assert np.allclose(o2[0], one[:512]) and np.allclose(l2[0], lse[1] + np.log(2))
    # spans, counts, and entries outside the cache
    a = A.sparse_attention(q[:1], cache, 16, np.array([[0, 5, 64 + 15, 7, 16, 64 + 16, 128]]), 0.05, block_span=64)
    assert np.allclose(a[0], out[:1])
    b = A.sparse_attention(q[:1], cache, 16, np.array([[0, 5, 31, 7, 9, 10]]), 0.05, n_sel=[4])
    assert np.allclose(b[0], out[:1]) and np.allclose(b[1], lse[:1])


def test_disjoint_lists_join_by_their_lse():
    rng = np.random.default_rng(6)
    cache = _random_cache(rng, 2, 16)
    q = rng.normal(size=(1, 2, 576))
    o, l, _, _ = A.sparse_attention(q, cache, 16, np.arange(32)[None], 0.1)
    o1, l1, _, _ = A.sparse_attention(q, cache, 16, np.arange(11)[None], 0.1)
    o2, l2, _, _ = A.sparse_attention(q, cache, 16, np.arange(11, 32)[None], 0.1)
    l12 = np.logaddexp(l1, l2)
    assert np.allclose(l12, l)
    assert np.allclose(np.exp(l1 - l12)[..., None] * o1 + np.exp(l2 - l12)[..., None] * o2, o)


def test_binary32_attention_with_bf16_weights_stays_within_the_stated_errors():
    rng = np.random.default_rng(7)
    for n, amp in ((1, 1.0), (33, 2.0), (700, 4.0)):
        tok = torch.tensor(rng.normal(size=(n, 576))).bfloat16()
        q = torch.tensor(rng.normal(size=(3, 576)) * amp).bfloat16()
        out, lse, oerr, lerr = A.sparse_attention_row(q.double().numpy(), tok.double().numpy(), 576 ** -0.5)
        z = q.float() @ tok.float().T * 576 ** -0.5
        p = torch.exp(z - z.amax(1, keepdim=True))
        o = (p.bfloat16().float() @ tok.float()[:, :512] / p.sum(1, keepdim=True)).bfloat16()
        assert (np.abs(o.double().numpy() - out) <= oerr).all()
        assert (np.abs(torch.logsumexp(z, 1).double().numpy() - lse) <= lerr).all()


def test_scale_code_255_stands_for_nan():
    cache = np.zeros((1, 16 * 644), dtype=np.uint8)
    A.kv_put(cache, 16, 2, np.zeros(512), np.zeros(64), [127, 255, 134, 0])
    t = A.kv_token(cache, 16, 2)
    assert np.isnan(t[128:256]).all() and (np.delete(t, np.arange(128, 256)) == 0).all()
