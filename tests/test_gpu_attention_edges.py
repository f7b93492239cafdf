"""Edges of the inserts, the read-back and the sparse attention: values that are not finite."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import attention as A
from oracle.codecs import bf16_encode

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
