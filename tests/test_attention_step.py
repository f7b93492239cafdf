"""The layer's decode step on the host: what it refuses, in which order it calls, and where (CPU only).

The step's calls are replaced by records of themselves, so nothing is computed and no GPU is needed.
"""

import contextlib

import numpy as np
import pytest
import torch

from oracle.attention import sparse_attention_row
from sparse_attention_indexer_fp8_gb300 import pipeline

B, H, L, BS = 3, 8, 256, 64
CALLS = ["idx_k_norm_rope_quant_and_cache", "idx_kv_norm_rope_quant_and_cache", "idx_q_rope_quant",
         "idx_paged_mqa_logits_decode", "idx_topk", "idx_sparse_attention"]


@pytest.fixture
def calls(monkeypatch):
    """Names of the calls made, in order."""
    made = []
    for name in CALLS:
        monkeypatch.setattr(pipeline, name, lambda *a, _n=name, **k: made.append(_n))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return made


def arguments(**change):
    f = torch.zeros
    a = dict(new_k=f(B, 128), new_kv=f(B, 576), k_weight=f(128), k_bias=None, kv_weight=f(512),
             positions=f(B, dtype=torch.int32), cos_sin=f(L, 64), new_slots=f(B, dtype=torch.int64),
             q_index=f(B, 64, 128), w_index=f(B, 64), q=f(B, H, 576, dtype=torch.bfloat16),
             k_cache=f(12, 8704, dtype=torch.uint8), kv_cache=f(12, 41472, dtype=torch.uint8),
             block_table=f(B, L // BS, dtype=torch.int32), ctx_lens=f(B, dtype=torch.int32))
    a.update(change)
    return a


def test_one_step_calls_everything_once(calls):
    step = pipeline.AttentionDecodeStep(B, L, heads=H, topk=64, device="cpu")
    step.run(**arguments())
    assert calls == CALLS
    step.run(**arguments(q_index=torch.zeros(B, 8192)))          # heads laid out in one row
    assert calls == 2 * CALLS
    # tables and weights of a larger batch, of which the step uses the first rows
    step.run(**arguments(block_table=torch.zeros(B + 5, 4, dtype=torch.int32), w_index=torch.zeros(B + 1, 64)))
    assert calls == 3 * CALLS


@pytest.mark.parametrize("name,value", [
    ("ctx_lens", torch.zeros(B - 1, dtype=torch.int32)),         # the selection reads one length per row of the step
    ("ctx_lens", torch.zeros(B, dtype=torch.int64)),
    ("ctx_lens", torch.zeros(2 * B, dtype=torch.int32)[::2]),
    ("block_table", torch.zeros(B - 1, 4, dtype=torch.int32)),
    ("block_table", torch.zeros(B, 4, dtype=torch.int64)),
    ("q_index", torch.zeros(B + 1, 64, 128)),                    # the step's q8 has B rows
    ("q_index", torch.zeros(B - 1, 64, 128)),
    ("q_index", torch.zeros(B, 32, 128)),
    ("q_index", torch.zeros(B, 8191)),
    ("w_index", torch.zeros(B, 32)),
    ("w_index", torch.zeros(B - 1, 64)),
    ("w_index", torch.zeros(64)),
    ("new_k", torch.zeros(B - 1, 128)),                          # with it go the positions that q is rotated by
    ("q", torch.zeros(B, H + 1, 576, dtype=torch.bfloat16)),
    ("q", torch.zeros(B + 1, H, 576, dtype=torch.bfloat16)),
])
def test_a_step_refuses_other_shapes_before_it_enqueues_anything(calls, name, value):
    step = pipeline.AttentionDecodeStep(B, L, heads=H, topk=64, device="cpu")
    with pytest.raises(ValueError, match=name):
        step.run(**arguments(**{name: value}))
    assert calls == []


class OnDevice:
    """What the step sees of a tensor on another device than the current one."""

    def __init__(self, tensor, index):
        self.tensor, self.device, self.index = tensor, torch.device("cuda", index), index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.tensor, name)

    def __getitem__(self, at):
        return OnDevice(self.tensor[at], self.index)


@pytest.mark.parametrize("method", ["run", "insert"])
def test_a_step_on_another_device_makes_every_call_there(calls, monkeypatch, method):
    current = [0]
    seen = []

    @contextlib.contextmanager
    def device(d):
        was, current[0] = current[0], torch.device(d).index if not isinstance(d, int) else d
        yield
        current[0] = was

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    for name in CALLS:
        monkeypatch.setattr(pipeline, name, lambda *a, _n=name, **k: seen.append((_n, current[0])))
    step = pipeline.AttentionDecodeStep(B, L, heads=H, topk=64, device="cpu")
    step.out = OnDevice(step.out, 1)
    args = {k: OnDevice(v, 1) if isinstance(v, torch.Tensor) else v for k, v in arguments().items()}
    if method == "run":
        step.run(**args)
        assert seen == [(n, 1) for n in CALLS]
    else:
        step.insert(*(args[n] for n in ("new_k", "new_kv", "k_weight", "k_bias", "kv_weight", "positions", "cos_sin",
                                        "new_slots", "k_cache", "kv_cache")))
        assert [n for n, _ in seen] == CALLS[:2]        # they choose the device of their tensors themselves
    assert current[0] == 0


def test_the_default_scale_is_that_of_the_heads_before_absorption(calls):
    # heads of 128 dims without and 64 with position: their attention, and the absorbed query's over the latents
    rng = np.random.default_rng(3)
    heads, n = 4, 40
    up = rng.normal(size=(heads, 128, 512)) / 512 ** 0.5           # latent -> key dims of each head
    q_nope, q_pe = rng.normal(size=(heads, 128)), rng.normal(size=(heads, 64))
    tokens = rng.normal(size=(n, 576))
    keys = np.einsum("hdc,nc->hnd", up, tokens[:, :512])
    z = (np.einsum("hd,hnd->hn", q_nope, keys) + q_pe @ tokens[:, 512:].T) / 192 ** 0.5
    p = np.exp(z - z.max(axis=1, keepdims=True))
    want = p / p.sum(axis=1, keepdims=True) @ tokens[:, :512]
    absorbed = np.concatenate([np.einsum("hd,hdc->hc", q_nope, up), q_pe], axis=1)
    step = pipeline.AttentionDecodeStep(B, L, heads=H, topk=64, device="cpu")
    out, lse, _, _ = sparse_attention_row(absorbed, tokens, step.softmax_scale)
    assert np.allclose(out, want, rtol=1e-10, atol=1e-12)
    assert np.allclose(lse, np.log(np.exp(z).sum(axis=1)), rtol=1e-10)
    assert pipeline.AttentionDecodeStep(B, L, heads=H, topk=64, device="cpu", softmax_scale=0.5).softmax_scale == 0.5
