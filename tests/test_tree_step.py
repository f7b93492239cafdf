"""The step of drafted trees on the host: which tensors its calls get, and what it refuses (CPU only).

The step's calls are replaced by records of themselves that do on the host what the test looks at, so no GPU is needed.
"""

import contextlib

import pytest
import torch

from sparse_attention_indexer_fp8_gb300 import pipeline

B, ROWS, H, BS, PAGES = 3, 12, 8, 16, 5


@pytest.fixture
def calls(monkeypatch):
    """(name, base_lens as they are when the masks are made) of the calls, in order."""
    made = []

    def tables(cached, new, free, table, bs, ctx, cu, *a, **k):
        made.append(("tables", None))
        ctx.copy_(cached + new)  # as the header allows, also where ctx is cached

    def masks(parents, cu, mask, base_lens=None, positions=None, stream=None):
        made.append(("masks", base_lens.tolist()))

    monkeypatch.setattr(pipeline, "idx_build_tables", tables)
    monkeypatch.setattr(pipeline, "idx_tree_mask", masks)
    monkeypatch.setattr(pipeline, "idx_kv_norm_rope_quant_and_cache", lambda *a, **k: made.append(("insert", None)))
    monkeypatch.setattr(pipeline, "idx_tree_attention", lambda *a, **k: made.append(("attention", None)))
    monkeypatch.setattr(pipeline, "idx_paged_attention_workspace_bytes", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return made


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def plan_arguments(**change):
    a = dict(cached_lens=i32(B), new_lens=i32(B) + 2, parents=i32(ROWS), free_blocks=i32(20), block_table=i32(B, PAGES))
    a.update(change)
    return a


def test_lengths_that_the_step_advances_itself(calls):
    """cached_lens may be the step's own ctx_lens: positions count from the lengths before the step."""
    step = pipeline.TreeStep(B, ROWS, H, block_size=BS, device="cpu")
    step.plan(**plan_arguments(cached_lens=torch.tensor([5, 0, 9], dtype=torch.int32)))
    step.plan(**plan_arguments(cached_lens=step.ctx_lens))
    step.plan(**plan_arguments(cached_lens=step.ctx_lens))
    assert step.ctx_lens.tolist() == [11, 6, 15]
    assert [c for c in calls if c[0] == "masks"] == [("masks", [5, 0, 9]), ("masks", [7, 2, 11]), ("masks", [9, 4, 13])]


def layer_arguments(**change):
    a = dict(kv=torch.zeros(ROWS, 576), kv_weight=torch.zeros(512), cos_sin=torch.zeros(64, 64),
             q=torch.zeros(ROWS, H, 576, dtype=torch.bfloat16), kv_cache=torch.zeros(9, 10752, dtype=torch.uint8),
             block_table=i32(B, PAGES))
    a.update(change)
    return a


def test_one_step_calls_everything_once(calls):
    step = pipeline.TreeStep(B, ROWS, H, block_size=BS, device="cpu")
    step.plan(**plan_arguments())
    step.layer(**layer_arguments())
    # strided queries that the attention takes
    step.layer(**layer_arguments(q=torch.zeros(H, ROWS, 584, dtype=torch.bfloat16).transpose(0, 1)[:, :, :576]))
    assert [c[0] for c in calls] == ["tables", "masks"] + 2 * ["insert", "attention"]


@pytest.mark.parametrize("name,value", [
    ("parents", i32(ROWS - 1)),                     # the tables would count their blocks before the masks refuse it
    ("parents", i32(ROWS + 1)),
    ("parents", i32(ROWS).long()),
    ("parents", i32(2 * ROWS)[::2]),
    ("parents", i32(ROWS, 1)),
    ("cached_lens", i32(B + 1)),
    ("cached_lens", i32(B).long())])
def test_a_plan_refuses_other_tensors_before_it_enqueues_anything(calls, name, value):
    step = pipeline.TreeStep(B, ROWS, H, block_size=BS, device="cpu")
    with pytest.raises(ValueError, match=name):
        step.plan(**plan_arguments(**{name: value}))
    assert calls == []


@pytest.mark.parametrize("name,value", [
    ("q", torch.zeros(ROWS + 1, H, 576, dtype=torch.bfloat16)),
    ("q", torch.zeros(ROWS - 1, H, 576, dtype=torch.bfloat16)),
    ("q", torch.zeros(ROWS, H + 1, 576, dtype=torch.bfloat16)),
    ("q", torch.zeros(ROWS, H, 512, dtype=torch.bfloat16)),
    ("q", torch.zeros(ROWS, H, 576)),
    ("q", torch.zeros(ROWS, H, 580, dtype=torch.bfloat16)[:, :, :576]),              # heads 1160 bytes apart
    ("q", torch.zeros(ROWS * H * 576 + 4, dtype=torch.bfloat16)[4:].view(ROWS, H, 576)),  # begins between 16-byte boundaries
    ("q", torch.zeros(1, H, 576, dtype=torch.bfloat16).expand(ROWS, H, 576)),
    ("block_table", i32(B + 1, PAGES)),
    ("block_table", i32(B, PAGES).long()),
    ("block_table", i32(B, 2 * PAGES)[:, ::2])])
def test_a_layer_refuses_other_tensors_before_it_enqueues_anything(calls, name, value):
    step = pipeline.TreeStep(B, ROWS, H, block_size=BS, device="cpu")
    with pytest.raises(ValueError, match=name):
        step.layer(**layer_arguments(**{name: value}))
    assert calls == []


@pytest.mark.parametrize("change,match", [
    ({"words": 0}, "words"), ({"words": 33}, "words"), ({"heads": 1025}, "heads"), ({"requests": 8193}, "requests"),
    ({"block_size": 48}, "block_size"), ({"softmax_scale": float("inf")}, "softmax_scale")])
def test_a_step_that_no_call_would_take_is_not_made(calls, change, match):
    with pytest.raises(ValueError, match=match):
        pipeline.TreeStep(**{"requests": B, "rows": ROWS, "heads": H, "device": "cpu", **change})
