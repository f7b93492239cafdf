"""Extents beyond 32 bits are refused by the bindings, not cut to their lower half (CPU only)."""

import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx


def meta(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(1, 1 << 31), (1, (1 << 32) + 5), ((1 << 32) + 1, 1)])
def test_lists_and_tables(shape):
    with pytest.raises(ValueError, match="2\\*\\*31"):
        idx._mat("f", "slots", meta(*shape), -1, torch.int32, None, None)


def test_the_longest_extents_that_fit():
    assert idx._mat("f", "slots", meta(1, (1 << 31) - 1), -1, torch.int32, 1, None)[1] == (1 << 31) - 1


@pytest.mark.parametrize("shape", [((1 << 32) + 1, 1, 576), (1, (1 << 32) + 1, 576)])
def test_heads(shape):
    with pytest.raises(ValueError, match="2\\*\\*31"):
        idx._heads("f", "q", meta(*shape, dtype=torch.bfloat16), -1, None, None, 576)


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 64, -(1 << 31) - 1])
def test_whole_numbers(value):
    with pytest.raises(ValueError, match="block_span .* 32 bits"):
        idx._int32("f", "block_span", value)
    for sizes in ((value, 8, 8), (8, value, 8), (8, 8, value)):
        with pytest.raises(ValueError, match="32 bits"):
            idx.idx_sparse_attention_workspace_bytes(*sizes)
    assert idx._int32("f", "block_span", 64) == 64
