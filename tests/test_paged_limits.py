"""Sizes at which the sums and products of the step tables would no longer fit their types (CPU only).

Every call fails its validation before anything is enqueued, so the fake pointers are never used.
"""

import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from test_paged_args import TABLES, UNSUPPORTED, _args, lib  # noqa: F401


@pytest.mark.parametrize("B,pages", [(4, 1 << 29), (2, (1 << 30) + 1), (8192, 1 << 18), (3, (1 << 31) - 1)])
def test_tables_of_more_entries_than_32_bits_count(lib, B, pages):  # noqa: F811
    """A fresh block is found by its number among all requests', which is at most the number of the table's entries."""
    assert lib.idx_build_tables(*_args(TABLES, {"B": B, "pages": pages, "ld_bt": pages})) == UNSUPPORTED


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 64, -(1 << 32) + 64])
def test_block_sizes_beyond_32_bits(monkeypatch, value):
    """ctypes would cut them to a size that is taken."""
    made = []
    monkeypatch.setattr(idx, "_cuda_device", lambda fn, name, t: -1)
    monkeypatch.setattr(idx, "_call", lambda *a: made.append(a))

    def ints(n, dtype=torch.int32):
        return torch.zeros(n, dtype=dtype)

    def build(block_size):
        idx.idx_build_tables(ints(2), ints(2), ints(9), ints(8).view(2, 4), block_size, ints(2), ints(3), ints(5), ints(5, torch.int64))

    with pytest.raises(ValueError, match="block_size .* 32 bits"):
        build(value)
    assert not made
    build(64)
    assert len(made) == 1
