"""Sizes at which the sums and products of the step tables would no longer fit their types (CPU only).

Every call fails its validation before anything is enqueued, so the fake pointers are never used.
"""

import pytest

from test_paged_args import TABLES, UNSUPPORTED, _args, lib  # noqa: F401


@pytest.mark.parametrize("B,pages", [(4, 1 << 29), (2, (1 << 30) + 1), (8192, 1 << 18), (3, (1 << 31) - 1)])
def test_tables_of_more_entries_than_32_bits_count(lib, B, pages):  # noqa: F811
    """A fresh block is found by its number among all requests', which is at most the number of the table's entries."""
    assert lib.idx_build_tables(*_args(TABLES, {"B": B, "pages": pages, "ld_bt": pages})) == UNSUPPORTED
