"""Order of the attention kernel's tensor-memory reads, shown from its source (CPU only).

A barrier's wait tests one parity bit, so it holds a warp only if that warp has followed the barrier's
earlier phases. Of the two ``o_done`` barriers the softmax warps follow both; a loader warp follows its own stage's.
"""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sparse_attention_indexer_fp8_gb300", "csrc", "attention.cu")


class Barrier:
    """One arrival completes a phase; a parity wait passes while the phase before the pending one has that parity."""

    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def passes(self, parity):
        return (self.phase - 1) & 1 == parity


def early_passes(tiles):
    """Groups of loaders that a parity wait on the last O product would let pass before that product is complete.

    Group g may come to its end as soon as its last tile is stored: once O of that tile's predecessor in the stage is
    complete, which is when its next-to-last phase of ``o_done[g]`` is."""
    last = tiles - 1
    early = set()
    for group in (0, 1):
        own = [i for i in range(tiles) if i % 2 == group]
        first = own[-1] - 2 if own else -1         # O of tiles 0 .. first is complete at the earliest
        for done in range(max(first, -1) + 1, last + 1):  # ... and of tiles 0 .. done - 1, the last one's is not
            bars = (Barrier(), Barrier())
            for i in range(done):
                bars[i & 1].arrive()
            if bars[last & 1].passes((last >> 1) & 1):
                early.add(group)
    return early


def test_a_wait_by_parity_does_not_hold_the_other_stages_loaders():
    assert early_passes(1) == early_passes(2) == set()
    assert all(early_passes(n) for n in range(3, 40))


@pytest.fixture(scope="module")
def epilogue():
    with open(SOURCE) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text[text.index("- epilogue\n"):text.index("tmem_dealloc(tmem")])
    return [m.group(0) for m in re.finditer(
        r"wait_bar\(|epilogue_bar\(|__syncthreads\(|tc_fence_after\(|tc_fence_before\(|tmem_ld\w*\(|if \(warp < 4\)|if \(warp >= 4\)",
        text)]


def test_only_warps_that_followed_both_stages_wait_for_the_last_product(epilogue):
    at = epilogue.index("wait_bar(")
    assert epilogue.count("wait_bar(") == 1 and epilogue[at - 1] == "if (warp < 4)"
    # what they saw is passed on by the block barrier, fenced on both sides
    assert epilogue[at + 1:at + 4] == ["tc_fence_after(", "tc_fence_before(", "epilogue_bar("]


def test_every_tensor_memory_read_is_fenced_after_the_barrier_that_orders_it(epilogue):
    fenced = False
    reads = 0
    for what in epilogue:
        if what in ("wait_bar(", "epilogue_bar("):
            fenced = False
        elif what == "tc_fence_after(":
            fenced = True
        elif what.startswith("tmem_ld"):
            assert fenced
            reads += 1
    assert reads > 0
