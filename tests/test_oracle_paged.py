"""The host statements of the step tables, the trees and the attention over contexts, pinned by hand and by brute force."""

import numpy as np

from oracle import attention as A
from oracle import paged as P
from oracle.codecs import bf16_encode, e4m3_decode


def test_tables_by_hand():
    # blocks of 16: request 0 has 15 tokens in one block and brings 3, request 1 brings nothing, request 2 starts with 17
    table = [[7, -1, -1], [9, 4, -1], [-1, -1, -1]]
    r = P.build_tables([15, 20, 0], [3, 0, 17], [30, 31, 32, 33], table, 16, 22, start=1)
    assert r["table"].tolist() == [[7, 31, -1], [9, 4, -1], [32, 33, -1]]
    assert r["ctx_lens"].tolist() == [18, 20, 17] and r["cu_rows"].tolist() == [0, 3, 3, 20]
    assert r["cu_ctx"].tolist() == [0, 18, 38, 55] and r["held"].tolist() == [2, 2, 2] and r["free_end"] == 4
    assert r["positions"].tolist() == [15, 16, 17] + list(range(17)) + [0, 0]
    assert r["slots"].tolist() == [7 * 16 + 15, 31 * 16, 31 * 16 + 1] + [32 * 16 + i for i in range(16)] + [33 * 16, -1, -1]
    assert r["row_to_req"].tolist() == [0] * 3 + [2] * 17 + [0, 0]
    assert r["row_ke"].tolist() == [16, 17, 18] + list(range(1, 18)) + [0, 0]


def test_tables_without_room():
    # held pages are kept and used, and where the free blocks end the rest has no slot
    r = P.build_tables([0, 0], [20, 20], [5], [[8, 9], [-1, -1]], 16, 40, held=[2, 0])
    assert r["table"].tolist() == [[8, 9], [5, -1]] and r["held"].tolist() == [2, 1] and r["free_end"] == 1
    assert r["slots"][:20].tolist() == [8 * 16 + i for i in range(16)] + [9 * 16 + i for i in range(4)]
    assert r["slots"][20:].tolist() == [5 * 16 + i for i in range(16)] + [-1] * 4


def test_tree_by_hand():
    #   0      3
    #  1 2     4
    #    5
    sets = P.tree_sets([-1, 0, 0, -1, 3, 2])
    assert sets == [{0}, {0, 1}, {0, 2}, {3}, {3, 4}, {0, 2, 5}]
    assert P.mask_words(sets, 1)[:, 0].tolist() == [1, 3, 5, 8, 24, 37]
    chain = P.mask_words(P.tree_sets(range(-1, 39)), 2).view(np.uint32)
    assert chain[39].tolist() == [0xFFFFFFFF, 0xFF] and chain[31].tolist() == [0xFFFFFFFF, 0] and chain[32].tolist() == [0xFFFFFFFF, 1]
    assert P.tree_seen(3, 6, [37]) == [0, 1, 2, 3, 5, 8] and P.tree_seen(0, 2, [0]) == [] and P.tree_seen(1, 40, [1]) == [0, 1]


def test_window_by_hand():
    assert P.window_seen(5, 2, 0) == [4, 5] and P.window_seen(5, 2, 1) == [0, 4, 5] and P.window_seen(5, 100, 3) == list(range(6))
    assert P.window_seen(1, 1, 4) == [0, 1] and P.window_seen(-1, 3, 2) == []


def test_context_reads_the_records():
    rng = np.random.default_rng(0)
    bs, cache = 16, rng.integers(0, 256, (3, 16 * 644 + 16)).astype(np.uint8)
    cache[:, 640 * bs:644 * bs] = rng.integers(120, 130, (3, 64))
    cache[:, :512 * bs] &= 0x77  # no NaN codes
    pe = bf16_encode(rng.normal(size=(3, bs * 64)).astype(np.float32))
    cache[:, 512 * bs:640 * bs] = pe.view(np.uint8)
    got = P.context(cache, bs, [2, 0, 7], 40)
    for j in (0, 5, 16, 31):
        slot = [2, 0][j // bs] * bs + j % bs
        assert np.array_equal(got[j], A.kv_token(cache, bs, slot))
    assert np.isnan(got[32:]).all() and e4m3_decode(cache[2, :1])[0] * 2.0 ** (int(cache[2, 640 * bs]) - 127) == got[0, 0]


def test_attention_is_the_softmax_of_what_is_seen():
    rng = np.random.default_rng(1)
    tok, q = rng.normal(size=(9, 576)), rng.normal(size=(2, 3, 576))
    seen = [[0, 4, 8], []]
    out, lse, _, _ = P.attention(q, lambda t: tok, lambda t: seen[t], 0.1)
    w = np.exp(q[0] @ tok[seen[0]].T * 0.1)
    assert np.allclose(out[0], w @ tok[seen[0], :512] / w.sum(axis=1, keepdims=True)) and np.allclose(lse[0], np.log(w.sum(axis=1)))
    assert not out[1].any() and np.isneginf(lse[1]).all()
