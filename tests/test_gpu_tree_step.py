"""Steps of a speculative server: tables, masks, inserts and tree attention one after the other, over several steps."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import paged as P
from sparse_attention_indexer_fp8_gb300 import workloads as W
from sparse_attention_indexer_fp8_gb300.pipeline import TreeStep

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Server:
    """Requests of ``cached`` tokens, their pages and the projections of every token that was ever inserted."""

    def __init__(self, B, H, bs, rows, pages, seed):
        self.B, self.H, self.bs, self.rows = B, H, bs, rows
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.step = TreeStep(B, rows, H, words=2, block_size=bs, device=DEV)
        self.cache = torch.zeros((B * pages, W.kv_block_stride_bytes(bs)), dtype=torch.uint8, device=DEV)
        self.table = torch.full((B, pages), -1, dtype=torch.int32, device=DEV)
        self.free = i32(self.rng.permutation(B * pages))
        self.cached = np.zeros(B, dtype=np.int64)
        ang = torch.rand((500, 32), generator=self.g, device=DEV) * 6.28
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1)
        self.weight = torch.randn(512, generator=self.g, device=DEV)
        self.first = True

    def random(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV).bfloat16()

    def run(self, parents, kv):
        """``parents`` of each request, ``kv`` of its rows; returns (q, out, lse) of the step."""
        counts = [len(x) for x in parents]
        pad = self.rows - sum(counts)
        st = self.step
        keep = {} if self.first else {"held_pages": st.held_pages.clone(), "free_start": st.free_end.clone()}
        self.first = False
        st.plan(i32(self.cached), i32(counts), i32(sum(parents, []) + [7] * pad), self.free, self.table, **keep)
        q = 2 * self.random(self.rows, self.H, 576)
        st.out.fill_(3)
        st.layer(torch.cat([kv, self.random(pad, 576)]), self.weight, self.cos_sin, q, self.cache, self.table)
        idx.idx_device_error()
        return q

    def check(self, parents, q):
        counts = [len(x) for x in parents]
        st = self.step
        cache, table = self.cache.cpu().numpy(), self.table.cpu().numpy()
        tokens = [P.context(cache, self.bs, table[b], int(self.cached[b]) + counts[b]) for b in range(self.B)]
        rows = [(b, i) for b, n in enumerate(counts) for i in range(n)]
        sets = [P.tree_sets(x) for x in parents]
        qs = q.double().cpu().numpy()[:len(rows)]

        def seen(t):
            b, i = rows[t]
            return list(range(int(self.cached[b]))) + sorted(int(self.cached[b]) + m for m in sets[b][i])

        out, lse, oerr, lerr = P.attention(qs, lambda t: tokens[rows[t][0]], seen, st.softmax_scale)
        n = len(rows)
        assert (np.abs(st.out[:n].double().cpu().numpy() - out) <= oerr).all()
        assert (np.abs(st.lse[:n].double().cpu().numpy() - lse) <= lerr).all()
        assert (st.out[n:] == 3).all()
        assert st.positions[:n].tolist() == [int(self.cached[b]) + len(sets[b][i]) - 1 for b, i in rows]


@pytest.mark.parametrize("B,H,bs", [(3, 20, 16), (5, 64, 64), (1, 128, 16)])
def test_prompt_drafts_and_acceptance(B, H, bs):
    s = Server(B, H, bs, rows=64 * B, pages=200 // bs + 1, seed=B)
    # prompts: chains
    lens = [int(n) for n in s.rng.integers(1, 60, B)]
    kv = s.random(sum(lens), 576)
    chain = [list(range(-1, n - 1)) for n in lens]
    q = s.run(chain, kv)
    s.check(chain, q)
    accepted = list(torch.split(kv, lens))  # projections of each request's tokens, in order
    s.cached += lens
    pending = [torch.zeros((0, 576), dtype=torch.bfloat16, device=DEV)] * B  # accepted, not yet at their own slots
    for _ in range(3):
        trees, rows = [], []
        for b in range(B):
            k, n = len(pending[b]), int(s.rng.integers(2, 20))
            # accepted tokens in a chain, the new tree below the last of them
            up = list(range(-1, k - 1)) + [k - 1 if i == 0 else int(s.rng.integers(max(k, k + i - 4), k + i)) for i in range(n)]
            trees.append(up)
            rows.append(torch.cat([pending[b], s.random(n, 576)]))
        q = s.run(trees, torch.cat(rows))
        s.check(trees, q)
        for b in range(B):
            k = len(pending[b])
            s.cached[b] += k  # at their own slots now
            accepted[b] = torch.cat([accepted[b], pending[b]])
            path, at = [], len(trees[b]) - 1 if b % 2 else k
            while at >= k:
                path.append(at)
                at = trees[b][at]
            pending[b] = rows[b][path[::-1]]
    # every request's records are those of its tokens inserted one after the other
    pages = s.table.shape[1]
    for b in range(B):
        n = int(s.cached[b])
        fresh = torch.zeros((pages, s.cache.shape[1]), dtype=torch.uint8, device=DEV)
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        kv = accepted[b].contiguous()
        idx.idx_kv_norm_rope_quant_and_cache(kv[:, :512], kv[:, 512:], s.weight, 1e-6, pos, s.cos_sin, pos.long(), fresh, bs)
        got = P.context(s.cache.cpu().numpy(), bs, s.table[b].tolist(), n)
        assert np.array_equal(got, P.context(fresh.cpu().numpy(), bs, range(pages), n))
    idx.idx_device_error()


def test_a_captured_step():
    """Plan and layer in one graph, replayed with other lengths and parents in the same tensors."""
    B, H, bs, rows = 4, 16, 16, 40
    s = Server(B, H, bs, rows, 12, seed=11)
    lens = [30, 17, 1, 5]
    chain = [list(range(-1, n - 1)) for n in lens]
    s.step = TreeStep(B, 64, H, words=2, block_size=bs, device=DEV)
    s.rows = 64
    s.run(chain, s.random(sum(lens), 576))
    held, end = s.step.held_pages.clone(), s.step.free_end.clone()
    s.cached += lens
    st = s.step = TreeStep(B, rows, H, words=2, block_size=bs, device=DEV)
    s.rows = rows
    cached, new, parents = i32(s.cached), i32([0] * B), i32([0] * rows)
    kv, q = s.random(rows, 576), 2 * s.random(rows, H, 576)

    def run():
        st.plan(cached, new, parents, s.free, s.table, held_pages=held, free_start=end)
        st.layer(kv, s.weight, s.cos_sin, q, s.cache, s.table)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for counts in ([3, 0, 12, 8], [10, 10, 10, 10], [0, 1, 0, 0]):
        trees = [[-1] * min(n, 1) + [int(s.rng.integers(-1, i)) for i in range(1, n)] for n in counts]
        new.copy_(i32(counts))
        parents.copy_(i32(sum(trees, []) + [0] * (rows - sum(counts))))
        st.out.fill_(3)
        g.replay()
        idx.idx_device_error()
        s.check(trees, q)
