"""Steps of drafted trees that carry their own lengths on, and what a step refuses, on the GPU."""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp8_gb300 as idx
from oracle import paged as P
from sparse_attention_indexer_fp8_gb300.pipeline import TreeStep
from test_gpu_tree_step import Server

pytestmark = pytest.mark.gpu
DEV = "cuda"
BS, PAGES = 16, 12


@pytest.fixture(scope="module", autouse=True)
def _library():
    from sparse_attention_indexer_fp8_gb300.build import build_library

    build_library()
    idx.library()
    yield
    idx.idx_device_error()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("how", ["eager", "stream", "raw stream", "graph"])
def test_lengths_pages_and_blocks_carried_on_in_place(how):
    """ctx_lens, held_pages and free_end of one step are the inputs of the next, in the step's own tensors."""
    B, rows = 4, 40
    rng = np.random.default_rng(3)
    step = TreeStep(B, rows, 2, words=2, block_size=BS, device=DEV)
    ids = rng.permutation(B * PAGES)
    table, free = torch.full((B, PAGES), -1, dtype=torch.int32, device=DEV), i32(ids)
    new, parents = i32([0] * B), i32([-1] * rows)
    side = torch.cuda.Stream() if how != "eager" else torch.cuda.current_stream()
    stream = {"stream": side, "raw stream": side.cuda_stream}.get(how)

    def plan():
        step.plan(step.ctx_lens, new, parents, free, table, held_pages=step.held_pages, free_start=step.free_end, stream=stream)

    graph = None
    if how == "graph":
        with torch.cuda.stream(side):
            plan()  # of no tokens: loads the kernels before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan()
    host_table, ctx, held, at = np.full((B, PAGES), -1), np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64), 0
    for counts in ([30, 0, 1, 8], [3, 5, 20, 12], [0, 0, 0, 0], [10, 1, 7, 16]):
        trees = [[int(rng.integers(max(-1, i - 4), i)) for i in range(n)] for n in counts]
        new.copy_(i32(counts))
        parents.copy_(i32(sum(trees, []) + [9] * (rows - sum(counts))))
        torch.cuda.synchronize()
        graph.replay() if graph else plan()
        torch.cuda.synchronize()
        idx.idx_device_error()
        want = P.build_tables(ctx, counts, ids, host_table, BS, rows, held, at)
        n = sum(counts)
        base = np.repeat(ctx, counts)
        depth = [len(s) - 1 for t in trees for s in P.tree_sets(t)]
        assert step.positions[:n].tolist() == [int(b) + d for b, d in zip(base, depth)]
        assert step.row_positions.tolist() == want["positions"].tolist() and step.slots.tolist() == want["slots"].tolist()
        assert np.array_equal(table.cpu().numpy(), want["table"])
        host_table, ctx, held, at = want["table"], want["ctx_lens"], want["held"], want["free_end"]
        assert step.ctx_lens.tolist() == ctx.tolist() and step.held_pages.tolist() == held.tolist() and step.free_end.item() == at


def test_a_refused_plan_takes_no_blocks():
    """After a refusal the same step is planned again, with the step's own pages and start: every block counts once."""
    B, rows = 2, 30
    step = TreeStep(B, rows, 2, words=1, block_size=BS, device=DEV)
    table, free = torch.full((B, PAGES), -1, dtype=torch.int32, device=DEV), torch.arange(50, dtype=torch.int32, device=DEV)
    lens, parents = i32([20, 10]), i32([-1] * rows)
    for bad in (parents[:-1], parents.long(), i32([-1] * 2 * rows)[::2]):
        with pytest.raises(ValueError, match="parents"):
            step.plan(step.ctx_lens, lens, bad, free, table, held_pages=step.held_pages, free_start=step.free_end)
    step.plan(step.ctx_lens, lens, parents, free, table, held_pages=step.held_pages, free_start=step.free_end)
    idx.idx_device_error()
    assert step.ctx_lens.tolist() == [20, 10] and step.held_pages.tolist() == [2, 1] and step.free_end.item() == 3
    assert table[:, :3].tolist() == [[0, 1, -1], [2, -1, -1]]


@pytest.mark.parametrize("H,graph", [(16, False), (16, True), (128, True)])
def test_a_step_over_contexts_that_are_cut(H, graph):
    """Prompts long enough that the step's attention shares its work out, then drafted trees over them; captured, too."""
    B, lens = 3, [900, 300, 1000]
    s = Server(B, H, 16, sum(lens) + 5, 1200 // 16, seed=H)
    s.step = TreeStep(B, s.rows, H, words=32, block_size=16, device=DEV)
    s.cos_sin = torch.cat([s.cos_sin] * 3)
    s.run([list(range(-1, n - 1)) for n in lens], s.random(sum(lens), 576))
    held, end = s.step.held_pages.clone(), s.step.free_end.clone()
    s.cached += lens
    rows = 30
    st = s.step = TreeStep(B, rows, H, words=1, block_size=16, device=DEV)
    s.rows = rows
    cached, new, parents = i32(s.cached), i32([0] * B), i32([0] * rows)
    kv, q = s.random(rows, 576), 2 * s.random(rows, H, 576)

    def run():
        st.plan(cached, new, parents, s.free, s.table, held_pages=held, free_start=end)
        st.layer(kv, s.weight, s.cos_sin, q, s.cache, s.table)

    run()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
    for counts in ([3, 0, 12], [10, 10, 10], [0, 1, 0], [1, 1, 1]):
        trees = [[-1] * min(n, 1) + [int(s.rng.integers(-1, i)) for i in range(1, n)] for n in counts]
        new.copy_(i32(counts))
        parents.copy_(i32(sum(trees, []) + [0] * (rows - sum(counts))))
        st.out.fill_(3)
        st.ws.fill_(255)
        g.replay() if graph else run()
        idx.idx_device_error()
        assert (st.ws != 255).any()  # every worker noted its cut
        s.check(trees, q)


def test_an_accepted_chain_stays_where_it_is():
    """Nodes accepted from the first on, each the child of the one before, are counted by the next step and not brought again."""
    B, H, bs = 2, 16, 16
    s = Server(B, H, bs, rows=80, pages=10, seed=21)
    lens = [20, 7]
    kv = s.random(sum(lens), 576)
    s.run([list(range(-1, n - 1)) for n in lens], kv)
    tokens = list(torch.split(kv, lens))
    s.cached += lens
    for keep in ((4, 1), (6, 0), (2, 5)):
        # a chain of six and, for the second request, siblings behind it
        trees = [list(range(-1, 5)), list(range(-1, 5)) + [2, 2, -1]]
        kv = s.random(sum(len(t) for t in trees), 576)
        q = s.run(trees, kv)
        s.check(trees, q)
        parts = torch.split(kv, [len(t) for t in trees])
        for b in range(B):
            tokens[b] = torch.cat([tokens[b], parts[b][:keep[b]]])
            s.cached[b] += keep[b]
    for b in range(B):
        n = int(s.cached[b])
        fresh = torch.zeros((10, s.cache.shape[1]), dtype=torch.uint8, device=DEV)
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        x = tokens[b].contiguous()
        idx.idx_kv_norm_rope_quant_and_cache(x[:, :512], x[:, 512:], s.weight, 1e-6, pos, s.cos_sin, pos.long(), fresh, bs)
        got = P.context(s.cache.cpu().numpy(), bs, s.table[b].tolist(), n)
        assert np.array_equal(got, P.context(fresh.cpu().numpy(), bs, range(10), n))
    idx.idx_device_error()
