"""Captured attention calls: every graph by itself, in any order, between eager
calls, gives what the eager call gives (bit for bit)."""

from __future__ import annotations

import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from tests.test_gpu_kv import DEV, filled, queries

pytestmark = pytest.mark.gpu


def case(new, ctx, heads, n_kv, d, seed):
    cache, rows = filled(ctx, n_kv, d, 16, "int8", seed=seed)
    return cache, R.kv_batch(new, ctx, rows, DEV), queries(sum(new), heads, d, seed)


def capture(cache, batch, q, **kw):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = R.kv_attend(cache, q, batch, **kw)
    return graph, y


# decode steps of two batch sizes (split contexts), a prompt beside them (both kernels), a split prompt
CASES = [([1, 1], [3000, 500], 8, 2, 128), ([1] * 5, [700, 2500, 1, 64, 4000], 8, 2, 128), ([150, 1, 2], [150, 400, 90], 64, 64, 64),
         ([1100], [4300], 8, 8, 64)]


@pytest.mark.parametrize("first", range(len(CASES)))
def test_graphs_without_a_workspace_replay_in_any_order(first):
    """Captured one after the other with no warm-up; the first replays begin with
    a later capture; larger eager calls, which replace the eager workspace, and
    other allocations in between."""
    data = [case(*c, seed=50 + i) for i, c in enumerate(CASES)]
    graphs = [capture(*x) for x in data]
    order = list(range(first, len(CASES))) + list(range(first))
    for turn in range(3):
        for i in order:
            cache, batch, q = data[i]
            q.copy_(torch.randn_like(q))
            graphs[i][1].fill_(float("nan"))
            graphs[i][0].replay()
            got = graphs[i][1].clone()
            want = R.kv_attend(cache, q, batch)
            junk = torch.full((40 << 20,), float("nan"), device=DEV)   # what an allocator might hand out next
            torch.cuda.synchronize()
            assert torch.equal(got, want), (turn, i)
            del junk


def test_graphs_replayed_on_two_streams():
    """Captures of one stream share nothing: replayed at once on two streams."""
    data = [case(*CASES[i], seed=60 + i) for i in (1, 1, 3)]
    graphs = [capture(*x) for x in data]
    want = [R.kv_attend(c, q, b) for c, b, q in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (g, y), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                y.fill_(float("nan"))
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for (g, y), w in zip(graphs, want):
            assert torch.equal(y, w)


def test_capture_on_a_warm_stream_outlives_the_eager_workspace():
    """A capture on a stream whose eager calls have a workspace: the workspace
    grows afterwards, and its old memory is filled with other things."""
    cache, batch, q = case(*CASES[0], seed=70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.kv_attend(cache, q, batch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = R.kv_attend(cache, q, batch)
    big = case(*CASES[3], seed=71)
    with torch.cuda.stream(side):
        R.kv_attend(big[0], big[2], big[1])
        junk = [torch.full((1 << 20,), -1, dtype=torch.int32, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, R.kv_attend(cache, q, batch)) and all(bool((t == -1).all()) for t in junk)
