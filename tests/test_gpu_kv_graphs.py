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


def test_graphs_that_share_a_workspace_clear_it_each():
    """A workspace that an FFN call used last, passed to two captures: the second
    is replayed alone, then both in turn, then eager calls of either kind."""
    from activation_sparse_predictor_amd import binding as B
    from synthetic import custom_config, make_layer, make_tokens
    cfg = custom_config("relu", 256, 1000, 64, mean=0.2, number=120)
    layer = R.to_device(make_layer(cfg), DEV)
    x = make_tokens(cfg, 1).to(DEV)
    fy, idx, cnt = R.decode(layer, x)
    data = [case(*CASES[i], seed=80 + i) for i in (1, 0, 3)]
    need = max([B.pi_workspace_size(B.PI_OP_DECODE, 1, cfg.d, cfg.r, cfg.ffn)]
               + [B.pi_kv_workspace_size(len(b["ctx"]), q.shape[0], b["max_q"], q.shape[1], c["k"].shape[1], q.shape[2]) for c, b, q in data])
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def ffn():
        y = torch.empty_like(fy)
        B.check(B.pi_ffn_decode(B.PI_FFN_RELU, x, 1, cfg.d, cfg.ffn, layer["P1"], None, B.PI_ACT_RELU, layer["P2"], layer["b2"],
                                cfg.r, 0.5, layer["W_up"], layer["b_up"], None, None, layer["W_down"], torch.empty_like(idx),
                                torch.empty_like(cnt), y, 0, ws, ws.numel()), "pi_ffn_decode")
        torch.cuda.synchronize()
        return y

    def same(i):
        graphs[i][1].fill_(float("nan"))
        graphs[i][0].replay()
        torch.cuda.synchronize()
        return torch.equal(graphs[i][1], want[i])

    want = [R.kv_attend(c, q, b) for c, b, q in data]
    assert torch.equal(ffn(), fy)
    graphs = [capture(*d, ws=ws) for d in data]
    for i in (2, 1, 2, 0, 1, 0):
        assert same(i), i
    assert torch.equal(ffn(), fy)
    for i, (c, b, q) in enumerate(data):
        assert torch.equal(R.kv_attend(c, q, b, ws=ws), want[i])
    assert all(same(i) for i in (1, 0, 2)) and torch.equal(ffn(), fy)
    assert torch.equal(R.kv_attend(data[0][0], data[0][2], data[0][1], ws=ws), want[0])
