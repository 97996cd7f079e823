"""Pieces of more than 64 tiles that begin with drafted ones, in the kernel of many rows: its
table of looked-up granules holds 64 tiles at a time and is refilled behind them.

The sequences share their pages (one long context, of which each takes its own
length), and a few contents are repeated over all of them, so that the float64
reference is only needed for those: a copy's results are its own bit for bit.
The bound is test_gpu_tree.py's.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O
from oracle import kv as KV
from tests.test_gpu_kv import filled, host
from tests.test_gpu_tree import DEV, drafted, queries, trees

pytestmark = pytest.mark.gpu


def contents(lengths, nodes, copies, heads, n_kv, d, fmt, seed):
    """The batch, its inputs (contents in turn, `copies` times) and the cached keys and values in float64."""
    cache, rows = filled([max(lengths)], n_kv, d, 64, fmt, seed=seed)
    n = len(lengths)
    batch = R.kv_batch([nodes] * (n * copies), lengths * copies, rows * (n * copies), DEV)
    tree = R.kv_tree(trees([nodes] * n, seed), device=DEV)
    pos = (torch.tensor(lengths, device=DEV).repeat_interleave(nodes) + tree["depth"]).to(torch.int32)
    one = [queries(n * nodes, heads, d, seed + 5), *drafted(n * nodes, n_kv, d, seed + 6)]
    q, k, v = (t.repeat(copies, 1, 1) for t in one)
    kept = host(cache)
    stored = []
    for name, at in zip("kv", KV.places(64, d)):
        codes = KV.decode(kept[name][rows[0]].reshape(len(rows[0]), n_kv, -1)[:, :, at], fmt)
        x = codes * kept[name + "_scale"][rows[0]].astype(np.float64)[:, :, None, None]   # pages x n_kv x 64 x d
        stored.append(x.transpose(0, 2, 1, 3).reshape(-1, n_kv, d)[:max(lengths)])
    assert all(np.array_equal(stored["kv".index(name)][j], KV.stored(kept, rows[0], j, name)) for name in "kv" for j in (0, 77, max(lengths) - 1))
    return cache, batch, q, k, v, tree["mask"].repeat(copies, 1), pos.repeat(copies), one, stored


def check(lengths, nodes, copies, heads, n_kv, d, fmt, window, some, seed=3):
    cache, batch, q, k, v, mask, pos, (q1, k1, v1), (ck, cv) = contents(lengths, nodes, copies, heads, n_kv, d, fmt, seed)
    n, group = len(lengths), heads // n_kv
    y = R.kv_attend_tree(cache, q, k, v, batch, mask, pos=pos if window else None, window=window)
    torch.cuda.synchronize()
    y = y.view(copies, n * nodes, heads, d)
    assert torch.equal(y, y[:1].expand_as(y))
    got, words, pos = y[0].cpu().numpy().astype(np.float64), mask.cpu().numpy().view(np.uint64), pos.cpu().numpy()
    q1, k1, v1 = (t.cpu().numpy().astype(np.float64) for t in (q1, k1, v1))
    for s, ctx in enumerate(lengths):
        for row in sorted({0, nodes - 1, *np.random.default_rng(s).integers(0, nodes, some).tolist()}):
            at = s * nodes + row
            lo = min(ctx, max(0, max(int(pos[at]), ctx) - window + 1)) if window else 0
            take = [s * nodes + j for j in O.bits(words[at], nodes)]
            for h in range(n_kv):
                kk, vv = (np.concatenate([c[lo:ctx, h], x[take, h]]) for c, x in ((ck, k1), (cv, v1)))
                z = q1[at, h * group:(h + 1) * group] @ kk.T * d ** -0.5
                e = np.exp(z - z.max(1, keepdims=True))
                e /= e.sum(1, keepdims=True)
                want, a = e @ vv, e @ np.abs(vv)
                off = np.abs(got[at, h * group:(h + 1) * group] - want) / (2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25)
                assert off.max() <= 1.0, (s, ctx, row, h, off.max())


T = 64


@pytest.mark.parametrize("window", [0, 100 * T + 3])
@pytest.mark.parametrize("fmt,heads,n_kv,d,nodes,copies", [
    ("int8", 8, 2, 128, 32, 100), ("fp8", 8, 2, 64, 32, 100), ("int8", 2, 1, 128, 200, 40), ("fp8", 4, 1, 64, 130, 40),
    ("int8", 4, 1, 256, 70, 24), ("int8", 6, 1, 80, 65, 50)])
def test_whole_contexts(fmt, heads, n_kv, d, nodes, copies, window):
    """More items than run at once: each is one piece, of one to four drafted tiles and cached ones to either side of the
    table's 64 and 128."""
    check([62 * T + 5, 63 * T, 64 * T - 1, 127 * T, 129 * T + 33, 191 * T + 1], nodes, copies, heads, n_kv, d, fmt, window, some=3)


@pytest.mark.parametrize("window", [0, 5000])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_twelve_trees(fmt, window):
    """12 trees of 64 rows of 64 heads, 8 kv, on about 8192 tokens: pieces of up to 129 tiles."""
    check([8192, 8191, 7300], 64, 4, 64, 8, 128, fmt, window, some=2)


def test_several_pieces():
    """Fewer items than run at once: a context in several pieces, each longer than the table, the first behind drafted tiles."""
    check([400 * T + 9, 399 * T], 64, 3, 64, 8, 128, "int8", 0, some=1)
