"""pi_kv_attend where its rows go to the prompt kernel (more than 32 rows of a
sequence, and more than 512 tiles of 16 rows over all kv heads), against the
float64 oracle; the bounds are those derived in test_gpu_kv.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import kv as O
from tests.test_gpu_kv import DEV, check_attend, filled, queries

pytestmark = pytest.mark.gpu


def many(new, heads, n_kv):
    """Whether the call's rows reach the prompt kernel."""
    rows = [n * heads // n_kv for n in new]
    each = len(new) * -(-max(rows) // 16)
    return max(rows) > 32 and min(each, sum(rows) // 16 + len(new)) * n_kv > 512


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,page", [(64, 64, 64, 16), (66, 33, 128, 16), (40, 40, 80, 32), (33, 33, 256, 16),
                                               (64, 64, 16, 64), (60, 30, 112, 16), (34, 34, 144, 128), (96, 16, 128, 256)])
@pytest.mark.parametrize("new,ctx", [([130], [130]), ([33, 1, 0, 97, 64], [200, 70, 5, 97, 65]), ([150, 3, 129], [149, 40, 700])])
def test_rows(fmt, heads, n_kv, d, page, new, ctx):
    """Whole prompts, prompts beside single tokens and idle sequences, a row
    before position 0, a prompt on a longer context."""
    if not many(new, heads, n_kv):
        new = [n * 3 if n > 32 else n for n in new]
        ctx = [c * 3 if n > 32 else c for n, c in zip(new, ctx)]
    assert many(new, heads, n_kv)
    cache, rows = filled(ctx, n_kv, d, page, fmt, seed=31)
    check_attend(cache, R.kv_batch(new, ctx, rows, DEV), queries(sum(new), heads, d))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("window", [1, 40, 64, 130, 1000])
@pytest.mark.parametrize("heads,n_kv,d", [(64, 64, 64), (36, 36, 256), (99, 33, 128)])
def test_windows(fmt, window, heads, n_kv, d):
    new, ctx = [160, 40, 2], [160, 300, 90]
    cache, rows = filled(ctx, n_kv, d, 16, fmt, seed=32)
    assert many(new, heads, n_kv)
    check_attend(cache, R.kv_batch(new, ctx, rows, DEV), queries(sum(new), heads, d), window=window)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d", [(8, 8, 64), (10, 5, 128), (9, 9, 256)])
def test_split_over_the_context(fmt, heads, n_kv, d):
    """Row tiles whose keys are split over several workgroups and joined, with and without a window."""
    new, ctx = [1100], [4300]
    cache, rows = filled(ctx, n_kv, d, 64, fmt, seed=33)
    new = [1100 if many([1100], heads, n_kv) else 2100]
    assert many(new, heads, n_kv)
    q = queries(new[0], heads, d)
    batch = R.kv_batch(new, ctx, rows, DEV)
    # the oracle on the first and last rows of every row tile; all rows for equality of repeats
    y = R.kv_attend(cache, q, batch)
    z = R.kv_attend(cache, q, batch, window=3000)
    assert torch.equal(R.kv_attend(cache, q, batch), y) and torch.equal(R.kv_attend(cache, q, batch, window=3000), z)
    host_c = {n: (t.cpu().numpy() if isinstance(t, torch.Tensor) else t) for n, t in cache.items()}
    for i in (0, 1, 63, 64, 127, 128, 500, new[0] - 1):
        pos = ctx[0] - new[0] + i
        one = {"q_start": np.array([0, 1]), "ctx": np.array([pos + 1]), "table": np.array(rows)}
        for got, window in ((y, 0), (z, 3000)):
            want, _, a = O.attend(host_c, one, q[i:i + 1].cpu().numpy(), d ** -0.5, window)
            tol = 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25
            assert np.all(np.abs(got[i:i + 1].cpu().numpy().astype(np.float64) - want) <= tol), i


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_scales_far_apart(fmt):
    def gain(rng, tok):
        return np.where(np.arange(tok) // 16 % 5 == 4, 0.0, 2.0 ** (np.arange(tok) // 16 % 3 * 10 - 14))
    cache, rows = filled([300], 48, 64, 16, fmt, seed=34, v_gain=gain)
    batch = R.kv_batch([180], [300], rows, DEV)
    assert many([180], 48, 48)
    check_attend(cache, batch, queries(180, 48, 64))
    cache, rows = filled([300], 48, 64, 16, fmt, seed=35, v_gain=lambda rng, tok: np.zeros(tok))
    assert not torch.any(check_attend(cache, R.kv_batch([180], [300], rows, DEV), queries(180, 48, 64)))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_ignores_what_is_masked(fmt):
    """NaN codes and scales in slots that no row of a tile attends to change nothing."""
    ctx, page, d, n, kv, window = [245], 16, 64, 150, 64, 40
    cache, rows = filled(ctx, kv, d, page, fmt, seed=36)
    q = queries(n, kv, d)
    assert many([n], kv, kv)
    batch = R.kv_batch([n], ctx, rows, DEV)
    y0 = check_attend(cache, batch, q, window=window)
    first = ctx[0] - n - window + 1
    for s in rows[0][:first // page]:
        for m in ("k", "v"):
            cache[m][s] = 0xFF
            cache[m + "_scale"][s] = float("nan")
    at = O.places(page, d)
    for m, place in zip("kv", at):
        flat = cache[m][rows[0][-1]].view(kv, -1)
        flat[:, torch.from_numpy(place[ctx[0] % page:].reshape(-1)).to(DEV)] = 0x7F
    y1 = R.kv_attend(cache, q, batch, window=window)
    torch.cuda.synchronize()
    assert first >= page and torch.equal(y0, y1)


def test_poisoned_block_and_query_reach_only_their_readers():
    ctx, page, d, n, kv = [200, 50], 16, 64, 150, 64
    cache, rows = filled(ctx, kv, d, page, "int8", seed=37)
    q = queries(n + 1, kv, d)
    assert many([n, 1], kv, kv)
    batch = R.kv_batch([n, 1], ctx, rows, DEV)
    q2 = q.clone()
    q2[70, 3, 5] = float("nan")
    y, y2 = R.kv_attend(cache, q, batch), R.kv_attend(cache, q2, batch)
    torch.cuda.synchronize()
    assert torch.isnan(y2[70, 3]).all()
    y2[70, 3] = y[70, 3]
    assert torch.equal(y, y2)
    cache["v_scale"][rows[0][9], 1] = float("nan")
    cache["k_scale"][rows[0][5], 2] = float("nan")
    check_attend(cache, batch, q, window=33, lse=False)
    rows[0][11] = -1
    check_attend(cache, R.kv_batch([n, 1], ctx, rows, DEV), q, window=20, lse=False)


@pytest.mark.parametrize("n", [1, 150])
def test_scale_signs(n):
    """A negative scale, and a scale of 0 (the mean of what is attended to)."""
    cache, rows = filled([200], 64, 64, 16, "fp8", seed=38)
    batch = R.kv_batch([n], [200], rows, DEV)
    q = queries(n, 64, 64)
    check_attend(cache, batch, q, scale=-0.2)
    check_attend(cache, batch, q, scale=0.0)


def test_offsets_beyond_32_bits():
    n_kv, d, page, n = 64, 64, 16, 150
    n_pages = (1 << 32) // (n_kv * d * page) + 40
    cache = R.kv_cache(n_pages, n_kv, d, page, "int8", DEV)
    ids = [n_pages - 1 - 3 * i for i in range(10)]
    assert ids[-1] * n_kv * d * page > 1 << 32
    k, v = (torch.randn(n, n_kv, d, device=DEV).half() for _ in range(2))
    batch = R.kv_batch([n], [n], [ids], DEV)
    R.kv_append(cache, k, v, batch)
    q = queries(n, 64, d)
    assert many([n], 64, n_kv)
    y = R.kv_attend(cache, q, batch)
    small = {m: (t[ids].contiguous() if isinstance(t, torch.Tensor) else t) for m, t in cache.items()}
    torch.cuda.synchronize()
    del cache
    want = R.kv_attend(small, q, R.kv_batch([n], [n], [list(range(10))], DEV))
    assert torch.equal(y, want)


def test_graph_replay():
    """A mixed call (both kernels) captured and replayed between eager ones."""
    new, ctx = [150, 1, 2], [150, 400, 90]
    cache, rows = filled(ctx, 64, 64, 16, "int8", seed=39)
    batch = R.kv_batch(new, ctx, rows, DEV)
    assert many(new, 64, 64)
    q = queries(sum(new), 64, 64)
    y = torch.empty_like(q)
    ws = R.kv_workspace(3, sum(new), 150, 64, 64, 64, DEV)
    R.kv_attend(cache, q, batch, y=y, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.kv_attend(cache, q, batch, y=y, ws=ws)
    for step in range(4):
        q.copy_(torch.randn_like(q))
        y.fill_(float("nan"))
        graph.replay()
        want = R.kv_attend(cache, q, batch)
        torch.cuda.synchronize()
        assert torch.equal(y, want), step
