"""pi_kv_attend_tree on the GPU against the float64 oracle (oracle/draft.py).

The bound is test_gpu_kv.py's: the drafted rows' products are fp16 x fp16 with
fp32 sums as the cached ones', their weights in two halves under the same
reference, the output rounded once.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O
from tests.test_gpu_kv import DEV, filled, host, host_batch, queries

pytestmark = pytest.mark.gpu


def trees(counts, seed=0):
    rng = np.random.default_rng(seed)
    return [[-1] + [max(0, j - 1 - int(rng.exponential(2.0))) for j in range(1, n)] if n else [] for n in counts]


def drafted(n, n_kv, d, seed=31, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, n_kv, d, generator=g) * gain).half().to(DEV) for _ in range(2)]


def case(counts, ctx, heads, n_kv, d, page, fmt, seed=0, **kw):
    cache, rows = filled(ctx, n_kv, d, page, fmt, seed=seed, **kw)
    batch = R.kv_batch(counts, ctx, [r or [0] for r in rows], DEV)
    t = R.kv_tree(trees(counts, seed), device=DEV)
    pos = (torch.repeat_interleave(batch["ctx"], torch.tensor(counts, device=DEV)) + t["depth"]).to(torch.int32)
    n = sum(counts)
    return cache, batch, t["mask"], pos, queries(n, heads, d, seed + 5), *drafted(n, n_kv, d, seed + 6)


def check(cache, batch, mask, pos, q, k, v, window=0, scale=None, **kw):
    d = q.shape[2]
    sc = d ** -0.5 if scale is None else scale
    lse = torch.full(q.shape[:2], 77.0, device=DEV)
    y = R.kv_attend_tree(cache, q, k, v, batch, mask, pos=pos if window else None, window=window, scale=scale, lse=lse, **kw)
    torch.cuda.synchronize()
    words = mask.cpu().numpy().view(np.uint64)
    want, want_lse, a = O.attend_tree(host(cache), host_batch(batch), q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), words, sc,
                                      window, pos.cpu().numpy())
    got, gl = y.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    tol = 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1.0, f"{worst:.2f} times the bound"
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(gl), none) and np.all(got[none] == 0)
    f = ~none
    assert np.all(np.abs(gl[f] - want_lse[f]) <= 2.0 ** -11 + 2.0 ** -21 * np.abs(want_lse[f]))
    return y


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,page", [(4, 4, 128, 16), (8, 1, 64, 32), (6, 2, 80, 16), (16, 1, 128, 64), (3, 1, 256, 16),
                                               (2, 2, 16, 16), (5, 5, 128, 32), (71, 1, 64, 128), (2, 1, 208, 16)])
@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("counts", [[3, 1, 0, 5, 2, 1], [16, 17, 1, 33, 4, 2], [65, 1, 2, 64, 63, 7]])
def test_trees(fmt, heads, n_kv, d, page, window, counts):
    """Contexts of no token, of one, and around the granule, page and tile ends; trees of one row and up."""
    check(*case(counts, [131, 0, 1, 64, 65, 300], heads, n_kv, d, page, fmt, seed=len(counts)), window=window)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,counts,ctx", [
    (64, 8, 128, [130, 3, 40], [700, 65, 0]), (32, 32, 64, [256, 1], [130, 4]), (24, 8, 256, [200, 64], [1, 257]),
    (16, 16, 80, [129, 130, 1], [64, 0, 63]), (128, 8, 64, [63, 20], [2000, 128])])
@pytest.mark.parametrize("window", [0, 70])
def test_many_rows(fmt, heads, n_kv, d, counts, ctx, window):
    """More 16-row items than the kernel of few rows takes: the prompts' kernel, up to 256 drafted rows."""
    check(*case(counts, ctx, heads, n_kv, d, 16, fmt, seed=d), window=window)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,counts", [(1, 1, 128, [1, 7, 3]), (8, 2, 64, [20, 1, 66]), (64, 8, 128, [100, 1, 70]), (2, 1, 256, [9, 2, 2])])
def test_long_contexts(fmt, heads, n_kv, d, counts):
    """Split over many workgroups and joined; the drafted rows are in one of the pieces."""
    c = case(counts, [9001, 40, 4096], heads, n_kv, d, 64, fmt, seed=8)
    check(*c)
    check(*c, window=3000)


@pytest.mark.parametrize("heads,n_kv,counts", [(4, 2, [20, 70, 3, 9]), (32, 16, [200, 90, 40, 1])])
def test_any_masks(heads, n_kv, counts):
    """Masks that are no trees: rows that see nothing drafted, rows that see nothing at all, bits behind the last
    row, words behind the last tile."""
    cache, batch, mask, pos, q, k, v = case(counts, [100, 0, 0, 33], heads, n_kv, 64, 16, "int8", seed=9)
    g = torch.Generator().manual_seed(1)
    n, words = sum(counts), 4
    mask = torch.randint(-2 ** 62, 2 ** 62, (n, words), generator=g)
    mask[::3] = 0
    mask[1::5] = -1
    check(cache, batch, mask.to(DEV), pos, q, k, v)
    check(cache, batch, mask.to(DEV), pos, q, k, v, window=5)
    check(cache, batch, torch.zeros_like(mask).to(DEV), pos, q, k, v, window=1)


@pytest.mark.parametrize("n,heads,n_kv", [(9, 4, 2), (70, 4, 2), (100, 64, 16)])
def test_positions_and_windows_at_their_ends(n, heads, n_kv):
    """Positions before the context count as its end, far ones leave only the mask's rows; the widest windows are none."""
    cache, batch, mask, pos, q, k, v = case([n], [200], heads, n_kv, 64, 16, "fp8", seed=10)
    y0 = check(cache, batch, mask, pos, q, k, v)
    for window in (2 ** 31 - 1, 200 + n):
        assert torch.equal(check(cache, batch, mask, pos, q, k, v, window=window), y0)
    odd = pos.clone()
    odd[::2] = -5
    odd[1::4] = 2 ** 31 - 1
    check(cache, batch, mask, odd, q, k, v, window=60)
    check(cache, batch, mask, odd, q, k, v, window=2 ** 30 + 7)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("n,heads,n_kv", [(5, 4, 2), (80, 4, 2), (100, 64, 16)])
def test_scales_far_apart(fmt, n, heads, n_kv):
    """Cached blocks 2^20 apart and of zeros beside drafted values of 1, of 2^-12 and of 2^10."""
    def gain(rng, tok):
        return np.where(np.arange(tok) // 16 % 5 == 4, 0.0, 2.0 ** (np.arange(tok) // 16 % 3 * 10 - 14))
    cache, batch, mask, pos, q, k, v = case([n], [400], heads, n_kv, 64, 16, fmt, seed=11, v_gain=gain)
    for g in (1.0, 2.0 ** -12, 2.0 ** 10, 0.0):
        check(cache, batch, mask, pos, q, k, v * g)
    check(cache, batch, mask, pos, q * 8, k, v, scale=0.0625)
    check(cache, batch, mask, pos, q, k, v, scale=-0.125)


@pytest.mark.parametrize("d", [64, 80, 128, 256])
@pytest.mark.parametrize("n,heads,n_kv", [(6, 4, 2), (70, 4, 2), (100, 64, 16)])
def test_what_is_masked_may_hold_anything(n, heads, n_kv, d):
    """NaN and infinities in a drafted row change nothing, bit for bit, for rows that do not attend to it, and make
    NaN of the heads that do."""
    cache, batch, mask, pos, q, k, v = case([n], [70], heads, n_kv, d, 16, "int8", seed=12)
    y0 = check(cache, batch, mask, pos, q, k, v)
    sick = n // 2
    bits = mask.cpu().numpy().view(np.uint64)
    sees = torch.tensor([bool(int(bits[r, sick // 64]) >> (sick % 64) & 1) for r in range(n)], device=DEV)
    assert sees.any() and not sees.all()
    for value in (float("nan"), float("inf"), -float("inf")):
        for which in ("k", "v"):
            for dim in (0, d - 1):
                k2, v2 = k.clone(), v.clone()
                (k2 if which == "k" else v2)[sick, 1, dim] = value
                y = R.kv_attend_tree(cache, q, k2, v2, batch, mask)
                mine = torch.zeros(n, heads, dtype=torch.bool, device=DEV)
                mine[:, heads // n_kv:2 * (heads // n_kv)] = sees[:, None]
                assert torch.equal(y[~mine], y0[~mine])
                if which == "v" or value != value:
                    assert torch.isnan(y[mine]).all()
    # all the garbage at once, in a row that nobody attends to
    gone = mask.clone()
    gone[:, sick // 64] &= ~torch.tensor(1 << (sick % 64) if sick % 64 < 63 else -2 ** 63, dtype=torch.int64)
    y1 = check(cache, batch, gone, pos, q, k, v)
    k[sick], v[sick] = float("nan"), float("inf")
    assert torch.equal(R.kv_attend_tree(cache, q, k, v, batch, gone), y1)


@pytest.mark.parametrize("n,heads,n_kv", [(6, 4, 2), (70, 4, 2), (100, 64, 16)])
def test_a_query_that_is_not_finite_is_its_own(n, heads, n_kv):
    cache, batch, mask, pos, q, k, v = case([n], [70], heads, n_kv, 64, 16, "int8", seed=13)
    y0 = R.kv_attend_tree(cache, q, k, v, batch, mask)
    q[n // 2, 1, 7] = float("nan")
    y = R.kv_attend_tree(cache, q, k, v, batch, mask)
    assert torch.isnan(y[n // 2, 1]).all()
    y[n // 2, 1] = y0[n // 2, 1]
    assert torch.equal(y, y0)


@pytest.mark.parametrize("counts,heads,n_kv", [([3, 1, 9], 4, 2), ([70, 1, 20], 4, 2), ([100, 1, 70], 64, 8)])
def test_repeats_bitwise_with_strides_and_own_buffers(counts, heads, n_kv):
    d = 128
    cache, batch, mask, pos, q, k, v = case(counts, [3000, 17, 400], heads, n_kv, d, 16, "fp8", seed=14)
    y0 = check(cache, batch, mask, pos, q, k, v)
    n = sum(counts)
    wide = torch.cat([t.reshape(n, -1) for t in (q, k, v)], 1)
    ws_, (qs, ks, vs) = R.kv_workspace(3, n, max(counts), heads, n_kv, d, DEV), (
        t.unflatten(1, (-1, d)) for t in wide.split([heads * d, n_kv * d, n_kv * d], 1))
    y = torch.full_like(y0, float("nan"))
    for _ in range(3):
        assert R.kv_attend_tree(cache, qs, ks, vs, batch, mask, y=y, ws=ws_) is y
        torch.cuda.synchronize()
        assert torch.equal(y, y0)
    # the same workspace serves attention without drafted rows
    plain = R.kv_batch([1, 1, 1], [3000, 17, 400], batch["table"].tolist(), DEV)
    want = R.kv_attend(cache, q[:3].contiguous(), plain)
    assert torch.equal(R.kv_attend(cache, q[:3].contiguous(), plain, ws=ws_), want)
    assert torch.equal(R.kv_attend_tree(cache, q, k, v, batch, mask, ws=ws_), y0)


def test_rows_of_no_sequence_are_left_and_broken_ranges_stay_inside():
    counts = [5, 3]
    cache, batch, mask, pos, q, k, v = case(counts, [40, 33], 4, 2, 64, 16, "int8", seed=15)
    y0 = R.kv_attend_tree(cache, q, k, v, batch, mask)
    short = dict(batch, q_start=torch.tensor([0, 5, 5], dtype=torch.int32, device=DEV))
    y = torch.full_like(y0, 3.0)
    R.kv_attend_tree(cache, q, k, v, short, mask, y=y)
    assert torch.equal(y[:5], y0[:5]) and torch.all(y[5:] == 3.0)
    wild = dict(batch, q_start=torch.tensor([-7, 5, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    assert torch.equal(R.kv_attend_tree(cache, q, k, v, wild, mask), y0)
    wild = dict(batch, ctx=torch.tensor([-2 ** 31, 33], dtype=torch.int32, device=DEV))
    y = R.kv_attend_tree(cache, q, k, v, wild, mask)
    assert torch.equal(y[5:], y0[5:])


@pytest.mark.parametrize("heads,n_kv", [(4, 2), (64, 16)])
def test_more_rows_than_the_mask_has_stay_inside(heads, n_kv):
    """Row ranges on the device that exceed max_q and the mask: those rows are unspecified, others are not touched."""
    n, d = 400, 64
    cache, rows = filled([5000, 33], n_kv, d, 16, "int8", seed=21)
    q, (k, v) = queries(n, heads, d), drafted(n, n_kv, d)
    batch = R.kv_batch([64, 3], [5000, 33], rows, DEV)
    batch.update(n_tok=n, max_q=64, q_start=torch.tensor([0, 397, 400], dtype=torch.int32, device=DEV))
    mask = torch.full((n, 1), 7, dtype=torch.int64, device=DEV)
    y = torch.full((n + 8, heads, d), 5.0, dtype=torch.float16, device=DEV)
    R.kv_attend_tree(cache, q, k, v, batch, mask, y=y[:n])
    torch.cuda.synchronize()
    assert torch.all(y[n:] == 5.0)
    # (the split of the work, and with it the order of the sums, is the whole batch's: within the bound, not bit for bit)
    want, _, a = O.attend_tree(host(cache), {"q_start": [0, 3], "ctx": [33], "table": [rows[1]]},
                               *(t[397:].cpu().numpy() for t in (q, k, v)), np.full((3, 1), 7, np.uint64), d ** -0.5)
    assert np.all(np.abs(y[397:400].cpu().numpy() - want) <= 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25)


def test_a_page_that_does_not_exist_is_its_readers():
    cache, batch, mask, pos, q, k, v = case([5, 3], [40, 33], 4, 2, 64, 16, "int8", seed=16)
    y0 = R.kv_attend_tree(cache, q, k, v, batch, mask)
    for bad in (-1, 10 ** 6):
        table = batch["table"].clone()
        table[0, 0] = bad
        y = R.kv_attend_tree(cache, q, k, v, dict(batch, table=table), mask)
        assert torch.isnan(y[:5]).all() and torch.equal(y[5:], y0[5:])
        y = R.kv_attend_tree(cache, q, k, v, dict(batch, table=table), mask, pos=pos, window=20)
        assert torch.isfinite(y).all()


def test_many_sequences():
    rng = np.random.default_rng(20)
    counts = [int(x) for x in rng.integers(0, 6, 150)]
    ctx = [int(x) for x in rng.integers(0, 60, 150)]
    check(*case(counts, ctx, 2, 1, 64, 16, "int8", seed=17))


def test_another_stream_and_captured_graphs():
    """Lengths, masks and rows that change between the replays; two graphs, with and without a workspace of their own."""
    small, large = case([7, 1, 9], [800, 0, 65], 8, 2, 128, 16, "int8", seed=18), case([100, 70], [300, 900], 64, 8, 64, 32, "fp8", seed=19)
    graphs = []
    for (cache, batch, mask, pos, q, k, v), ws in ((small, None), (large, None), (small, R.kv_workspace(3, 17, 9, 8, 2, 128, DEV))):
        want = R.kv_attend_tree(cache, q, k, v, batch, mask)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        y = R.kv_attend_tree(cache, q, k, v, batch, mask, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = R.kv_attend_tree(cache, q, k, v, batch, mask, pos=pos, window=500, ws=ws)
        graphs.append((graph, y, (cache, batch, mask, pos, q, k, v)))
    for turn in range(3):
        for graph, y, (cache, batch, mask, pos, q, k, v) in graphs[::-1] if turn % 2 else graphs:
            q.copy_(torch.randn_like(q))
            v.copy_(torch.randn_like(v))
            batch["ctx"] -= batch["ctx"].clamp(max=1)
            pos -= 1
            y.fill_(float("nan"))
            graph.replay()
            got = y.clone()
            torch.cuda.synchronize()
            assert torch.equal(got, R.kv_attend_tree(cache, q, k, v, batch, mask, pos=pos, window=500))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,counts,ctx", [(2, 1, 64, [200, 3], [9000, 30]), (1, 1, 128, [256], [20000]), (1, 1, 256, [250, 70], [700, 5000]),
                                                     (2, 2, 128, [129], [400]), (1, 1, 64, [256, 1], [0, 64])])
def test_several_drafted_tiles_beside_cached_ones(fmt, heads, n_kv, d, counts, ctx):
    """The kernel of few items: up to all waves of a workgroup have a drafted tile, the others share the cached ones meanwhile."""
    c = case(counts, ctx, heads, n_kv, d, 32, fmt, seed=d + counts[0])
    check(*c)
    check(*c, window=260)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,n", [(64, 8, 128, 4), (64, 32, 64, 16), (16, 8, 256, 16), (64, 8, 128, 5)])
def test_many_sequences_of_two_items(fmt, heads, n_kv, d, n):
    """More 16-row items than the kernel of few rows takes for chains, on either side of 32 rows a kv head."""
    rng = np.random.default_rng(d)
    counts = [n] + [int(x) for x in rng.integers(0, n + 1, 39)]
    ctx = [int(x) for x in rng.integers(0, 300, 40)]
    c = case(counts, ctx, heads, n_kv, d, 16, fmt, seed=n)
    check(*c)
    check(*c, window=100)
