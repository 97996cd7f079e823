"""pi_kv_attend on both sides of the rule that picks its kernel (attend.hip,
uses_prompt), and what holds on either side alike.

Tiny differences of weights.  Rows that attend to a few keys whose values are
+b and -b, b the largest code times the scale: y = sum +-w / sum w * b lies far
below A = b, so an error of a weight stands beside y's own rounding and not
under it.  Queries are -1, 0 or 1 and the scores small: sum |q k| scale log2(e)
is at most 4, |x2| = |x log2(e)| at most 8.
  scores     exact for whole codes; for e4m3 codes at most 8 chained fp32 sums
             of numbers up to 4, each off by 2^-23 of them: 2^-18
  exponent   x2 + log2 vs - M + lift: the factor ks scale log2(e) off by
             3 2^-24, log2 vs by 2^-21, and three fp32 roundings of numbers under
             32 (2^-20 each): together under 2^-18
  weights    an exponent off by 2^-17 is a factor of 1 + 2^-17.5; two fp16
             halves, exp2, the sums and the quotient add under 2^-18.5
An error e of every weight is 2 e A in y: under 2^-16 A, beside y's rounding to
fp16 (2^-11 |y|, 2^-25 below its normal range).  Weights rounded to fp16 once
would be off by up to 2^-11 A.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R
from oracle import kv as O
from tests.test_gpu_kv import DEV, check_attend, filled, host, host_batch, queries, tables

pytestmark = pytest.mark.gpu


def items(new, heads, n_kv):
    """16-row items that the call's sizes allow for, over all kv heads."""
    g = heads // n_kv
    return min(len(new) * -(-max(new) * g // 16), sum(new) * g // 16 + len(new)) * n_kv


def to_prompt(new, heads, n_kv):
    return max(new) * heads // n_kv > 16 and items(new, heads, n_kv) > 384


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("window", [2, 5])
@pytest.mark.parametrize("heads,n_kv,d,new", [(64, 64, 64, 160), (40, 40, 80, 200), (40, 40, 128, 200), (40, 40, 112, 200), (36, 36, 256, 200),
                                              (36, 36, 208, 200), (4, 2, 128, 90), (3, 3, 64, 1), (2, 1, 256, 20)])
def test_weights_are_not_rounded_once(fmt, window, heads, n_kv, d, new):
    rng = np.random.default_rng(d + new)
    ctx, page = 200, 16
    rows, n_pages = tables([ctx], page, rng)
    cache = R.kv_cache(n_pages, n_kv, d, page, fmt, DEV)
    k = torch.from_numpy(rng.standard_normal((ctx, n_kv, d)).astype(np.float16)).to(DEV)
    v = torch.ones(ctx, n_kv, d, dtype=torch.float16, device=DEV)
    v[1::2] = -1
    R.kv_append(cache, k, v, R.kv_batch([ctx], [ctx], rows, DEV))
    q = torch.from_numpy(rng.integers(-1, 2, (new, heads, d)).astype(np.float16)).to(DEV)
    scale = 0.25 / d ** 0.5
    batch = R.kv_batch([new], [ctx], rows, DEV)
    y = R.kv_attend(cache, q, batch, scale=scale, window=window)
    torch.cuda.synchronize()
    H = host(cache)
    kk = np.stack([O.stored(H, rows[0], j, "k") for j in range(ctx)])   # [keys, n_kv, d]
    x2 = np.matmul(q.cpu().numpy().astype(np.float64).reshape(new, n_kv, -1, d).transpose(1, 0, 2, 3).reshape(n_kv, -1, d),
                   kk.transpose(1, 2, 0)) * scale * 1.4427
    assert np.max(np.abs(x2)) < 8 and np.max(np.abs(kk).sum(-1)) * scale * 1.4427 < 8   # (of q's signs a third are 0)
    want, _, a = O.attend(H, host_batch(batch), q.cpu().numpy(), scale, window)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -16 * a + 2.0 ** -25
    worst = np.max(np.abs(y.cpu().numpy().astype(np.float64) - want) / tol)
    assert worst <= 1.0, f"{worst:.2f} times the bound"


@pytest.mark.parametrize("heads,n_kv,d,new,split", [(8, 8, 64, 1100, True), (10, 5, 128, 2100, True), (4, 4, 256, 1600, True),
                                                   (9, 9, 256, 1100, False)])
def test_a_join_that_waits_in_vain_ends_in_nan(heads, n_kv, d, new, split):
    """The prompt kernel's join waits for a count of pieces.  Set to one too few
    from outside (which the workspace rules forbid), the bounded wait runs out:
    the joined rows are NaN, the others (all, where the items fill the GPU by
    themselves and none is split) as before, and the next call is right again."""
    ctx = [4300]
    assert to_prompt([new], heads, n_kv)
    cache, rows = filled(ctx, n_kv, d, 64, "int8", seed=41)
    q, batch = queries(new, heads, d), R.kv_batch([new], ctx, rows, DEV)
    ws = R.kv_workspace(1, new, new, heads, n_kv, d, DEV)
    lse = torch.empty(new, heads, device=DEV)
    want = R.kv_attend(cache, q, batch, ws=ws)
    torch.cuda.synchronize()
    counters = ws[8192:8192 + 65536].view(torch.int32).view(1024, 16)
    assert not torch.any(counters)
    counters[:, 1] = -1
    y = R.kv_attend(cache, q, batch, ws=ws, lse=lse)
    torch.cuda.synchronize()
    lost = torch.isnan(y).any(2)
    assert bool(torch.any(lost)) == split and torch.equal(torch.isnan(y).all(2), lost) and torch.equal(torch.isnan(lse), lost)
    assert torch.equal(y[~lost], want[~lost])
    assert torch.equal(R.kv_attend(cache, q, batch, ws=ws), want)


def prompt_chosen(new, heads, n_kv, d):
    """Which kernel the library's own rule picks, read off the workspace it asks
    for (1024 pieces of the prompt kernel's rows, or of 16)."""
    kj = 1 if d <= 64 else 2 if d <= 128 else 4
    size = B.pi_kv_workspace_size(len(new), sum(new), max(new), heads, n_kv, d) - B.PI_KV_WS_ZERO_BYTES
    rows = size / (1024 * (64 * kj + 2) * 4)
    assert rows in (16, 64 if kj == 4 else 128)
    return rows > 16


SIDES = [
    # most rows a sequence 16 and 17
    ([16] * 13, 32, 32, False), ([17] * 13, 32, 32, True), ([4] * 13, 128, 32, False), ([5] + [4] * 12, 128, 32, True),
    # 16-row items 384 and more
    ([96], 64, 64, False), ([96], 65, 65, True), ([97], 55, 55, True), ([20] * 12, 16, 16, False), ([20] * 13, 16, 16, True),
    ([30, 1, 7] * 5, 8, 4, False), ([30, 1, 7] * 5, 64, 32, True),
    # one token a sequence, more than 16 query heads a kv head
    ([1] * 76, 71, 1, False), ([1] * 77, 71, 1, True), ([1] * 96, 34, 2, False), ([1] * 97, 34, 2, True),
]


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("d", [64, 80, 128, 256])
@pytest.mark.parametrize("window", [0, 21])
@pytest.mark.parametrize("new,heads,n_kv,prompt", SIDES)
def test_both_sides_of_the_rule(fmt, d, window, new, heads, n_kv, prompt):
    """Calls just on either side of the rule, against the oracle: ragged contexts,
    some shorter than the call's rows."""
    assert to_prompt(new, heads, n_kv) == prompt == prompt_chosen(new, heads, n_kv, d)
    ctx = [(37 * i) % 150 if i % 5 else n + 90 for i, n in enumerate(new)]
    cache, rows = filled(ctx, n_kv, d, 16, fmt, seed=42)
    check_attend(cache, R.kv_batch(new, ctx, [r or [0] for r in rows], DEV), queries(sum(new), heads, d), window=window)


def near(cache, rows, ctx, new, q, y, picks, row0=0, window=0):
    """Rows `picks` of a sequence's new rows against the oracle."""
    H = host(cache)
    for i in picks:
        one = {"q_start": np.array([0, 1]), "ctx": np.array([ctx - new + i + 1]), "table": np.array([rows])}
        want, _, a = O.attend(H, one, q[row0 + i:row0 + i + 1].cpu().numpy(), q.shape[2] ** -0.5, window)
        tol = 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25
        assert np.all(np.abs(y[row0 + i:row0 + i + 1].cpu().numpy().astype(np.float64) - want) <= tol), i


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("window", [0, 700])
def test_wide_heads_split_over_the_context(fmt, window):
    """Heads of 256 and 240 in the prompt kernel with its row tiles' keys split and joined."""
    for d in (256, 240):
        ctx, new, heads = 4300, 1600, 4
        cache, rows = filled([ctx], heads, d, 64, fmt, seed=43)
        q = queries(new, heads, d)
        assert prompt_chosen([new], heads, heads, d)
        y = R.kv_attend(cache, q, R.kv_batch([new], [ctx], rows, DEV), window=window)
        near(cache, rows[0], ctx, new, q, y, (0, 63, 64, 801, new - 1), window=window)


def test_more_items_than_the_grid_is_high():
    """1024 sequences of 600 rows, 16 query heads on one kv head: 76800 row tiles of
    a head, above the 65535 workgroups a grid has in that direction."""
    n_seq, n, heads, d = 1024, 600, 16, 16
    assert n_seq * n * heads // 128 > 65535
    # two sequences' pages, named by all the others in turn
    cache, rows = filled([n, n], 1, d, 16, "int8", seed=44)
    batch = R.kv_batch([n] * n_seq, [n] * n_seq, [rows[s % 2] for s in range(n_seq)], DEV)
    q = torch.randn(n_seq * n, heads, d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).half()
    y = torch.full_like(q, float("nan"))
    R.kv_attend(cache, q, batch, y=y)
    assert not torch.isnan(y).any()
    for s in (0, 511, 1022, 1023):
        near(cache, rows[s % 2], n, n, q, y, (0, 7, 8, 300, n - 1), row0=s * n)


def test_row_ranges_that_overlap_leave_the_counters_at_zero():
    """More rows on the device than the host's sizes allow for: every unit still
    runs and ends, and a sound call on the same workspace afterwards is right."""
    n_kv, d = 512, 16
    ctx = [900, 900, 40]
    cache, rows = filled(ctx, n_kv, d, 16, "int8", seed=45)
    good = R.kv_batch([2, 1, 1], ctx, rows, DEV)
    q = queries(4, 2 * n_kv, d)
    ws = R.kv_workspace(3, 4, 2, q.shape[1], n_kv, d, DEV)
    want = R.kv_attend(cache, q, good, ws=ws)
    bad = dict(good, q_start=torch.tensor([0, 4, 0, 4], dtype=torch.int32, device=DEV))
    R.kv_attend(cache, q, bad, ws=ws)
    torch.cuda.synchronize()
    assert not torch.any(ws[8192:B.PI_KV_WS_ZERO_BYTES])
    assert torch.equal(R.kv_attend(cache, q, good, ws=ws), want)
