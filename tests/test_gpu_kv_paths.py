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

from activation_sparse_predictor_amd import runtime as R
from oracle import kv as O
from tests.test_gpu_kv import DEV, filled, host, host_batch, queries, tables

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
