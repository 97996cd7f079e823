"""Turned keys beyond fp16's largest number: codes and scale hold them, attention takes them as they are, the
read back gives infinity."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import kv as KV
from tests.test_gpu_kv import DEV, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_keys_beyond_fp16(fmt, layout):
    d, n = 64, 20
    rng = np.random.default_rng(4)
    k = torch.from_numpy((rng.choice([-1.0, 1.0], (n, 1, d)) * rng.uniform(3e4, 6e4, (n, 1, d))).astype(np.float16)).to(DEV)
    v = torch.from_numpy(rng.standard_normal((n, 1, d)).astype(np.float16)).to(DEV)
    q = torch.from_numpy((rng.standard_normal((1, 1, d)) * 2.0 ** -9).astype(np.float16)).to(DEV)
    cache = R.kv_cache(2, 1, d, 16, fmt)
    batch = R.kv_batch([n], [n], [[1, 0]])
    R.kv_append_rope(cache, k, v, batch, R.rope(d, layout=layout, gain=4.0, freqs=np.linspace(0.1, 3.0, d // 2)))
    y = R.kv_attend(cache, q, R.kv_batch([1], [n], [[1, 0]]), scale=2.0 ** -10)
    back, _ = R.kv_read(cache, batch)
    torch.cuda.synchronize()
    kept = host(cache)
    kk, vv = (np.stack([KV.stored(kept, [1, 0], j, name)[0] for j in range(n)]) for name in "kv")
    assert np.abs(kk).max() > 2e5
    far = np.abs(kk) >= 65520.0   # rounds to infinity
    got = back.cpu().numpy()[:, 0]
    assert far.any() and np.array_equal(np.isinf(got), far) and np.array_equal(np.sign(got[far]), np.sign(kk[far]))
    x = kk @ q.cpu().numpy()[0, 0].astype(np.float64) * 2.0 ** -10
    e = np.exp(x - x.max())
    e /= e.sum()
    want, a = e @ vv, e @ np.abs(vv)
    assert 1e-3 < e.max() < 0.999
    off = np.abs(y.cpu().numpy()[0, 0] - want) / (2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25)
    assert off.max() <= 1.0
