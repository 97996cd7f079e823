"""What the example's decoder layer stores: every code of every token so far,
against the oracle's append of the layer's own k and v (strided slices of one
projection)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from examples.decode_layer import Layer
from oracle import kv as O
from synthetic import CONFIGS, make_tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv", [(4, 4), (4, 2), (16, 1)])
def test_codes_of_the_layers_own_keys_and_values(fmt, heads, n_kv):
    cfg = CONFIGS["c1"]
    layer = Layer(cfg, heads, n_kv, 64, 3, fmt)
    d, page = layer.d, layer.page
    host = {n: (t.cpu().numpy() if isinstance(t, torch.Tensor) else t) for n, t in layer.cache.items()}
    x = make_tokens(cfg, 40).to("cuda")
    for new in ([17, 1, 6], [1, 1, 1], [1, 0, 16], [1, 30, 1]):
        x = x[:sum(new)].contiguous()
        before = list(layer.lengths)
        qkv = (x @ layer.w_qkv.t()).cpu().numpy()
        _, k, v = (a.reshape(len(x), -1, d) for a in np.split(qkv, [heads * d, (heads + n_kv) * d], 1))
        batch = {"q_start": np.concatenate([[0], np.cumsum(new)]), "ctx": np.array(before) + new, "table": np.array(layer.table)}
        host = O.append(host, batch, k, v)
        layer.step(x, new)
        got = {n: (t.cpu().numpy() if isinstance(t, torch.Tensor) else t) for n, t in layer.cache.items()}
        for m, at in zip("kv", O.places(page, d)):
            for s, n in enumerate(batch["ctx"]):
                for p0 in range(0, int(n), page):
                    pid, used = layer.table[s][p0 // page], at[:min(page, int(n) - p0)]
                    a, b = (O.decode(c[m][pid].reshape(n_kv, -1)[:, used], fmt) for c in (got, host))
                    assert np.array_equal(a, b) and np.array_equal(got[m + "_scale"][pid], host[m + "_scale"][pid]), (m, s, p0)
        x = make_tokens(cfg, 40).to("cuda")
