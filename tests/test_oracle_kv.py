"""Pins for the cache oracle (run without a GPU): formats against torch's and
hand-worked values, byte order against the written formulas, the block rules
on hand-worked blocks, attention against closed forms."""

import math

import numpy as np
import pytest
import torch

from oracle import kv as O


def test_e4m3_values_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_values(), want, equal_nan=True)


def test_encode_fp8_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * np.exp2(rng.integers(-12, 8, 20000)),
                        O.e4m3_values()[:127], (O.e4m3_values()[:126] + O.e4m3_values()[1:127]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.encode(x, "fp8"), want)


def test_encode_int8_ties_to_even_and_clamps():
    assert O.encode([0.5, 1.5, -0.5, -2.5, 127.4, 300, -300], "int8").tolist() == [128, 130, 128, 126, 255, 255, 1]


def test_places_cover_a_page_once():
    for page, d in ((16, 16), (32, 80), (64, 128)):
        for at in O.places(page, d):
            assert sorted(at.reshape(-1)) == list(range(page * d))
    k, v = O.places(32, 64)
    assert k[5, 18] == 1 * 256 + 1 * 64 + 1 * 16 + 2 and v[17, 3] == 16 * 64 + 3 * 16 + 1


def _cache(fmt, n_pages=2, n_kv=1, page=16, d=16):
    return {"fmt": fmt, "k": np.full((n_pages, n_kv, page, d), 7, np.uint8), "v": np.full((n_pages, n_kv, page, d), 7, np.uint8),
            "k_scale": np.full((n_pages, n_kv), 5, np.float32), "v_scale": np.full((n_pages, n_kv), 5, np.float32)}


def _batch(n, ctx, table):
    return {"q_start": np.concatenate([[0], np.cumsum(n)]), "ctx": np.array(ctx), "table": np.array(table)}


def test_append_by_hand():
    """A first token with largest value 1.27 (scale 0.01), a second with 2.54: the
    scale doubles, the first token's codes halve (63.5 to the even 64), and a smaller third keeps it."""
    c = _cache("int8")
    x = np.zeros((1, 1, 16), np.float32)
    x[0, 0, :3] = [1.27, -0.02, 0.63]
    c = O.append(c, _batch([1], [1], [[1]]), x, x)
    assert c["k_scale"][1, 0] == np.float32(1.27) / np.float32(127)
    assert O.stored(c, [1], 0, "k")[0, :3] == pytest.approx([1.27, -0.02, 0.63], abs=1e-6)
    assert np.all(c["k"][0] == 7) and np.all(c["k"][1, 0].reshape(-1)[O.places(16, 16)[0][1:]] == 7)
    z = np.zeros((1, 1, 16), np.float32)
    z[0, 0, 0] = -2.54
    c = O.append(c, _batch([1], [2], [[1]]), z, z)
    at = O.places(16, 16)[0]
    assert O.decode(c["k"][1, 0].reshape(-1)[at[0, :3]], "int8").tolist() == [64.0, -1.0, 32.0]
    assert c["k_scale"][1, 0] == np.float32(2.54) / np.float32(127)
    s = c["k_scale"][1, 0]
    c = O.append(c, _batch([1], [3], [[1]]), x, x)
    assert c["k_scale"][1, 0] == s and O.decode(c["k"][1, 0].reshape(-1)[at[2, 0]], "int8") == 64


def test_append_zeros_nonfinite_and_places():
    for fmt in ("int8", "fp8"):
        c = _cache(fmt)
        z = np.zeros((3, 1, 16), np.float32)
        d = O.append(c, _batch([1, 2], [0, 1], [[0], [1]]), z, z)   # rows before position 0 have no place
        assert np.all(d["k"][0] == c["k"][0]) and d["k_scale"][0, 0] == 5 and d["k_scale"][1, 0] == 0
        assert np.all(O.stored(d, [1], 0, "v") == 0)
        z[2, 0, 3] = np.inf
        e = O.append(d, _batch([1, 2], [0, 3], [[0], [1]]), z, z)
        assert np.isnan(e["v_scale"][1, 0]) and np.all(np.isnan(O.stored(e, [1], 0, "v")))
        z[:] = 1
        e = O.append(e, _batch([0, 1], [0, 4], [[0], [1]]), z, z)
        assert np.isnan(e["v_scale"][1, 0])
        e = O.append(e, _batch([0, 3], [0, 3], [[0], [1]]), z, z)   # from the first token again
        assert e["v_scale"][1, 0] == np.float32(1) / np.float32(O.QMAX[fmt])
        f = O.append(e, _batch([0, 1], [0, 1], [[0], [9]]), z, z)
        assert np.array_equal(f["k"], e["k"])


def test_attend_closed_forms():
    """Equal keys give the mean of the values; one far larger key gives its
    value; a window cuts; a negative position gives 0 and -infinity."""
    c = _cache("int8", page=16)
    k = np.ones((5, 1, 16), np.float32)
    v = np.arange(5, dtype=np.float32)[:, None, None] * np.ones((1, 1, 16), np.float32)
    c = O.append(c, _batch([5], [5], [[0]]), k, v)
    vals = np.stack([O.stored(c, [0], j, "v")[0] for j in range(5)])
    q = np.ones((2, 2, 16), np.float32)
    y, lse, a = O.attend(c, _batch([2], [5], [[0]]), q, 0.25)
    assert np.allclose(y[1, 0], vals.mean(0)) and np.allclose(y[0, 1], vals[:4].mean(0)) and np.allclose(a, y)
    assert lse[1, 0] == pytest.approx(4.0 + math.log(5), abs=1e-6)
    y, _, _ = O.attend(c, _batch([2], [5], [[0]]), q, 0.25, window=2)
    assert np.allclose(y[1, 0], vals[3:].mean(0))
    y, lse, _ = O.attend(c, _batch([2], [1], [[0]]), q, 0.25)
    assert np.all(y[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(y[1], vals[0])
    k[2] = 50
    c = O.append(_cache("fp8"), _batch([5], [5], [[0]]), k, v)
    y, _, _ = O.attend(c, _batch([1], [5], [[0]]), q[:1], 1.0)
    assert np.allclose(y[0, 0], O.stored(c, [0], 2, "v")[0])
