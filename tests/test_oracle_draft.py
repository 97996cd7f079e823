"""Pins for the oracle of rotary positions and speculative decoding (run
without a GPU): complex numbers, closed forms, and the property that makes
verification what it is: what comes out is distributed as the target says."""

import itertools
import math

import numpy as np
import pytest

from oracle import draft as O
from oracle import kv as K


def test_rotation_is_a_product_of_complex_numbers():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 12))
    f = np.array([1.0, 0.3, 0.01, 2.5])
    for layout, a, b in (("half", slice(0, 4), slice(4, 8)), ("pairs", slice(0, 8, 2), slice(1, 8, 2))):
        y = O.rotate(x, [0, 5, -7], f, layout, 1.5)
        z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * np.array([0, 5, -7])[:, None, None] * f)
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag) and np.array_equal(y[..., 8:], x[..., 8:])


def test_scores_depend_on_distances():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f, _ = O.frequencies(16)
    dots = [float(np.sum(O.rotate(q, [i + 3], f) * O.rotate(k, [i], f))) for i in (0, 10, 1000)]
    assert np.allclose(dots, dots[0])


def test_frequencies():
    own, one = O.frequencies(64)
    assert own[0] == 1 and own[16] == pytest.approx(10000 ** -0.5) and one == 1
    assert np.allclose(O.frequencies(64, scaling="linear", factor=4)[0], own / 4)
    ntk = O.frequencies(64, scaling="ntk", factor=8)[0]
    assert ntk[0] == 1 and ntk[-1] == pytest.approx(own[-1] / 8)
    assert O.frequencies(2, scaling="ntk", factor=8)[0].tolist() == [1.0]
    y, gain = O.frequencies(64, scaling="yarn", factor=8, trained=4096, slow=1, fast=32)
    n = 4096 * own / (2 * math.pi)
    assert np.allclose(y[n >= 32], own[n >= 32]) and np.allclose(y[n <= 1], own[n <= 1] / 8) and gain == pytest.approx(0.1 * math.log(8) + 1)
    mid = (n > 1) & (n < 32)
    assert mid.any() and np.all(y[mid] < own[mid]) and np.all(y[mid] > own[mid] / 8)


def first_token(p, q, drafts):
    """Distribution of the token after the root when its children are `drafts`, by the oracle's steps."""
    out, reach, P = np.zeros(len(p)), 1.0, p.copy()
    for x in drafts:
        keep = min(1.0, P[x] / (1.0 if q is None else q[x]))
        # the threshold in u is where the oracle says it is
        for u in (keep * 0.999, min(keep * 1.001, 1 - 1e-9)):
            assert O.stays(P, q, x, u) == (u < keep)
        out[x] += reach * keep
        reach *= 1 - keep
        P = O.left(P, q, x)
    return out + reach * P


@pytest.mark.parametrize("children", [1, 2, 3])
def test_verified_tokens_are_distributed_as_the_target(children):
    rng = np.random.default_rng(children)
    p, q = rng.dirichlet(np.ones(4)), rng.dirichlet(np.ones(4))
    total = np.zeros(4)
    for xs in itertools.product(range(4), repeat=children):
        total += math.prod(q[x] for x in xs) * first_token(p, q, xs)
    assert np.allclose(total, p, atol=1e-12)
    for xs in itertools.product(range(4), repeat=children):   # fixed proposals: for each of them
        assert np.allclose(first_token(p, None, xs), p, atol=1e-12)


def test_choose():
    P = np.array([0.0, 0.25, 0.0, 0.5, 0.25])
    assert [O.choose(P, u) for u in (0.0, 0.2, 0.25, 0.74, 0.75, 0.999)] == [1, 1, 3, 3, 4, 4]
    assert O.choose(np.zeros(3), 0.5) == -1 and O.choose(np.array([np.nan, 1]), 0.5) == -1 and O.choose(np.array([np.inf, 1]), 0.5) == -1


def test_a_walk_by_hand():
    """Root with children 1 (of probability 0) and 2; 3 hangs below 2; row 4 hangs below 1 and is never tried."""
    p = np.array([[0.5, 0.5, 0.0], [1, 0, 0], [0.1, 0.2, 0.7], [0, 0, 1], [1, 0, 0.0]])
    tokens, parent = [9, 2, 1, 2, 0], [-1, 0, 0, 2, 1]
    # 0.9 is not below row 0's 0.5 at token 1: both children go, token 0 is all that is left
    assert O.verify_one(tokens, parent, p, None, [0, 0.1, 0.9, 0.6, 0.0], 0.5) == ([0], 0)
    assert O.verify_one(tokens, parent, p, None, [0, 0.1, 0.4, 0.6, 0.0], 0.5) == ([0, 2, 3], 2)
    # 0.7 is not below 0.7: token 2 is taken out, a third and two thirds are left
    assert O.verify_one(tokens, parent, p, None, [0, 0.1, 0.4, 0.7, 0.0], 0.5) == ([0, 2], 1)
    rows, start, ctx, nxt = O.verify([0, 0, 5], [3, 7], tokens, parent, p, [0, 0.1, 0.4, 0.6, 0.0], [0.5, 0.5])
    assert rows == [0, 2, 3, -1, -1] and start == [0, 0, 3] and ctx == [3, 10] and nxt == [-1, 2]


def test_attention_of_a_tree_is_the_caches_attention_of_each_branch():
    """A branch's rows, appended to a cache in their order, see what the tree's rows see (up to the cache's codes:
    here values that the codes hold exactly)."""
    rng = np.random.default_rng(3)
    page, d, n_kv = 16, 16, 1
    k, v = (rng.integers(-3, 4, (9, n_kv, d)).astype(np.float32) for _ in range(2))
    k[:, :, 0] = v[:, :, 0] = 127.0   # scale 1
    empty = {"fmt": "int8", "k": np.zeros((2, n_kv, page, d), np.uint8), "v": np.zeros((2, n_kv, page, d), np.uint8),
             "k_scale": np.zeros((2, n_kv), np.float32), "v_scale": np.zeros((2, n_kv), np.float32)}
    q = rng.standard_normal((4, 2, d))
    parent = [-1, 0, 0, 2]
    masks = []
    for j, p in enumerate(parent):
        masks.append((masks[p] if p >= 0 else 0) | 1 << j)
    first = {"q_start": [0, 5], "ctx": [5], "table": [[1]]}
    cache = K.append(empty, first, k[:5], v[:5])
    y, lse, _ = O.attend_tree(cache, {"q_start": [0, 4], "ctx": [5], "table": [[1]]}, q, k[5:], v[5:], [[m] for m in masks], 0.01)
    for branch in ([0, 1], [0, 2, 3]):
        full = K.append(cache, {"q_start": [0, len(branch)], "ctx": [5 + len(branch)], "table": [[1]]}, k[5:][branch], v[5:][branch])
        yb, lb, _ = K.attend(full, {"q_start": [0, len(branch)], "ctx": [5 + len(branch)], "table": [[1]]}, q[branch], 0.01)
        assert np.allclose(yb, y[branch]) and np.allclose(lb, lse[branch])
    none = O.attend_tree(empty, {"q_start": [0, 1], "ctx": [0], "table": [[1]]}, q[:1], k[:1], v[:1], [[0]], 0.01)
    assert np.all(none[0] == 0) and np.all(np.isneginf(none[1]))
