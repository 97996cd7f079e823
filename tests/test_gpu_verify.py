"""pi_verify on the GPU against the float64 oracle (oracle/draft.py): whole
numbers, equal.  The probabilities are random fp32 numbers, so a 64-bit sum's
last bit decides for no neighbour."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def tree(rng, n, chain=False):
    return [-1] + [j - 1 if chain else max(0, j - 1 - int(rng.exponential(2.5))) for j in range(1, n)]


def case(rng, counts, vocab, drawn, chain=False, sharp=2.0):
    """Inputs as a program has them: children drawn from the draft's distribution, or proposals among the likely tokens."""
    tok = sum(counts)
    z = rng.standard_normal((tok, vocab)) * sharp
    p, q = softmax(z), softmax(0.7 * z + rng.standard_normal((tok, vocab))) if drawn else None
    parent = np.concatenate([tree(rng, n, chain) for n in counts if n] or [[]]).astype(np.int32)
    tokens, at = np.zeros(tok, np.int32), 0
    for n in counts:
        for j in range(n):
            r = at + max(parent[at + j], 0)
            tokens[at + j] = rng.choice(vocab, p=(q[r] / q[r].sum(dtype=np.float64)).astype(np.float64) / np.sum(
                (q[r] / q[r].sum(dtype=np.float64)).astype(np.float64))) if drawn else np.argsort(-p[r], kind="stable")[rng.integers(min(vocab, 5))]
        at += n
    return dict(q_start=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), ctx=rng.integers(0, 1000, len(counts)).astype(np.int32),
                tokens=tokens, parent=parent, p=p, q=q, u=rng.random(tok, dtype=np.float32),
                u_next=rng.random(len(counts), dtype=np.float32))


def run(c, **kw):
    t = {n: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for n, a in c.items()}
    t.update(kw)
    batch = {"q_start": t["q_start"], "ctx": t["ctx"], "n_tok": c["tokens"].shape[0]}
    got = R.verify(batch, t["tokens"], t["parent"], t["p"], t["u"], t["u_next"], q=t["q"])
    return [got[n].cpu().tolist() for n in ("rows", "q_start", "ctx", "next")]


def same(c, **kw):
    want = O.verify(c["q_start"], c["ctx"], c["tokens"], c["parent"], c["p"], c["u"], c["u_next"], c["q"])
    got = run(c, **kw)
    for name, g, w in zip(("rows", "q_start", "ctx", "next"), got, want):
        assert g == [int(x) for x in w], (name, g, w)
    return want


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("counts,vocab", [
    ([1], 1), ([5], 2), ([3, 1, 0, 7], 31), ([0, 4], 1000), ([16] * 9, 1024), ([9, 33], 1025), ([64, 65, 63], 2047), ([130, 2], 4099),
    ([4, 4], 50257), ([6], 131072), ([2], 1 << 20)])
def test_equal(drawn, chain, counts, vocab):
    rng = np.random.default_rng(vocab + len(counts))
    for rep in range(3 if vocab < 5000 else 1):
        same(case(rng, counts, vocab, drawn, chain))


@pytest.mark.parametrize("drawn", [True, False])
def test_many_sequences(drawn):
    rng = np.random.default_rng(7)
    want = same(case(rng, [int(x) for x in rng.integers(0, 6, 1024)], 77, drawn))
    assert want[1][-1] > 1024 * 0.5


@pytest.mark.parametrize("drawn", [True, False])
def test_wide_trees(drawn):
    """Every row a child of the first: siblings beyond the 64 rows that are read at a time, tokens twice among them."""
    rng = np.random.default_rng(11)
    for vocab in (3, 40, 3000):
        c = case(rng, [200, 70], vocab, drawn, sharp=1.0)
        for a, e in ((0, 200), (200, 270)):
            c["parent"][a + 1:e] = 0
        c["u"][:] = np.where(rng.random(270) < 0.9, np.float32(0.9999), c["u"])   # mostly rejected
        same(c)


def test_strided_and_unaligned_rows():
    rng = np.random.default_rng(13)
    c = case(rng, [7, 9], 1001, True)
    for pad, off in ((3, 1), (8, 3), (0, 0)):
        wide = {n: torch.zeros(16, 1001 + pad, device=DEV) for n in "pq"}
        for n in "pq":
            wide[n][:, off:off + 1001] = torch.from_numpy(c[n]).to(DEV)
        same(c, p=wide["p"][:, off:off + 1001], q=wide["q"][:, off:off + 1001])


def test_greedy():
    """One-hot targets: the drafts that name the token stay, whatever the random numbers."""
    rng = np.random.default_rng(17)
    c = case(rng, [12, 12], 50, False)
    best = rng.integers(0, 50, 24)
    c["p"] = np.eye(50, dtype=np.float32)[best]
    for s in (0, 12):
        c["parent"][s:s + 12] = [-1, 0, 0, 1, 2, 2, 4, 4, 6, 5, 7, 9]
        c["tokens"][s + 2], c["tokens"][s + 4], c["tokens"][s + 1] = best[s], best[s + 2], (best[s] + 1) % 50
        c["tokens"][s + 5] = (best[s + 2] + 1) % 50
    for u in (0.0, 1 - 2.0 ** -24):
        c["u"][:] = u
        c["u_next"][:] = u
        rows, _, _, nxt = same(c)
        assert rows[:3] == [0, 2, 4] and nxt[0] == best[rows[run(c)[1][1] - 1]]


def test_ends_of_the_random_numbers():
    rng = np.random.default_rng(19)
    for drawn in (True, False):
        for u in (0.0, 1 - 2.0 ** -24):
            for w in (0.0, 1 - 2.0 ** -24):
                c = case(rng, [9, 5, 1], 2500, drawn)
                c["p"][:, -30:] = 0.0   # the last tokens have no probability
                c["p"][:, :7] = 0.0
                c["u"][:] = u
                c["u_next"][:] = w
                nxt = same(c)[3]
                assert all(7 <= t < 2470 for t in nxt)


def test_broken_inputs():
    """Tokens and parents outside their ranges, rows that hold NaN, infinity or nothing, distributions that leave nothing."""
    rng = np.random.default_rng(23)
    for drawn in (True, False):
        c = case(rng, [8] * 7, 300, drawn)
        c["tokens"][[1, 9, 17]] = [-1, 300, 2 ** 31 - 1]
        c["parent"][[2, 10, 18, 26]] = [2, 7, -5, 2 ** 31 - 1]
        c["parent"][0] = 0
        same(c)
        for value, where in ((np.nan, 3), (np.inf, 4), (0.0, 5)):
            one = {n: None if a is None else a.copy() for n, a in c.items()}
            one["p"][8 * where:8 * where + 8] = 0.0
            one["p"][8 * where:8 * where + 8, 250] = value
            nxt = run(one)[3]
            assert nxt[where] == -1
            keep = [s for s in range(7) if s != where]
            assert [nxt[s] for s in keep] == [run(c)[3][s] for s in keep]
    c = case(rng, [2], 3000, True)
    c["p"][0] = c["q"][0] = np.eye(3000, dtype=np.float32)[2999]
    c["tokens"][1] = 5          # of probability 0 in both: rejected, and p - q is 0 everywhere
    assert run(c) == [[0, -1], [0, 1], [int(c["ctx"][0]) + 1], [2999]]
    c = case(rng, [2], 3000, False)
    c["p"][0] = np.eye(3000, dtype=np.float32)[1500] * np.float32(0.5)
    c["tokens"][1], c["u"][1] = 1500, 0.75   # rejected, and it was all there was
    assert run(c) == [[0, -1], [0, 1], [int(c["ctx"][0]) + 1], [1500]]


def test_rows_of_no_sequence():
    """q_start that ends early: the rows behind are nobody's; one that is broken stays inside the arrays."""
    rng = np.random.default_rng(29)
    c = case(rng, [5, 4, 6], 200, True)
    c["q_start"] = np.array([0, 5, 9, 9], np.int32)
    want = O.verify(c["q_start"], c["ctx"], c["tokens"], c["parent"], c["p"], c["u"], c["u_next"], c["q"])
    got = run(c)
    assert got[0] == [int(x) for x in want[0]] and got[3] == want[3] and len(got[0]) == 15
    c["q_start"] = np.array([-7, 2 ** 31 - 1, -2 ** 31, 99], np.int32)
    assert all(-1 <= r < 15 for r in run(c)[0])


def test_same_answer_again_on_another_stream_and_replayed():
    rng = np.random.default_rng(31)
    c = case(rng, [11, 16, 3], 30011, True)
    want = run(c)
    t = {n: torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for n, a in c.items()}
    batch = {"q_start": t["q_start"], "ctx": t["ctx"], "n_tok": 30}

    def call(stream=None):
        return R.verify(batch, t["tokens"], t["parent"], t["p"], t["u"], t["u_next"], q=t["q"], stream=stream)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(side)
    torch.cuda.synchronize()
    assert [out[n].tolist() for n in ("rows", "q_start", "ctx", "next")] == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for rep in range(4):
        u = rng.random(30, dtype=np.float32)
        t["u"].copy_(torch.from_numpy(u))
        eager = {n: v.tolist() for n, v in call().items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert {n: v.tolist() for n, v in out.items()} == eager
