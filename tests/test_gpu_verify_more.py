"""pi_verify on the GPU: vocabularies whose sums' slices take several steps to search,
lengths updated in place, and host threads that share a stream."""

from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O
from tests.test_gpu_verify import DEV, case, run, same

pytestmark = pytest.mark.gpu


def wide(rng, counts, vocab, drawn):
    """Whole numbers of 2^-46 below 2^-24 as probabilities: every order of adding gives the same 64-bit sums, so the running
    sums decide alike everywhere."""
    tok = sum(counts)
    p = rng.integers(0, 1 << 22, (tok, vocab)).astype(np.float32) * np.float32(2.0 ** -46)
    p[rng.random((tok, vocab)) < 0.3] = 0.0
    q = rng.integers(0, 1 << 22, (tok, vocab)).astype(np.float32) * np.float32(2.0 ** -46) if drawn else None
    return dict(q_start=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), ctx=np.arange(len(counts), dtype=np.int32),
                tokens=rng.integers(0, vocab, tok).astype(np.int32), parent=np.concatenate([np.arange(n) - 1 for n in counts]).astype(np.int32),
                p=p, q=q, u=np.full(tok, 0.9375, np.float32), u_next=np.zeros(len(counts), np.float32))


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("vocab", [(1 << 20) + 1, (1 << 21) + 1025, 5000001, 1 << 24])
def test_slices_of_several_steps(drawn, vocab):
    rng = np.random.default_rng(vocab)
    c = wide(rng, [1, 1, 1] if vocab < 1 << 24 else [1], vocab, False)
    c["q"] = c["p"].copy() if drawn else None
    for u in (0.0, 0.123, 0.5, 0.77, 1 - 2.0 ** -24):
        c["u_next"][:] = np.float32(u)
        same(c)


@pytest.mark.parametrize("drawn", [True, False])
def test_several_steps_after_a_rejection(drawn):
    """A child that is rejected, and the next token from what it leaves."""
    vocab = (1 << 21) + 77
    rng = np.random.default_rng(5)
    c = wide(rng, [2, 2], vocab, drawn)
    c["tokens"][[1, 3]] = [11, vocab - 1]
    if drawn:
        c["q"][:, [11, vocab - 1]] = 0.5      # u q(x) > p(x), which is below 2^-24: rejected
    else:
        c["u"][:] = 0.9375                     # u > p(x)
    for u in (0.0, 0.25, 0.9, 1 - 2.0 ** -24):
        c["u_next"][:] = np.float32(u)
        want = same(c)
        assert want[1] == [0, 1, 2]


def test_lengths_in_place():
    """new_ctx may be ctx itself, as a step that updates its batch passes it."""
    rng = np.random.default_rng(7)
    c = case(rng, [5, 0, 9, 1], 3001, True)
    want = O.verify(c["q_start"], c["ctx"], c["tokens"], c["parent"], c["p"], c["u"], c["u_next"], c["q"])
    t = {n: torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for n, a in c.items()}
    out = {n: torch.zeros(k, dtype=torch.int32, device=DEV) for n, k in (("rows", 15), ("start", 5), ("next", 4))}
    size = B.pi_verify_workspace_size(4, 15, 3001)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    st = B.pi_verify(4, 15, 3001, t["q_start"], t["ctx"], t["tokens"], t["parent"], t["p"], 3001, t["q"], 3001, t["u"], t["u_next"],
                     out["rows"], out["start"], t["ctx"], out["next"], ws, size, torch.cuda.current_stream().cuda_stream)
    assert st == B.PI_OK
    got = [t.cpu().tolist() for t in (out["rows"], out["start"], t["ctx"], out["next"])]
    assert got == [[int(x) for x in w] for w in want]


def test_threads_that_share_a_stream():
    """Three threads, each with sequences and a vocabulary of its own, on the default stream: every result its thread's."""
    rng = np.random.default_rng(9)
    cases = [case(rng, counts, vocab, drawn) for counts, vocab, drawn in (([3, 7], 501, True), ([16] * 12, 2011, True), ([1, 30, 4], 977, False))]
    wants = [run(c) for c in cases]
    failed = []

    def work(c, want):
        try:
            t = {n: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for n, a in c.items()}
            batch = {"q_start": t["q_start"], "ctx": t["ctx"], "n_tok": len(c["tokens"])}
            for _ in range(4):
                outs = [R.verify(batch, t["tokens"], t["parent"], t["p"], t["u"], t["u_next"], q=t["q"]) for _ in range(50)]
                for o in outs:
                    if [o[n].cpu().tolist() for n in ("rows", "q_start", "ctx", "next")] != want:
                        raise AssertionError("another call's result")
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -1.0])
def test_the_draft_of_a_row_without_rejected_children_does_not_matter(value):
    """A draft model has no distribution for rows that nothing hangs below, and what the target's row gives is its own
    then: whatever lies in those rows of q, and in all rows once every child stays."""
    rng = np.random.default_rng(21)
    c = case(rng, [5, 1, 9, 16], 3001, True)
    for s in range(4):   # rows without children
        a, e = int(c["q_start"][s]), int(c["q_start"][s + 1])
        below = set(c["parent"][a + 1:e].tolist())
        for j in range(e - a):
            if j not in below:
                c["q"][a + j] = value
    for _ in range(4):
        c["u"][:] = rng.random(31, dtype=np.float32)
        c["u_next"][:] = rng.random(4, dtype=np.float32)
        same(c)
    c = case(rng, [4, 7], 501, True, chain=True)
    c["u"][:] = 0.0    # every child stays
    c["q"][:] = np.float32(value)
    for s, n in ((0, 4), (4, 7)):
        for j in range(1, n):
            c["q"][s + j - 1, c["tokens"][s + j]] = 0.25
    want = same(c)
    assert want[1] == [0, 4, 11] and min(want[3]) >= 0


def test_nothing_left_beside_an_endless_draft():
    """An infinite element of q takes its token away; where nothing is left the row's own p decides, that token's included."""
    c = dict(q_start=np.array([0, 2], np.int32), ctx=np.array([3], np.int32), tokens=np.array([0, 5], np.int32),
             parent=np.array([-1, 0], np.int32), p=np.zeros((2, 40), np.float32), q=np.zeros((2, 40), np.float32),
             u=np.array([0.0, 0.5], np.float32), u_next=np.array([0.5], np.float32))
    c["p"][0, 30] = 1.0
    c["q"][0, 30] = np.inf
    c["q"][0, 5] = 0.5    # the child's, of probability 0: rejected
    assert same(c)[3] == [30]
