"""pi_verify's outputs lie outside its inputs: refused on the host, before any HIP call."""

import os

import pytest

from activation_sparse_predictor_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")

A, APART = 1 << 20, 1 << 16   # aligned, never dereferenced addresses
N_SEQ, N_TOK, VOCAB, STRIDE = 2, 5, 100, 104
IN = {"q_start": 4 * (N_SEQ + 1), "ctx": 4 * N_SEQ, "tokens": 4 * N_TOK, "parent": 4 * N_TOK, "p": 4 * (4 * STRIDE + VOCAB),
      "q": 4 * (4 * STRIDE + VOCAB), "u": 4 * N_TOK, "u_next": 4 * N_SEQ}
OUT = {"rows": 4 * N_TOK, "start": 4 * (N_SEQ + 1), "new_ctx": 4 * N_SEQ, "next": 4 * N_SEQ}
AT = {n: A + i * APART for i, n in enumerate([*IN, *OUT, "ws"])}


def decide(**kw):
    a = {**AT, **kw}
    return B.pi_verify(N_SEQ, N_TOK, VOCAB, a["q_start"], a["ctx"], a["tokens"], a["parent"], a["p"], STRIDE, a["q"], STRIDE, a["u"],
                       a["u_next"], a["rows"], a["start"], a["new_ctx"], a["next"], a["ws"], 1 << 15, 0)


def refused(*names, **kw):
    return decide(**kw) == B.PI_ERR_INVALID_ARG and "overlaps" in B.last_error() and all(n in B.last_error() for n in names)


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("inp", IN)
def test_outputs_over_inputs_refused(out, inp):
    """At its first element, at its last, and with the output's own last element on its first."""
    places = [AT[inp], AT[inp] + IN[inp] - 4, AT[inp] - OUT[out] + 4]
    if (out, inp) == ("new_ctx", "ctx"):
        places = places[1:]   # itself is allowed
    for at in places:
        assert refused(out, inp, **{out: at})


@pytest.mark.parametrize("a", OUT)
@pytest.mark.parametrize("b", OUT)
def test_outputs_over_each_other_refused(a, b):
    if a != b:
        assert refused(a, b, **{a: AT[b] + OUT[b] - 4})


def test_workspaces_over_anything_refused():
    for name in (*IN, *OUT):
        assert refused("ws", name, ws=AT[name])
    need = B.pi_verify_workspace_size(N_SEQ, N_TOK, VOCAB)
    assert refused("ws", "rows", rows=AT["ws"] + need - 4)
