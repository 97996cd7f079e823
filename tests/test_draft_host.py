"""Rotary positions and verification without a GPU: the host-only functions
against the oracle, and refusals, which fail before any HIP call."""

import math
import os

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O
from tests.test_kv_host import A, BAD, UNSUP, WS, batch, cache

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,factor", [(2, 10000.0, 2.0), (64, 10000.0, 8.0), (128, 5e5, 32.0), (26, 100.0, 1.0)])
def test_frequencies(scaling, rot, base, factor):
    freqs, gain = B.pi_rope_frequencies(rot, base, B.ROPE_SCALINGS[scaling], factor, 4096.0, 1.0, 32.0)
    want, g = O.frequencies(rot, base, scaling, factor)
    assert np.allclose(freqs, want, rtol=1e-14) and gain == np.float32(g)


def test_turns():
    """Parts of a turn, to the nearest 2^-64, whole turns dropped."""
    f = np.array([0.0, 1.0, 2 * math.pi * 0.25, 7.0, 1e-4, 100.0])
    turns = [int(t) for t in B.pi_rope_turns(f)]
    for x, t in zip(f, turns):
        part = t / 2.0 ** 64
        assert abs((x / (2 * math.pi) - part + 0.5) % 1.0 - 0.5) < 1e-15
    plan = R.rope(8, freqs=f[:4], gain=2.0, layout="pairs", device="cpu")
    assert plan["turns"].tolist() == [t - (1 << 64) if t >> 63 else t for t in turns[:4]] and plan["gain"] == 2.0
    plan = R.rope(64, scaling="yarn", factor=4.0, device="cpu")
    assert plan["turns"].shape == (32,) and plan["gain"] == pytest.approx(0.1 * math.log(4) + 1)


@pytest.mark.parametrize("args", [
    (3, 1e4, 0, 1.0, 4096.0, 1.0, 32.0), (0, 1e4, 0, 1.0, 4096.0, 1.0, 32.0), (-2, 1e4, 0, 1.0, 4096.0, 1.0, 32.0),
    (8, 1.0, 0, 1.0, 4096.0, 1.0, 32.0), (8, NAN, 0, 1.0, 4096.0, 1.0, 32.0), (8, 1e4, 4, 1.0, 4096.0, 1.0, 32.0),
    (8, 1e4, 1, 0.5, 4096.0, 1.0, 32.0), (8, 1e4, 2, INF, 4096.0, 1.0, 32.0), (8, 1e4, 3, 2.0, 0.0, 1.0, 32.0),
    (8, 1e4, 3, 2.0, 4096.0, 32.0, 32.0), (8, 1e4, 3, 2.0, 4096.0, -1.0, 32.0), (8, 1e4, 3, 2.0, NAN, 1.0, 32.0)])
def test_frequencies_refused(args):
    with pytest.raises(B.PiError) as e:
        B.pi_rope_frequencies(*args)
    assert e.value.status == BAD


def test_turns_refused():
    for bad in ([-1.0], [NAN], [INF], [2.0 ** 21], []):
        with pytest.raises(B.PiError) as e:
            B.pi_rope_turns(np.array(bad))
        assert e.value.status == BAD


def plan(**kw):
    a = dict(layout=0, rot=64, gain=1.0, turns=A)
    a.update(kw)
    return B.Rope(*a.values())


PLANS = [(dict(layout=2), BAD), (dict(rot=0), BAD), (dict(rot=7), BAD), (dict(rot=66), BAD), (dict(gain=0.0), BAD),
         (dict(gain=NAN), BAD), (dict(gain=2048.0), BAD), (dict(gain=-1.0), BAD), (dict(turns=None), BAD), (dict(turns=A + 4), UNSUP)]
FAR = A + (1 << 24)


def turn(rope=None, **kw):
    a = dict(pos=A, n_tok=3, n_head=2, d=64, x=A, x_stride=128, y=FAR, y_stride=128)
    a.update(kw)
    return B.pi_rotate(plan() if rope is None else rope, *a.values(), 0)


def write(rope=None, c=None, b=None, **kw):
    a = dict(rows=None, n_src=3, k=A, k_stride=128, v=A, v_stride=128, q=A, q_stride=512, n_head=8, q_out=FAR, out_stride=512)
    a.update(kw)
    return B.pi_kv_append_rope(c or cache(), b or batch(), plan() if rope is None else rope, *a.values(), 0)


@pytest.mark.parametrize("kw,code", PLANS)
def test_plans_refused(kw, code):
    for st in (turn(plan(**kw)), write(plan(**kw)), write(plan(**kw), q=None)):
        assert st == code and B.last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(pos=None), BAD), (dict(pos=A + 2), UNSUP), (dict(n_tok=0), BAD), (dict(n_tok=(1 << 20) + 1), BAD), (dict(n_head=0), BAD),
    (dict(n_head=2049), BAD), (dict(d=0), BAD), (dict(d=68), UNSUP), (dict(d=264), UNSUP), (dict(x=None), BAD), (dict(y=None), BAD),
    (dict(x=A + 2), UNSUP), (dict(y=A + 8), UNSUP), (dict(x_stride=120), BAD), (dict(y_stride=120), BAD), (dict(x_stride=132), UNSUP),
    (dict(y=A, y_stride=256), BAD), (dict(y=A + 16), BAD), (dict(y=A + 3 * 256 - 16), BAD), (dict(x=A + 16, y=A), BAD)])
def test_rotate_refused(kw, code):
    assert turn(**kw) == code and B.last_error() != ""
    assert B.pi_rotate(None, A, 3, 2, 64, A, 128, FAR, 128, 0) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(rows=A + 2), UNSUP), (dict(n_src=2), BAD), (dict(n_src=0), BAD), (dict(n_src=(1 << 20) + 1), BAD), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(k=A + 8), UNSUP), (dict(k_stride=120), BAD), (dict(v_stride=132), UNSUP), (dict(rows=A), BAD),
    (dict(n_head=7), BAD), (dict(n_head=0), BAD), (dict(q=A + 2), UNSUP), (dict(q_out=None), BAD), (dict(q_out=A + 4), UNSUP),
    (dict(q_stride=504), BAD), (dict(out_stride=504), BAD), (dict(q_out=A + 64), BAD), (dict(q_out=A, out_stride=1024), BAD)])
def test_append_rope_refused(kw, code):
    assert write(**kw) == code and B.last_error() != ""


def test_append_rope_refuses_what_append_refuses():
    for kw, code in ((dict(fmt=2), BAD), (dict(page=24), UNSUP), (dict(k=None), BAD), (dict(d=72), UNSUP)):
        assert write(c=cache(**kw)) == code
    for kw, code in ((dict(n_seq=0), BAD), (dict(max_q=4), BAD), (dict(table=A + 1), UNSUP)):
        assert write(b=batch(**kw)) == code
    assert B.pi_kv_append_rope(None, batch(), None, None, 3, A, 128, A, 128, None, 0, 0, None, 0, 0) == BAD
    assert B.pi_kv_append_rope(cache(), None, None, None, 3, A, 128, A, 128, None, 0, 0, None, 0, 0) == BAD
    # queries need a plan
    assert B.pi_kv_append_rope(cache(), batch(), None, None, 3, A, 128, A, 128, A, 512, 8, FAR, 512, 0) == BAD


def tree(c=None, b=None, **kw):
    a = dict(q=A, q_stride=512, n_head=8, k=A, k_stride=128, v=A, v_stride=128, mask=A, words=1, pos=None, scale=0.1, window=0, y=A,
             lse=None, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return B.pi_kv_attend_tree(c or cache(), b or batch(), *a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(y=None), BAD), (dict(mask=None), BAD), (dict(mask=A + 4), UNSUP),
    (dict(words=0), BAD), (dict(words=5), BAD), (dict(window=3), BAD), (dict(window=3, pos=A + 2), UNSUP), (dict(pos=A + 2), UNSUP),
    (dict(window=-1), BAD), (dict(k=A + 8), UNSUP), (dict(v=A + 2), UNSUP), (dict(k_stride=120), BAD), (dict(v_stride=132), UNSUP),
    (dict(n_head=7), BAD), (dict(n_head=0), BAD), (dict(scale=NAN), BAD), (dict(q_stride=504), BAD), (dict(q=A + 2), UNSUP),
    (dict(y=A + 8), UNSUP), (dict(lse=A + 2), UNSUP), (dict(ws=None), WS), (dict(ws_bytes=100), WS), (dict(ws=A + 16), UNSUP)])
def test_tree_refused(kw, code):
    assert tree(**kw) == code and B.last_error() != ""


def test_tree_refuses_more_rows_than_the_mask_has():
    big = batch(n_tok=500, max_q=65)
    assert tree(b=big) == BAD and tree(b=big, words=2, ws=None) == WS
    assert tree(b=batch(n_tok=500, max_q=257), words=4) == BAD
    assert tree(c=cache(fmt=2)) == BAD and tree(b=batch(n_seq=0)) == BAD


def test_trees_from_lists():
    t = R.kv_tree([[-1, 0, 0, 2], [-1], [-1] + list(range(69))], device="cpu")
    assert t["mask"].shape == (75, 2) and t["parent"].tolist()[:6] == [-1, 0, 0, 2, -1, -1] and t["depth"].tolist()[:6] == [0, 1, 1, 2, 0, 0]
    assert t["mask"][:5, 0].tolist() == [1, 3, 5, 13, 1] and t["mask"][:5, 1].tolist() == [0] * 5
    assert t["mask"][5 + 63].tolist() == [-1, 0] and t["mask"][5 + 69].tolist() == [-1, 63] and t["depth"][-1] == 69
    assert R.kv_tree([[-1], [], [-1, 0]], device="cpu")["mask"].tolist() == [[1], [1], [3]]
    for bad in ([[0]], [[-1, 1]], [[-1, -2]]):
        with pytest.raises(ValueError):
            R.kv_tree(bad, device="cpu")


def decide(**kw):
    a = dict(n_seq=2, n_tok=5, vocab=100, q_start=A, ctx=A, tokens=A, parent=A, p=A, p_stride=100, q=A, q_stride=100, u=A, u_next=A,
             rows=A, start=A, new_ctx=A, next=A, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    return B.pi_verify(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), BAD), (dict(n_seq=1025), BAD), (dict(n_tok=0), BAD), (dict(n_tok=(1 << 20) + 1), BAD), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 24) + 1), BAD), (dict(p_stride=99), BAD), (dict(q_stride=99), BAD), (dict(p_stride=1 << 41), BAD),
    (dict(ws=None), WS), (dict(ws_bytes=16), WS), (dict(ws=A + 16), UNSUP)]
    + [({n: None}, BAD) for n in ("q_start", "ctx", "tokens", "parent", "p", "u", "u_next", "rows", "start", "new_ctx", "next")]
    + [({n: A + 2}, UNSUP) for n in ("q_start", "ctx", "tokens", "parent", "p", "q", "u", "u_next", "rows", "start", "new_ctx", "next")])
def test_verify_refused(kw, code):
    assert decide(**kw) == code and B.last_error() != ""


def test_verify_workspace_queries():
    assert 0 < B.pi_verify_workspace_size(1, 1, 1) < B.pi_verify_workspace_size(64, 1000, 128000)
    assert B.pi_verify_workspace_size(1024, 1 << 20, 1 << 24) < 1 << 28
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1025, 1, 1)):
        with pytest.raises(B.PiError) as e:
            B.pi_verify_workspace_size(*bad)
        assert e.value.status == BAD


def test_runtime_refuses_what_it_cannot_pass_on(monkeypatch):
    """Tensors of another place, type or shape raise before any call."""
    c = R.kv_cache(4, 2, 64, device="cpu")
    b = R.kv_batch([1, 2], [5, 6], [[0], [1]], device="cpu")
    x, pos, turns = torch.zeros(3, 2, 64).half(), torch.zeros(3, dtype=torch.int32), R.rope(64, device="cpu")
    i, f, p = torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros(3, 10)
    for call in (lambda: R.rotate(x, pos, turns), lambda: R.kv_append_rope(c, x, x, b, turns, q=x), lambda: R.verify(b, i, i, p, f, f[:2]),
                 lambda: R.kv_attend_tree(c, x, x, x, b, torch.ones(3, 1, dtype=torch.int64))):
        with pytest.raises(ValueError):   # the host is no place for them
            call()
    monkeypatch.setattr(R, "_is_elsewhere", lambda stream, dev: False)
    monkeypatch.setattr(R, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(R, "_capturing", lambda: False)
    done = []
    for name in ("pi_rotate", "pi_kv_append_rope", "pi_verify", "pi_kv_attend_tree"):
        monkeypatch.setattr(B, name, lambda *a, **k: done.append(a) or B.PI_OK)
    R.rotate(x, pos, turns)
    R.kv_append_rope(c, x, x, b, turns, q=x)
    R.kv_append_rope(c, torch.zeros(9, 2, 64).half(), torch.zeros(9, 2, 64).half(), b, rows=i)
    R.verify(b, i, i, p, f, f[:2], q=torch.zeros(3, 20)[:, :10])
    m, ws = torch.ones(3, 1, dtype=torch.int64), torch.zeros(1 << 10, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64).half()
    R.kv_attend_tree(c, q, x, x, b, m, pos, window=2 ** 40, ws=ws)
    assert len(done) == 5 and done[-1][13] == 2 ** 31 - 1
    refused = [
        lambda: R.kv_attend_tree(c, q, x, x, b, m.int(), ws=ws), lambda: R.kv_attend_tree(c, q, x, x, b, m[:2], ws=ws),
        lambda: R.kv_attend_tree(c, q, x, x, b, m[:, 0], ws=ws), lambda: R.kv_attend_tree(c, q, x[:2], x, b, m, ws=ws),
        lambda: R.kv_attend_tree(c, q, x, q, b, m, ws=ws), lambda: R.kv_attend_tree(c, q.float(), x, x, b, m, ws=ws),
        lambda: R.kv_attend_tree(c, q, x, x, b, m, pos.long(), ws=ws), lambda: R.kv_attend_tree(c, q, x, x, b, m, y=x, ws=ws),
        lambda: R.kv_attend_tree(c, q, x, x, b, m, lse=torch.zeros(3, 3), ws=ws),
        lambda: R.rotate(x.float(), pos, turns), lambda: R.rotate(x[0], pos, turns), lambda: R.rotate(x, pos.long(), turns),
        lambda: R.rotate(x, pos[:2], turns), lambda: R.rotate(x, pos, {**turns, "layout": "other"}),
        lambda: R.rotate(x, pos, {**turns, "rot": 32}), lambda: R.rotate(x, pos, {**turns, "turns": turns["turns"].int()}),
        lambda: R.rotate(x, pos, turns, out=x[:2]), lambda: R.rotate(x.transpose(1, 2), pos, turns),
        lambda: R.kv_append_rope(c, x, x[:2], b, turns), lambda: R.kv_append_rope(c, x, x, b, turns, q_out=x),
        lambda: R.kv_append_rope(c, x, x, b, rows=i.long()), lambda: R.kv_append_rope(c, x, x, b, rows=i[:2]),
        lambda: R.kv_append_rope(c, x, x, b, turns, q=x.float()), lambda: R.verify(b, i.long(), i, p, f, f[:2]),
        lambda: R.verify(b, i, i, p.half(), f, f[:2]), lambda: R.verify(b, i, i, p.t(), f, f[:2]),
        lambda: R.verify(b, i, i, p, f, f), lambda: R.verify(b, i, i, p, f, f[:2], q=p[:, :9]), lambda: R.verify(b, i[:2], i, p, f, f[:2]),
        lambda: R.rope(64, layout="x", device="cpu"), lambda: R.rope(64, freqs=[1.0], device="cpu")]
    for call in refused:
        with pytest.raises(ValueError):
            call()
    assert len(done) == 5
