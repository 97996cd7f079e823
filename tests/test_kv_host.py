"""The cache calls' refusals: every case fails before the library makes any HIP call (no GPU needed)."""

import os

import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")

A = 1 << 20   # an aligned, never dereferenced address
BAD, UNSUP, WS = B.PI_ERR_INVALID_ARG, B.PI_ERR_UNSUPPORTED, B.PI_ERR_WORKSPACE


def cache(**kw):
    a = dict(fmt=B.PI_KV_INT8, n_pages=4, n_kv=2, page=16, d=64, k=A, v=A, k_scale=A, v_scale=A)
    a.update(kw)
    return B.KvCache(*a.values())


def batch(**kw):
    a = dict(n_seq=2, n_tok=3, max_q=2, table_stride=4, q_start=A, ctx=A, table=A)
    a.update(kw)
    return B.KvBatch(*a.values())


def calls(c, b):
    yield B.pi_kv_append(c, b, A, 128, A, 128, 0)
    yield B.pi_kv_read(c, b, A, A, 0)
    yield B.pi_kv_attend(c, b, A, 512, 8, 0.1, 0, A, None, A, 1 << 40, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), BAD), (dict(n_pages=0), BAD), (dict(n_kv=0), BAD), (dict(n_kv=1025), BAD), (dict(page=0), BAD),
    (dict(page=24), UNSUP), (dict(page=8), UNSUP), (dict(page=512), UNSUP), (dict(d=0), BAD), (dict(d=72), UNSUP),
    (dict(d=272), UNSUP), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD),
    (dict(k=A + 8), UNSUP), (dict(v=A + 1), UNSUP), (dict(k_scale=A + 2), UNSUP)])
def test_caches_refused(kw, code):
    for st in calls(cache(**kw), batch()):
        assert st == code and B.last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), BAD), (dict(n_seq=1025), BAD), (dict(n_tok=0), BAD), (dict(n_tok=(1 << 20) + 1), BAD), (dict(max_q=0), BAD),
    (dict(max_q=4), BAD), (dict(table_stride=0), BAD), (dict(table_stride=1 << 27), BAD), (dict(q_start=None), BAD),
    (dict(ctx=None), BAD), (dict(table=None), BAD), (dict(table=A + 1), UNSUP)])
def test_batches_refused(kw, code):
    for st in calls(cache(), batch(**kw)):
        assert st == code and B.last_error() != ""


def test_null_descriptors_refused():
    for st in list(calls(None, batch())) + list(calls(cache(), None)):
        assert st == BAD


def append(**kw):
    a = dict(k=A, k_stride=128, v=A, v_stride=128)
    a.update(kw)
    return B.pi_kv_append(cache(), batch(), *a.values(), 0)


def attend(**kw):
    a = dict(q=A, q_stride=512, n_head=8, scale=0.1, window=0, y=A, lse=None, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return B.pi_kv_attend(cache(), batch(), *a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_stride=120), BAD), (dict(v_stride=-128), BAD), (dict(k_stride=132), UNSUP),
    (dict(k=A + 4), UNSUP), (dict(v_stride=1 << 41), BAD)])
def test_append_refused(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(y=None), BAD), (dict(n_head=0), BAD), (dict(n_head=7), BAD), (dict(n_head=2048), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(window=-1), BAD), (dict(q_stride=504), BAD),
    (dict(q_stride=516), UNSUP), (dict(q=A + 2), UNSUP), (dict(y=A + 8), UNSUP), (dict(lse=A + 2), UNSUP), (dict(ws=None), WS),
    (dict(ws_bytes=100), WS), (dict(ws=A + 16), UNSUP)])
def test_attend_refused(kw, code):
    assert attend(**kw) == code and B.last_error() != ""


def test_read_refused():
    assert B.pi_kv_read(cache(), batch(), None, A, 0) == BAD
    assert B.pi_kv_read(cache(), batch(), A, A + 2, 0) == UNSUP


def test_workspace_queries():
    n = B.pi_kv_workspace_size(4, 4, 1, 64, 8, 128)
    assert n > 0 and B.pi_kv_workspace_size(1, 2048, 2048, 64, 8, 128) > 0
    for bad in ((0, 4, 1, 64, 8, 128), (4, 4, 5, 64, 8, 128), (4, 4, 1, 63, 8, 128), (4, 4, 1, 64, 0, 128), (4, 4, 1, 64, 8, 0)):
        with pytest.raises(B.PiError) as e:
            B.pi_kv_workspace_size(*bad)
        assert e.value.status == BAD
    with pytest.raises(B.PiError):
        B.pi_kv_workspace_size(4, 4, 1, 64, 8, 100)


def test_runtime_refuses_what_it_cannot_pass_on():
    """Tensors of another place, type or shape raise before any call."""
    c = R.kv_cache(4, 2, 64, device="cpu")
    b = R.kv_batch([1, 2], [5, 6], [[0], [1]], device="cpu")
    assert b["n_tok"] == 3 and b["max_q"] == 2 and b["table"].tolist() == [[0], [1]] and b["q_start"].tolist() == [0, 1, 3]
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    for f in (lambda: R.kv_append(c, x, x, b), lambda: R.kv_read(c, b), lambda: R.kv_attend(c, x, b)):
        with pytest.raises(ValueError):
            f()
    assert R._kv_args(c, b, -1)[1].n_seq == 2
    for change in (dict(fmt="int4"), dict(k=c["k"].float()), dict(v=c["v"][:2]), dict(k_scale=c["k_scale"].double()),
                   dict(k=c["k"].transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            R._kv_args({**c, **change}, b, -1)
    for change in (dict(ctx=b["ctx"].long()), dict(table=b["table"][:1]), dict(q_start=b["q_start"][:2])):
        with pytest.raises(ValueError):
            R._kv_args(c, {**b, **change}, -1)
    assert R._kv_rows(x, 3, 2, 64, "k") == 128
    assert R._kv_rows(torch.zeros(3, 5, 128, dtype=torch.float16)[:, 1].view(3, 2, 64), 3, 2, 64, "k") == 640
    for t in (x.float(), x[:2], x[:, :1], x.transpose(0, 1), torch.zeros(3, 64, 2, dtype=torch.float16).transpose(1, 2)):
        with pytest.raises(ValueError):
            R._kv_rows(t, 3, 2, 64, "k")


def test_rows_above_the_limit_refused():
    """n_tok * n_head / n_kv above PI_KV_MAX_ROWS: attention refuses, append and read do not count heads."""
    b = batch(n_tok=1 << 20, max_q=1 << 20)
    st = B.pi_kv_attend(cache(n_kv=1), b, A, 64 * 64, 64, 0.1, 0, A, None, A, 1 << 40, 0)
    assert st == UNSUP and "PI_KV_MAX_ROWS" in B.last_error()
    with pytest.raises(B.PiError) as e:
        B.pi_kv_workspace_size(2, 1 << 20, 1 << 20, 64, 1, 64)
    assert e.value.status == UNSUP


LEAD = 8192 + 65536   # a workspace's header and attention's counters: what has to be zero


@pytest.fixture
def pretend(monkeypatch):
    """kv_attend over a stand-in for the library's call, on host tensors: what
    it is given, and the workspace's leading words, are noted."""
    seen, state = [], {"capturing": False}

    def attend(c, b, q, qs, heads, scale, window, y, lse, ws, size, st):
        need = B.pi_kv_workspace_size(b.n_seq, b.n_tok, b.max_q, heads, c.n_kv, c.d)
        if ws is None or size < need:
            return WS
        seen.append({"ws": ws, "at": ws.data_ptr(), "clean": not torch.any(ws[:LEAD]), "window": window})
        ws[:LEAD].fill_(1)
        return B.PI_OK

    monkeypatch.setattr(B, "pi_kv_attend", attend)
    monkeypatch.setattr(R, "_is_elsewhere", lambda stream, dev: False)
    monkeypatch.setattr(R, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(R, "_capturing", lambda: state["capturing"], raising=False)
    monkeypatch.setattr(R, "_KV_WS", {})
    c = R.kv_cache(40, 2, 64, device="cpu")

    def call(new=1, capturing=False, **kw):
        state["capturing"] = capturing
        b = R.kv_batch([new], [new], [list(range(40))], device="cpu")
        R.kv_attend(c, torch.zeros(new, 128, 64, dtype=torch.float16), b, **kw)
        return seen.pop()
    return call


def test_each_captured_call_has_a_workspace_of_its_own(pretend):
    """Without ws: eager calls of a stream share one that grows; a captured call
    gets its own, zeroed inside the capture, that no other call meets and that
    no growth gives away."""
    graphs = [pretend(capturing=True) for _ in range(2)]   # before any eager call
    assert R._KV_WS == {} or all(w.buf is None for w in R._KV_WS.values())
    small = pretend()
    assert pretend()["at"] == small["at"]
    graphs.append(pretend(capturing=True))
    large = pretend(new=500)
    assert large["at"] != small["at"] and pretend()["at"] == large["at"]
    graphs.append(pretend(capturing=True))
    at = [g["at"] for g in graphs]
    assert len(set(at)) == len(at) and small["at"] not in at and large["at"] not in at
    assert all(g["clean"] for g in graphs) and small["clean"] and large["clean"]


def test_a_workspace_that_is_passed_is_used_also_under_capture(pretend):
    ws = R.kv_workspace(1, 1, 1, 128, 2, 64, device="cpu")
    for capturing in (False, True):
        assert pretend(capturing=capturing, ws=ws)["at"] == ws.data_ptr()


def test_windows_outside_the_c_type(pretend):
    """A window beyond 32 bits is as wide as the type; a negative one stays negative (and is refused)."""
    for window, want in ((0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (1 << 62, 2 ** 31 - 1),
                         (-1, -1), (-(2 ** 32) + 5, -1)):
        for capturing in (False, True):
            assert pretend(window=window, capturing=capturing)["window"] == want
        assert pretend(window=window, ws=R.kv_workspace(1, 1, 1, 128, 2, 64, device="cpu"))["window"] == want
