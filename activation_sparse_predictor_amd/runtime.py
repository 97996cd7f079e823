"""Device-buffer plumbing around the C ABI: workspaces, outputs, layer bundles.

Nothing here computes part of the path.  torch provides device memory and the
stream; every arithmetic step runs in libpi's HIP kernels via `binding`.
A layer is a dict of device tensors named as in the C ABI (W_up, W_gate,
W_down, b_up, b_gate, P1, b1, P2, b2) plus kind, tau and sizes.
"""

from __future__ import annotations

import functools
import threading
from typing import Dict, Optional, Tuple

import torch

from . import binding as B


class Workspace:
    """A grow-only device byte buffer, 256-byte aligned (torch allocations are)."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.buf: Optional[torch.Tensor] = None

    def get(self, nbytes: int) -> Tuple[Optional[torch.Tensor], int]:
        if nbytes == 0:
            return None, 0
        buf = self.buf   # (read once: another thread may replace it)
        if buf is None or buf.numel() < nbytes:
            # zero-filled once: the library keeps epoch-tagged sync words in its header
            buf = self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        return buf, buf.numel()


_WS: Dict[Tuple[str, int], Workspace] = {}


def workspace(tag: str, device=None) -> Workspace:
    """The workspace kept under `tag` on a device.  Each layout (single-token
    and batched calls of an entry point, the dense baseline) gets its own tag,
    so that calls alternating between layouts never make the library clear a
    workspace, and a captured graph never meets a workspace that another
    layout wrote between its replays."""
    dev = torch.device(device or "cuda")
    key = (tag, dev.index if dev.index is not None else torch.cuda.current_device())
    if key not in _WS:
        _WS[key] = Workspace(dev)
    return _WS[key]


def _bits(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """fp16 tensors are passed by address; make sure they are contiguous fp16."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpi must be contiguous")
    return t


def predict(layer: dict, x: torch.Tensor, idx: Optional[torch.Tensor] = None,
            count: Optional[torch.Tensor] = None, act: str = "relu",
            tau: Optional[float] = None, n_hot: int = 0, stream=None):
    """idx (B x ffn int32) and count (B int32) for tokens x (B x d fp16).
    n_hot > 0: neurons [0, n_hot) of a hot-first layer are always listed and
    skip the predictor (pi_ffn_predict_hot)."""
    Bt, d = x.shape
    ffn, r = layer["ffn"], layer["r"]
    if idx is None:
        idx = torch.empty(Bt, ffn, dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty(Bt, dtype=torch.int32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_PREDICT, Bt, d, r, ffn)
    ws, wsb = workspace("predict" if Bt == 1 else "predict_batch", x.device).get(nbytes)
    t = float(layer["tau"] if tau is None else tau)
    if n_hot:
        st = B.pi_ffn_predict_hot(_bits(x), Bt, d, layer["P1"], layer.get("b1"), B.ACTS[act], layer["P2"],
                                  layer.get("b2"), r, ffn, int(n_hot), t, idx, count, ws, wsb, stream)
        B.check(st, "pi_ffn_predict_hot")
    else:
        st = B.pi_ffn_predict(_bits(x), Bt, d, layer["P1"], layer.get("b1"), B.ACTS[act], layer["P2"],
                              layer.get("b2"), r, ffn, t, idx, count, ws, wsb, stream)
        B.check(st, "pi_ffn_predict")
    return idx, count


def sparse(layer: dict, x: torch.Tensor, idx: Optional[torch.Tensor],
           count: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
           dense: bool = False, per_token: bool = False, check_idx: bool = False,
           stream=None) -> torch.Tensor:
    """y (B x d fp32) from the active rows (or every row with dense=True).

    For B >= 2 the library reads the union of the tokens' rows once (matrix
    cores); per_token=True runs each token through the single-token kernels.
    check_idx=True has the device check each list afterwards and fill y_t with
    NaN where it breaks the contract (ids in [0, ffn), strictly ascending).
    """
    Bt, d = x.shape
    ffn = layer["ffn"]
    if y is None:
        y = torch.empty(Bt, d, dtype=torch.float32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_SPARSE, Bt, d, layer.get("r", 8), ffn)
    tag = "sparse_dense" if dense else ("sparse" if Bt == 1 or per_token else "sparse_batch")
    ws, wsb = workspace(tag, x.device).get(nbytes)
    st = B.pi_ffn_sparse(B.KINDS[layer["kind"]], _bits(x), Bt, d, ffn, layer["W_up"],
                         layer.get("b_up"), layer.get("W_gate"), layer.get("b_gate"),
                         layer["W_down"], None if dense else idx, None if dense else count, y,
                         (B.PI_DENSE if dense else 0) | (B.PI_PER_TOKEN if per_token else 0)
                         | (B.PI_CHECK_IDX if check_idx else 0),
                         ws, wsb, stream)
    B.check(st, "pi_ffn_sparse")
    return y


def quantize_rows(W: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """INT4 codes (rows x d/2 uint8) and scales (rows x d/64 fp16) of fp16 rows W."""
    rows, d = W.shape
    q = torch.empty(rows, d // 2, dtype=torch.uint8, device=W.device)
    s = torch.empty(rows, d // 64, dtype=torch.float16, device=W.device)
    B.check(B.pi_quantize_rows(_bits(W), rows, d, q, s, stream), "pi_quantize_rows")
    return q, s


def quantize_layer(layer: dict, stream=None) -> dict:
    """The layer with W_up, W_gate, W_down and the predictor's P1, P2 as INT4
    rows (q_*, s_*); the biases are kept.  The predictor is quantised only
    when r is a multiple of 64 (the group); otherwise q_P1 .. s_P2 are None."""
    out = {k: v for k, v in layer.items() if k not in ("W_up", "W_gate", "W_down", "P1", "P2")}
    pred_ok = layer.get("P2") is not None and layer["P2"].shape[1] % 64 == 0
    for k, name in (("W_up", "up"), ("W_gate", "gate"), ("W_down", "down"), ("P1", "P1"), ("P2", "P2")):
        if layer.get(k) is not None and (pred_ok or k not in ("P1", "P2")):
            out["q_" + name], out["s_" + name] = quantize_rows(layer[k], stream)
        else:
            out["q_" + name], out["s_" + name] = None, None
    return out


def predict_q4(layer_q: dict, x: torch.Tensor, idx: Optional[torch.Tensor] = None,
               count: Optional[torch.Tensor] = None, act: str = "relu", tau: Optional[float] = None,
               n_hot: int = 0, stream=None):
    """pi_ffn_predict_q4 over a layer from quantize_layer: idx and count as predict()."""
    Bt, d = x.shape
    ffn, r = layer_q["ffn"], layer_q["r"]
    if idx is None:
        idx = torch.empty(Bt, ffn, dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty(Bt, dtype=torch.int32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_PREDICT, Bt, d, r, ffn)
    ws, wsb = workspace("predict_q4", x.device).get(nbytes)
    t = float(layer_q["tau"] if tau is None else tau)
    st = B.pi_ffn_predict_q4(_bits(x), Bt, d, layer_q["q_P1"], layer_q["s_P1"], layer_q.get("b1"), B.ACTS[act],
                             layer_q["q_P2"], layer_q["s_P2"], layer_q.get("b2"), r, ffn, int(n_hot), t, idx,
                             count, ws, wsb, stream)
    B.check(st, "pi_ffn_predict_q4")
    return idx, count


def sparse_q4(layer_q: dict, x: torch.Tensor, idx: Optional[torch.Tensor], count: Optional[torch.Tensor],
              y: Optional[torch.Tensor] = None, dense: bool = False, stream=None) -> torch.Tensor:
    """pi_ffn_sparse_q4 over a layer from quantize_layer."""
    Bt, d = x.shape
    ffn = layer_q["ffn"]
    if y is None:
        y = torch.empty(Bt, d, dtype=torch.float32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_SPARSE, Bt, d, layer_q.get("r", 8), ffn)
    ws, wsb = workspace("sparse_q4", x.device).get(nbytes)
    st = B.pi_ffn_sparse_q4(B.KINDS[layer_q["kind"]], _bits(x), Bt, d, ffn, layer_q["q_up"], layer_q["s_up"],
                            layer_q.get("b_up"), layer_q["q_gate"], layer_q["s_gate"], layer_q.get("b_gate"),
                            layer_q["q_down"], layer_q["s_down"], None if dense else idx,
                            None if dense else count, y, B.PI_DENSE if dense else 0, ws, wsb, stream)
    B.check(st, "pi_ffn_sparse_q4")
    return y


def decode(layer: dict, x: torch.Tensor, y: Optional[torch.Tensor] = None,
           idx: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
           act: str = "relu", tau: Optional[float] = None, per_token: bool = False,
           check_idx: bool = False, stream=None):
    """One decode step through pi_ffn_decode: the predicted list and the sparse
    FFN over it (one kernel for a single token).  Returns (y, idx, count)."""
    Bt, d = x.shape
    ffn, r = layer["ffn"], layer["r"]
    if y is None:
        y = torch.empty(Bt, d, dtype=torch.float32, device=x.device)
    if idx is None:
        idx = torch.empty(Bt, ffn, dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty(Bt, dtype=torch.int32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_DECODE, Bt, d, r, ffn)
    ws, wsb = workspace("decode", x.device).get(nbytes)
    st = B.pi_ffn_decode(B.KINDS[layer["kind"]], _bits(x), Bt, d, ffn, layer["P1"], layer.get("b1"),
                         B.ACTS[act], layer["P2"], layer.get("b2"), r,
                         float(layer["tau"] if tau is None else tau), layer["W_up"], layer.get("b_up"),
                         layer.get("W_gate"), layer.get("b_gate"), layer["W_down"], idx, count, y,
                         (B.PI_PER_TOKEN if per_token else 0) | (B.PI_CHECK_IDX if check_idx else 0),
                         ws, wsb, stream)
    B.check(st, "pi_ffn_decode")
    return y, idx, count


def decode_hot(layer: dict, x: torch.Tensor, n_hot: int, y: Optional[torch.Tensor] = None,
               idx: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
               act: str = "relu", tau: Optional[float] = None, per_token: bool = False,
               check_idx: bool = False, stream=None):
    """One decode step of a hot-first layer through pi_ffn_decode_hot: neurons
    [0, n_hot) always listed (their FFN computed beside the predictor for a
    single token), the rest predicted.  Returns (y, idx, count)."""
    Bt, d = x.shape
    ffn, r = layer["ffn"], layer["r"]
    if y is None:
        y = torch.empty(Bt, d, dtype=torch.float32, device=x.device)
    if idx is None:
        idx = torch.empty(Bt, ffn, dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty(Bt, dtype=torch.int32, device=x.device)
    nbytes = B.pi_workspace_size(B.PI_OP_DECODE_HOT, Bt, d, r, ffn)
    ws, wsb = workspace("decode_hot" if Bt == 1 else "decode_hot_batch", x.device).get(nbytes)
    st = B.pi_ffn_decode_hot(B.KINDS[layer["kind"]], _bits(x), Bt, d, ffn, layer["P1"], layer.get("b1"),
                             B.ACTS[act], layer["P2"], layer.get("b2"), r, int(n_hot),
                             float(layer["tau"] if tau is None else tau), layer["W_up"], layer.get("b_up"),
                             layer.get("W_gate"), layer.get("b_gate"), layer["W_down"], idx, count, y,
                             (B.PI_PER_TOKEN if per_token else 0) | (B.PI_CHECK_IDX if check_idx else 0),
                             ws, wsb, stream)
    B.check(st, "pi_ffn_decode_hot")
    return y, idx, count


def hot_workspace(layer: dict, device=None) -> torch.Tensor:
    """A fresh zero-filled workspace for the single-token hot decode of this
    layer's shape (for callers that keep one per layer)."""
    nbytes = B.pi_workspace_size(B.PI_OP_DECODE_HOT, 1, layer["d"], layer["r"], layer["ffn"])
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or layer["W_up"].device)


def decode_hot_begin(layer: dict, x: torch.Tensor, n_hot: int, idx: torch.Tensor, count: torch.Tensor,
                     ws: Optional[torch.Tensor] = None, act: str = "relu", tau: Optional[float] = None,
                     stream=None):
    """First launch of a single-token hot decode step (pi_ffn_decode_hot_begin):
    the list into idx / count and the hot prefix's FFN sum into the workspace."""
    d, ffn, r = layer["d"], layer["ffn"], layer["r"]
    if ws is None:
        ws, wsb = workspace("decode_hot", x.device).get(B.pi_workspace_size(B.PI_OP_DECODE_HOT, 1, d, r, ffn))
    else:
        wsb = ws.numel()
    st = B.pi_ffn_decode_hot_begin(B.KINDS[layer["kind"]], _bits(x), d, ffn, layer["P1"], layer.get("b1"), B.ACTS[act],
                                   layer["P2"], layer.get("b2"), r, int(n_hot),
                                   float(layer["tau"] if tau is None else tau), layer["W_up"], layer.get("b_up"),
                                   layer.get("W_gate"), layer.get("b_gate"), layer["W_down"], idx, count, ws, wsb,
                                   stream)
    B.check(st, "pi_ffn_decode_hot_begin")


def decode_hot_end(layer: dict, x: torch.Tensor, n_hot: int, idx: torch.Tensor, count: torch.Tensor,
                   y: torch.Tensor, ws: Optional[torch.Tensor] = None, check_idx: bool = False, stream=None):
    """Second launch (pi_ffn_decode_hot_end): the FFN over the list from n_hot on,
    plus the prefix's sum left by decode_hot_begin on the same workspace."""
    d, ffn, r = layer["d"], layer["ffn"], layer["r"]
    if ws is None:
        ws, wsb = workspace("decode_hot", x.device).get(B.pi_workspace_size(B.PI_OP_DECODE_HOT, 1, d, r, ffn))
    else:
        wsb = ws.numel()
    st = B.pi_ffn_decode_hot_end(B.KINDS[layer["kind"]], _bits(x), d, ffn, r, int(n_hot), layer["W_up"],
                                 layer.get("b_up"), layer.get("W_gate"), layer.get("b_gate"), layer["W_down"], idx,
                                 count, y, B.PI_CHECK_IDX if check_idx else 0, ws, wsb, stream)
    B.check(st, "pi_ffn_decode_hot_end")
    return y


# ---- the 8-bit paged cache.  A cache is a dict of device tensors named as in
# the C ABI (k and v: n_pages x n_kv x page x d bytes in the library's order,
# k_scale and v_scale: n_pages x n_kv floats) plus fmt ("int8" or "fp8"); a
# batch is a dict of the device arrays q_start, ctx and table (int32) plus the
# host's n_tok and max_q.


def kv_cache(n_pages: int, n_kv: int, d: int, page: int = 16, fmt: str = "int8", device="cuda") -> dict:
    """An empty cache.  Its memory is not initialised: no slot is read before it is written."""
    def bytes_():
        return torch.empty(n_pages, n_kv, page, d, dtype=torch.uint8, device=device)

    def scales():
        return torch.empty(n_pages, n_kv, dtype=torch.float32, device=device)

    return {"fmt": fmt, "k": bytes_(), "v": bytes_(), "k_scale": scales(), "v_scale": scales()}


def kv_batch(new, ctx, table, device="cuda") -> dict:
    """A batch from host lists: new[s] rows of the call for sequence s, ctx[s]
    its length with them, table[s] its page ids (rows may differ in length)."""
    start = [0]
    for n in new:
        start.append(start[-1] + int(n))
    width = max(1, max(len(r) for r in table))
    rows = [list(r) + [-1] * (width - len(r)) for r in table]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    return {"q_start": ints(start), "ctx": ints(list(ctx)), "table": ints(rows), "n_tok": start[-1],
            "max_q": max(int(n) for n in new)}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


_U8, _F16, _F32, _I32 = torch.uint8, torch.float16, torch.float32, torch.int32


def _kv_args(cache: dict, batch: dict, device: int):
    """The C descriptors of a cache and a batch on the GPU `device` (-1: the host)."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    start, ctx, table = batch["q_start"], batch["ctx"], batch["table"]
    fmt = B.KV_FMTS.get(cache["fmt"])
    shape, n_seq, rows = k.shape, ctx.shape, table.shape
    # one expression: this runs before every launch of a decode step
    if not (fmt is not None and len(shape) == 4 and v.shape == shape and k.dtype is _U8 and v.dtype is _U8
            and ks.shape == vs.shape == shape[:2] and ks.dtype is _F32 and vs.dtype is _F32
            and len(n_seq) == 1 and len(rows) == 2 and rows[0] == n_seq[0] and start.shape == (n_seq[0] + 1,)
            and start.dtype is _I32 and ctx.dtype is _I32 and table.dtype is _I32
            and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and start.is_contiguous() and ctx.is_contiguous() and table.is_contiguous()
            and k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == start.get_device()
            == ctx.get_device() == table.get_device() == device):
        raise ValueError("a cache is fmt ('int8' or 'fp8'), k and v (n_pages x n_kv x page x d uint8), k_scale and v_scale "
                         "(n_pages x n_kv float32); a batch is q_start (n_seq + 1), ctx (n_seq) and table (n_seq x pages), "
                         "int32, with n_tok and max_q; all contiguous and on one device")
    return (B.KvCache(fmt, shape[0], shape[1], shape[2], shape[3], k.data_ptr(), v.data_ptr(), ks.data_ptr(),
                      vs.data_ptr()),
            B.KvBatch(n_seq[0], batch["n_tok"], batch["max_q"], rows[1], start.data_ptr(), ctx.data_ptr(),
                      table.data_ptr()))


def _kv_rows(t: torch.Tensor, n_tok: int, heads: Optional[int], d: int, name: str, stride: bool = True) -> int:
    """Checks n_tok x heads x d fp16 rows; returns the elements between tokens."""
    shape = t.shape
    if not (t.dtype is _F16 and len(shape) == 3 and shape[0] == n_tok and shape[2] == d
            and (heads is None or shape[1] == heads)):
        raise ValueError(f"{name} must be fp16, n_tok x heads x d")
    if t.is_contiguous():
        return shape[1] * d
    if not (stride and (t.stride(2) == 1 or d == 1) and (t.stride(1) == d or shape[1] == 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous" if stride else f"{name} must be contiguous")
    return t.stride(0) if n_tok > 1 else shape[1] * d


# whether the current stream is being captured, and its handle, without making a torch.cuda.Stream of it
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _elsewhere(stream, device, tensors, call):
    """call() on another stream or device than the current ones: what it
    allocates belongs to that stream, and the caller's tensors are not reused
    by the allocator before that stream is done with them."""
    with torch.cuda.device(device):
        if stream is None:
            st = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            st = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        else:
            st = stream
        with torch.cuda.stream(st):
            out = call()
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(st)
        return out


def _is_elsewhere(stream, device: int) -> bool:
    if device < 0:
        raise ValueError("tensors must be on the GPU")
    return stream is not None or device != torch.cuda.current_device()


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, batch: dict, stream=None) -> None:
    """pi_kv_append: quantises k and v (n_tok x n_kv x d fp16, tokens any
    multiple of 8 elements apart) into the batch's places of the cache."""
    dev = k.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, k.device, (k, v, *cache.values(), *batch.values()),
                          lambda: kv_append(cache, k, v, batch))
    c, b = _kv_args(cache, batch, dev)
    ks = _kv_rows(k, b.n_tok, c.n_kv, c.d, "k")
    vs = _kv_rows(v, b.n_tok, c.n_kv, c.d, "v")
    _need(v.get_device() == dev, "k and v must be on one device")
    B.check(B.pi_kv_append(c, b, k, ks, v, vs, _raw_stream(dev)), "pi_kv_append")


def kv_read(cache: dict, batch: dict, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """pi_kv_read: the stored keys and values of the batch's tokens (n_tok x n_kv x d fp16)."""
    codes = cache["k"]
    dev = codes.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, codes.device, (k, v, *cache.values(), *batch.values()),
                          lambda: kv_read(cache, batch, k, v))
    c, b = _kv_args(cache, batch, dev)
    shape = (b.n_tok, c.n_kv, c.d)
    if k is None:
        k = torch.empty(shape, dtype=_F16, device=codes.device)
    else:
        _kv_rows(k, *shape, "k", stride=False)
        _need(k.get_device() == dev, "k must be on the cache's device")
    if v is None:
        v = torch.empty(shape, dtype=_F16, device=codes.device)
    else:
        _kv_rows(v, *shape, "v", stride=False)
        _need(v.get_device() == dev, "v must be on the cache's device")
    B.check(B.pi_kv_read(c, b, k, v, _raw_stream(dev)), "pi_kv_read")
    return k, v


_KV_WS: Dict[Tuple[int, int], Workspace] = {}


def kv_workspace(n_seq: int, n_tok: int, max_q: int, n_head: int, n_kv: int, d: int, device="cuda") -> torch.Tensor:
    """A fresh zero-filled workspace for kv_attend, for callers that keep their own."""
    nbytes = B.pi_kv_workspace_size(n_seq, n_tok, max_q, n_head, n_kv, d)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def kv_attend(cache: dict, q: torch.Tensor, batch: dict, y: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, window: int = 0, lse: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pi_kv_attend: attention of q (n_tok x n_head x d fp16, tokens any multiple
    of 8 elements apart) over the cache; scale defaults to 1 / sqrt(d), window 0
    is none, lse (n_tok x n_head floats) is filled if given.  Without ws, the
    eager calls of a stream share a workspace, and a call inside torch.cuda.graph
    has its own, allocated from the graph's pool and cleared in the capture (4 us
    a replay; a ws from kv_workspace, kept with the graph, saves them)."""
    dev = q.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, q.device, (q, y, lse, ws, *cache.values(), *batch.values()),
                          lambda: kv_attend(cache, q, batch, y, scale, window, lse, ws))
    c, b = _kv_args(cache, batch, dev)
    d = c.d
    qs = _kv_rows(q, b.n_tok, None, d, "q")
    heads = q.shape[1]
    if y is None:
        y = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _kv_rows(y, b.n_tok, heads, d, "y", stride=False)
        _need(y.get_device() == dev, "y must be on q's device")
    if lse is not None:
        _need(lse.shape == (b.n_tok, heads) and lse.dtype is _F32 and lse.is_contiguous()
              and lse.get_device() == dev, "lse must be n_tok x n_head floats")
    st = _raw_stream(dev)
    scale = d ** -0.5 if scale is None else float(scale)
    window = _window(window)
    ws, size, own = _attend_ws(ws, b, heads, c, q.device, dev, st)
    status = B.pi_kv_attend(c, b, q, qs, heads, scale, window, y, lse, ws, size, st)
    if status == B.PI_ERR_WORKSPACE and own is not None:   # too small for these sizes: nothing was launched
        ws, size = own.get(B.pi_kv_workspace_size(b.n_seq, b.n_tok, b.max_q, heads, c.n_kv, d))
        status = B.pi_kv_attend(c, b, q, qs, heads, scale, window, y, lse, ws, size, st)
    B.check(status, "pi_kv_attend")
    return y


def _window(window) -> int:
    return min(max(int(window), -1), 2 ** 31 - 1)   # (ctypes would drop what lies above 32 bits)


def _attend_ws(ws: Optional[torch.Tensor], b, heads: int, c, device, dev: int, st: int):
    """The caller's workspace or one of this module's, its bytes, and the keeper that can grow it if it is too small."""
    if ws is not None:
        _need(ws.get_device() == dev and ws.is_contiguous(), "ws must be contiguous and on q's device")
        return ws, ws.numel() * ws.element_size(), None
    if _capturing():
        # A graph's workspace is its alone: what other captures or eager calls on
        # this stream do is not replayed with it, and a kept buffer may be
        # replaced by a larger one.  The capture's pool holds the memory as long
        # as the graph lives and gives it to later allocations of the capture.
        size = B.pi_kv_workspace_size(b.n_seq, b.n_tok, b.max_q, heads, c.n_kv, c.d)
        ws = torch.empty(size, dtype=_U8, device=device)
        ws[:B.PI_KV_WS_ZERO_BYTES].zero_()
        return ws, size, None
    own = _KV_WS.get((dev, st))
    if own is None:
        own = _KV_WS[(dev, st)] = Workspace(device)
    buf = own.buf   # (read once: another thread may replace it by a larger one)
    return buf, 0 if buf is None else buf.numel(), own


def kv_tree(parents, device="cuda") -> dict:
    """From host lists, parents[s][j] the parent of row j of sequence s (-1: none; it
    lies before j): mask (n_tok x words int64, the bits of the C ABI's uint64), each row
    its ancestors and itself, parent and depth (n_tok int32)."""
    most = max(len(seq) for seq in parents)
    words = max(1, (most + 63) // 64)
    masks, depths = [], []
    for seq in parents:
        mine, depth = [], []
        for j, p in enumerate(seq):
            _need(-1 <= p < j, "a parent lies before its children")
            mine.append((mine[p] if p >= 0 else 0) | 1 << j)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        masks += [[(m >> 64 * w & (1 << 64) - 1) - (m >> 64 * w + 63 & 1) * (1 << 64) for w in range(words)] for m in mine]
        depths += depth
    return {"mask": torch.tensor(masks, dtype=torch.int64, device=device),
            "parent": torch.tensor([p for seq in parents for p in seq], dtype=_I32, device=device),
            "depth": torch.tensor(depths, dtype=_I32, device=device)}


def kv_attend_tree(cache: dict, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, batch: dict, mask: torch.Tensor,
                   pos: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   window: int = 0, lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """pi_kv_attend_tree: attention of drafted tokens, q (n_tok x n_head x d fp16),
    over the cache, whose lengths the batch's ctx are, and over each other, k and
    v (n_tok x n_kv x d fp16), as mask says (n_tok x words int64, kv_tree's).
    pos (n_tok int32) is needed under a window.  scale, y, lse and ws as kv_attend's."""
    dev = q.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, q.device, (q, k, v, mask, pos, y, lse, ws, *cache.values(), *batch.values()),
                          lambda: kv_attend_tree(cache, q, k, v, batch, mask, pos, y, scale, window, lse, ws))
    c, b = _kv_args(cache, batch, dev)
    d = c.d
    qs = _kv_rows(q, b.n_tok, None, d, "q")
    ks = _kv_rows(k, b.n_tok, c.n_kv, d, "k")
    vs = _kv_rows(v, b.n_tok, c.n_kv, d, "v")
    heads = q.shape[1]
    if not (mask.dtype is torch.int64 and mask.dim() == 2 and mask.shape[0] == b.n_tok and mask.is_contiguous()
            and k.get_device() == v.get_device() == mask.get_device() == dev
            and (pos is None or (pos.dtype is _I32 and pos.shape == (b.n_tok,) and pos.is_contiguous() and pos.get_device() == dev))):
        raise ValueError("mask is n_tok x words int64, pos n_tok int32; k, v, mask and pos on q's device")
    if y is None:
        y = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _kv_rows(y, b.n_tok, heads, d, "y", stride=False)
        _need(y.get_device() == dev, "y must be on q's device")
    if lse is not None:
        _need(lse.shape == (b.n_tok, heads) and lse.dtype is _F32 and lse.is_contiguous()
              and lse.get_device() == dev, "lse must be n_tok x n_head floats")
    st = _raw_stream(dev)
    scale = d ** -0.5 if scale is None else float(scale)
    window = _window(window)
    ws, size, own = _attend_ws(ws, b, heads, c, q.device, dev, st)
    words = mask.shape[1]
    status = B.pi_kv_attend_tree(c, b, q, qs, heads, k, ks, v, vs, mask, words, pos, scale, window, y, lse, ws, size, st)
    if status == B.PI_ERR_WORKSPACE and own is not None:
        ws, size = own.get(B.pi_kv_workspace_size(b.n_seq, b.n_tok, b.max_q, heads, c.n_kv, d))
        status = B.pi_kv_attend_tree(c, b, q, qs, heads, k, ks, v, vs, mask, words, pos, scale, window, y, lse, ws, size, st)
    B.check(status, "pi_kv_attend_tree")
    return y


# ---- rotary positions.  A plan is a dict: layout ("half" or "pairs"), rot, gain
# and turns (device, rot / 2 int64: the bits of the C ABI's uint64).


def rope(rot: int, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
         trained: float = 4096.0, slow: float = 1.0, fast: float = 32.0, freqs=None, gain: Optional[float] = None,
         device="cuda") -> dict:
    """A rotary plan for the first rot dimensions of a head: pi_rope_frequencies'
    (scaling "none", "linear", "ntk", "yarn", blended by each pair's turns as that
    method's paper words it, or "yarn-index", blended by the pair's number as the
    model code released with it does: what checkpoints stretched by that code
    need), or the caller's own freqs (rot / 2 radians a position) and gain, for
    a model stretched in any other way."""
    import numpy as np
    _need(layout in B.ROPE_LAYOUTS and scaling in B.ROPE_SCALINGS, "layout is 'half' or 'pairs', scaling 'none', 'linear', 'ntk', 'yarn' or 'yarn-index'")
    if freqs is None:
        freqs, own = B.pi_rope_frequencies(int(rot), float(base), B.ROPE_SCALINGS[scaling], float(factor), float(trained),
                                           float(slow), float(fast))
        gain = own if gain is None else gain
    freqs = np.asarray(freqs, dtype=np.float64)
    _need(freqs.shape == (rot // 2,), "freqs must be rot / 2 numbers")
    turns = torch.from_numpy(B.pi_rope_turns(freqs).view(np.int64)).to(device)
    return {"layout": layout, "rot": int(rot), "gain": 1.0 if gain is None else float(gain), "turns": turns}


def _rope_args(plan: dict, device: int):
    turns, layout, rot = plan["turns"], B.ROPE_LAYOUTS.get(plan["layout"]), plan["rot"]
    if not (layout is not None and turns.dtype is torch.int64 and turns.shape == (rot // 2,) and turns.is_contiguous()
            and turns.get_device() == device):
        raise ValueError("a rotary plan is layout ('half' or 'pairs'), rot, gain and turns (rot / 2 int64), on the tensors' device")
    return B.Rope(layout, rot, plan["gain"], turns.data_ptr())


def rotate(x: torch.Tensor, pos: torch.Tensor, plan: dict, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pi_rotate: x (n_tok x n_head x d fp16, tokens any multiple of 8 elements
    apart) turned by the positions pos (n_tok int32), into out (x itself: in place)."""
    dev = x.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, x.device, (x, pos, out, plan["turns"]), lambda: rotate(x, pos, plan, out))
    _need(x.dim() == 3, "x must be fp16, n_tok x heads x d")
    n, heads, d = x.shape
    xs = _kv_rows(x, n, heads, d, "x")
    _need(pos.dtype is _I32 and pos.shape == (n,) and pos.is_contiguous() and pos.get_device() == dev,
          "pos must be n_tok int32 on x's device")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ys = heads * d
    else:
        ys = _kv_rows(out, n, heads, d, "out")
        _need(out.get_device() == dev, "out must be on x's device")
    B.check(B.pi_rotate(_rope_args(plan, dev), pos, n, heads, d, x, xs, out, ys, _raw_stream(dev)), "pi_rotate")
    return out


def kv_append_rope(cache: dict, k: torch.Tensor, v: torch.Tensor, batch: dict, rope: Optional[dict] = None,
                   q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   rows: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """pi_kv_append_rope: kv_append with k turned by its cache positions (rope: a
    plan) on the way, and q (n_tok x n_head x d) by the same into q_out (q itself:
    in place), which is returned.  rows (n_tok int32): the batch's row i is row
    rows[i] of k and v, as verify gives them."""
    dev = k.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, k.device, (k, v, q, q_out, rows, rope["turns"] if rope else None, *cache.values(), *batch.values()),
                          lambda: kv_append_rope(cache, k, v, batch, rope, q, q_out, rows))
    c, b = _kv_args(cache, batch, dev)
    n_src = b.n_tok
    if rows is not None:
        _need(rows.dtype is _I32 and rows.shape == (b.n_tok,) and rows.is_contiguous() and rows.get_device() == dev,
              "rows must be n_tok int32 on k's device")
        n_src = k.shape[0]
    ks = _kv_rows(k, n_src, c.n_kv, c.d, "k")
    vs = _kv_rows(v, n_src, c.n_kv, c.d, "v")
    _need(v.get_device() == dev, "k and v must be on one device")
    plan = None if rope is None else _rope_args(rope, dev)
    qs = os_ = heads = 0
    if q is not None:
        qs = _kv_rows(q, b.n_tok, None, c.d, "q")
        heads = q.shape[1]
        _need(q.get_device() == dev, "q must be on k's device")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            os_ = heads * c.d
        else:
            os_ = _kv_rows(q_out, b.n_tok, heads, c.d, "q_out")
            _need(q_out.get_device() == dev, "q_out must be on k's device")
    else:
        _need(q_out is None, "q_out without q")
    B.check(B.pi_kv_append_rope(c, b, plan, rows, n_src, k, ks, v, vs, q, qs, heads, q_out, os_, _raw_stream(dev)),
            "pi_kv_append_rope")
    return q_out


# Of each host thread, by device and stream: pi_verify's second launch reads what its first left
# in the workspace, and another thread's call on the same stream may be queued between the two.
_VERIFY_WS = threading.local()
_verify_bytes = functools.lru_cache(maxsize=256)(B.pi_verify_workspace_size)


def verify(batch: dict, tokens: torch.Tensor, parent: torch.Tensor, p: torch.Tensor, u: torch.Tensor, u_next: torch.Tensor,
           q: Optional[torch.Tensor] = None, stream=None) -> dict:
    """pi_verify: which drafted tokens stay.  batch: q_start, ctx and n_tok of the
    rows; tokens and parent (n_tok int32); p and q (n_tok x vocab float32, rows
    any number of elements apart; q None: fixed proposals); u (n_tok float32) and
    u_next (n_seq).  Returns rows (n_tok int32, -1 behind the last), q_start, ctx
    and next: {**batch, **verify(...)} is the batch of the tokens that stay, whose
    rows kv_append_rope takes."""
    start, ctx, n_tok = batch["q_start"], batch["ctx"], batch["n_tok"]
    dev = p.get_device()
    if _is_elsewhere(stream, dev):
        return _elsewhere(stream, p.device, (start, ctx, tokens, parent, p, u, u_next, q),
                          lambda: verify(batch, tokens, parent, p, u, u_next, q))
    seqs, shape = ctx.shape, p.shape
    # one expression: this runs before every step of a serving loop
    if not (len(seqs) == 1 and len(shape) == 2 and shape[0] == n_tok and start.shape == (seqs[0] + 1,) and u_next.shape == seqs
            and tokens.shape == parent.shape == u.shape == (n_tok,)
            and start.dtype is _I32 and ctx.dtype is _I32 and tokens.dtype is _I32 and parent.dtype is _I32
            and p.dtype is _F32 and u.dtype is _F32 and u_next.dtype is _F32
            and start.is_contiguous() and ctx.is_contiguous() and tokens.is_contiguous() and parent.is_contiguous()
            and u.is_contiguous() and u_next.is_contiguous() and (p.stride(1) == 1 or shape[1] == 1)
            and start.get_device() == ctx.get_device() == tokens.get_device() == parent.get_device() == u.get_device()
            == u_next.get_device() == dev
            and (q is None or (q.shape == shape and q.dtype is _F32 and (q.stride(1) == 1 or shape[1] == 1) and q.get_device() == dev))):
        raise ValueError("q_start (n_seq + 1), ctx (n_seq), tokens and parent (n_tok) are int32, u (n_tok), u_next (n_seq), p and q "
                         "(n_tok x vocab, rows of neighbours) float32; all on one device")
    n_seq, vocab = seqs[0], shape[1]
    on, st = p.device, _raw_stream(dev)
    rows, new_start = torch.empty(n_tok, dtype=_I32, device=on), torch.empty(n_seq + 1, dtype=_I32, device=on)
    new_ctx, after = torch.empty(n_seq, dtype=_I32, device=on), torch.empty(n_seq, dtype=_I32, device=on)
    size = _verify_bytes(n_seq, n_tok, vocab)
    if _capturing():   # the graph's own, from its pool
        ws = torch.empty(size, dtype=_U8, device=on)
    else:              # a thread's calls on a stream share one: it holds nothing from call to call
        kept = _VERIFY_WS.__dict__
        ws = kept.get((dev, st))
        if ws is None or ws.numel() < size:
            ws = kept[(dev, st)] = torch.empty(size, dtype=_U8, device=on)
    B.check(B.pi_verify(n_seq, n_tok, vocab, start, ctx, tokens, parent, p, p.stride(0) if n_tok > 1 else vocab, q,
                        0 if q is None else q.stride(0) if n_tok > 1 else vocab, u, u_next, rows, new_start, new_ctx, after, ws,
                        size, st), "pi_verify")
    return {"rows": rows, "q_start": new_start, "ctx": new_ctx, "next": after}


def profile(X: torch.Tensor, W_fire: torch.Tensor, b_fire: Optional[torch.Tensor],
            counts: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    n, d = X.shape
    ffn = W_fire.shape[0]
    if counts is None:
        counts = torch.zeros(ffn, dtype=torch.int32, device=X.device)
    B.check(B.pi_profile(_bits(X), n, d, ffn, W_fire, b_fire, counts, None, 0, stream), "pi_profile")
    return counts


def reorder(counts_host, hot_share: float = 0.8):
    """Host plan: (perm int32 numpy new->old, hot_count)."""
    import numpy as np
    c = np.ascontiguousarray(np.asarray(counts_host, dtype=np.uint32))
    perm = np.empty(c.size, dtype=np.int32)
    hot = np.zeros(1, dtype=np.int32)
    B.check(B.pi_reorder(c, c.size, hot_share, perm, hot), "pi_reorder")
    return perm, int(hot[0])


def permute_rows(src: torch.Tensor, perm_dev: torch.Tensor, stream=None) -> torch.Tensor:
    dst = torch.empty_like(src)
    rows = src.shape[0]
    row_bytes = src[0].numel() * src.element_size() if src.dim() > 1 else src.element_size()
    B.check(B.pi_permute_rows(src, dst, rows, row_bytes, perm_dev, stream), "pi_permute_rows")
    return dst


ROW_KEYS = ("W_up", "W_gate", "W_down", "P2", "b_up", "b_gate", "b2")


def permute_layer(layer: dict, perm_dev: torch.Tensor, stream=None) -> dict:
    """Hot-first copy of a layer: every neuron-indexed tensor gathered by perm."""
    out = dict(layer)
    for k in ROW_KEYS:
        if layer.get(k) is not None:
            out[k] = permute_rows(layer[k], perm_dev, stream)
    return out


def to_device(layer: dict, device="cuda") -> dict:
    out = {}
    for k, v in layer.items():
        out[k] = v.to(device).contiguous() if isinstance(v, torch.Tensor) else v
    return out
