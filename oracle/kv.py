"""Oracle of the 8-bit paged cache and the attention over it (include/pi.h,
pi_kv_append / pi_kv_read / pi_kv_attend): plain numpy, a token and a block at
a time.  Codes and scales are rounded where the definition rounds them (fp32);
everything that is computed from stored values is in float64."""

import math

import numpy as np

QMAX = {"int8": 127.0, "fp8": 448.0}


def e4m3_values():
    """The 256 values of OCP e4m3: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; 0x7F and 0xFF are NaN, there are no infinities."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        mag = math.nan if b & 127 == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -mag if b & 128 else mag
    return out


_E4M3 = e4m3_values()
_POS = _E4M3[:127]   # ascending: 0 .. 448


def decode(byte, fmt):
    byte = np.asarray(byte, dtype=np.uint8)
    return byte.astype(np.float64) - 128.0 if fmt == "int8" else _E4M3[byte]


def encode(x, fmt):
    """Bytes of x rounded to the nearest code, ties to even, after clamping to +-QMAX."""
    x = np.clip(np.asarray(x, dtype=np.float64), -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return (np.rint(x) + 128).astype(np.uint8)
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, mag, side="left"), 0, 126)   # first code >= |x|
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - mag, mag - _POS[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (up == 0), hi, lo)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def places(page, d):
    """Byte of (token, dimension) inside a page and head, for K and for V: [page, d] each."""
    t = np.arange(page)[:, None]
    i = np.arange(d)[None, :]
    return t // 4 * 4 * d + i // 16 * 64 + t % 4 * 16 + i % 16, t // 16 * 16 * d + i * 16 + t % 16


def tokens(batch):
    """(sequence, row, position) of every row of the batch."""
    start, ctx = [int(v) for v in batch["q_start"]], [int(v) for v in batch["ctx"]]
    out = []
    for s in range(len(ctx)):
        n = start[s + 1] - start[s]
        out += [(s, start[s] + i, ctx[s] - n + i) for i in range(n)]
    return out


def append(cache, batch, k, v):
    """A copy of the cache (dict of numpy arrays, k and v: n_pages x n_kv x page x d bytes) with the rows written."""
    c = {n: (a.copy() if isinstance(a, np.ndarray) else a) for n, a in cache.items()}
    fmt = c["fmt"]
    n_pages, n_kv, page, d = c["k"].shape
    where = dict(zip("kv", places(page, d)))
    blocks = {}
    for s, row, p in tokens(batch):
        if p >= 0:
            blocks.setdefault((s, p // page), []).append((p % page, row))
    for (s, blk), rows in blocks.items():
        pid = int(batch["table"][s][blk])
        if not 0 <= pid < n_pages:
            continue
        first = min(t for t, _ in rows)
        for h in range(n_kv):
            for name, src in (("k", k), ("v", v)):
                flat = c[name][pid, h].reshape(-1)
                scale = c[name + "_scale"]
                new = np.stack([src[row, h] for _, row in rows]).astype(np.float32)
                s0 = scale[pid, h] if first > 0 else np.float32(0)
                m = np.float32(np.max(np.abs(new))) if np.all(np.isfinite(new)) else np.float32(np.nan)
                if not (np.isfinite(m) and np.isfinite(s0)):
                    s1 = np.float32(np.nan)
                else:
                    s1 = max(s0, m / np.float32(QMAX[fmt]))
                if s1 > s0 and first > 0:
                    r = s0 / s1
                    at = where[name][:first]
                    flat[at] = encode(decode(flat[at], fmt).astype(np.float32) * r, fmt)
                for (t, _), x in zip(rows, new):
                    flat[where[name][t]] = encode(x / s1 if s1 > 0 else np.zeros(d, np.float32), fmt)
                scale[pid, h] = s1
    return c


def stored(cache, table_row, p, name):
    """The stored values of position p: [n_kv, d] float64; NaN for a page that does not exist."""
    n_pages, n_kv, page, d = cache[name].shape
    pid = int(table_row[p // page])
    if not 0 <= pid < n_pages:
        return np.full((n_kv, d), np.nan)
    at = places(page, d)["kv".index(name)][p % page]
    return decode(cache[name][pid].reshape(n_kv, -1)[:, at], cache["fmt"]) * cache[name + "_scale"][pid].astype(np.float64)[:, None]


def read(cache, batch):
    """k and v, n_tok x n_kv x d float64 (before the rounding to fp16)."""
    n_tok, (_, n_kv, _, d) = int(batch["q_start"][-1]), cache["k"].shape
    out = {n: np.zeros((n_tok, n_kv, d)) for n in "kv"}
    for s, row, p in tokens(batch):
        if p >= 0:
            for n in "kv":
                out[n][row] = stored(cache, batch["table"][s], p, n)
    return out["k"], out["v"]


def attend(cache, batch, q, scale, window=0):
    """y and lse (float64), and the attention of |V| in the place of V, which
    bounds what an error of the weights can do to y."""
    n_tok, n_head, d = q.shape
    n_kv = cache["k"].shape[1]
    g = n_head // n_kv
    y, a, lse = np.zeros((n_tok, n_head, d)), np.zeros((n_tok, n_head, d)), np.full((n_tok, n_head), -np.inf)
    keep = {}
    for s, row, p in tokens(batch):
        if p < 0:
            continue
        if s not in keep:
            keep[s] = [np.stack([stored(cache, batch["table"][s], j, n) for j in range(int(batch["ctx"][s]))]) for n in "kv"]
        lo = max(0, p - window + 1) if window else 0
        kk, vv = (t[lo:p + 1].transpose(1, 0, 2) for t in keep[s])   # [n_kv, keys, d]
        x = np.einsum("hgd,hjd->hgj", q[row].astype(np.float64).reshape(n_kv, g, d), kk) * scale
        m = x.max(-1, keepdims=True)
        e = np.exp(x - m)
        l = e.sum(-1, keepdims=True)
        y[row] = (np.einsum("hgj,hjd->hgd", e, vv) / l).reshape(n_head, d)
        a[row] = (np.einsum("hgj,hjd->hgd", e, np.abs(vv)) / l).reshape(n_head, d)
        lse[row] = (m + np.log(l))[..., 0].reshape(n_head)
    return y, lse, a
