"""Oracle of rotary positions, of the cache's rotating append and of a step of
speculative decoding (include/pi.h: pi_rotate, pi_kv_append_rope,
pi_kv_attend_tree, pi_verify): plain numpy in float64, one row, block or token
at a time."""

import math
from fractions import Fraction

import numpy as np

from . import kv


def pairs(layout, rot):
    """The two dimensions of each pair."""
    m = np.arange(rot // 2)
    return (m, m + rot // 2) if layout == "half" else (2 * m, 2 * m + 1)


def turns(f):
    """f / (2 pi) mod 1 in units of 2^-64, to the nearest, from a double f: in rationals, pi from Machin's series."""
    one = 1 << 400

    def arctan_inverse(x):
        total, term, n = 0, one // x, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    tau = Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)
    units = Fraction(f) / tau * 2 ** 64
    return math.floor(units + Fraction(1, 2)) % 2 ** 64


def rotate(x, pos, freqs, layout="half", gain=1.0):
    """x (rows x heads x d) with its first 2 len(freqs) dimensions turned."""
    y = np.array(x, dtype=np.float64)
    a, b = pairs(layout, 2 * len(freqs))
    for i, p in enumerate(pos):
        t = int(p) * np.asarray(freqs, dtype=np.float64)
        c, s = np.cos(t), np.sin(t)
        xa, xb = y[i][:, a].copy(), y[i][:, b].copy()
        y[i][:, a] = gain * (xa * c - xb * s)
        y[i][:, b] = gain * (xb * c + xa * s)
    return y


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, trained=4096.0, slow=1.0, fast=32.0):
    """(radians a position of each pair, gain)"""
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    own = [base ** (-2 * m / rot) for m in range(rot // 2)]
    if scaling in ("none", "ntk"):
        return np.array(own), 1.0
    if scaling == "linear":
        return np.array([f / factor for f in own]), 1.0
    if scaling == "yarn-index":
        def pair(n):   # the (fractional) number of the pair that turns n times over the trained length: trained base^(-2 i / rot) = 2 pi n
            return rot / 2 * math.log(trained / (2 * math.pi * n), base) if n else rot
        a = max(0, math.floor(pair(fast)))
        b = max(a + 0.001, min(rot - 1, math.ceil(pair(slow))))
        blend = [f / factor + min(1.0, max(0.0, (b - m) / (b - a))) * (f - f / factor) for m, f in enumerate(own)]
        return np.array(blend), 0.1 * math.log(factor) + 1.0
    out = []
    for f in own:
        n = trained * f / (2 * math.pi)   # turns over the trained length
        c = 0.0 if n <= slow else 1.0 if n >= fast else (n - slow) / (fast - slow)
        out.append((1 - c) * f / factor + c * f)
    return np.array(out), 0.1 * math.log(factor) + 1.0


def left(P, q, x):
    """What a rejected child of token x leaves of distribution P (q None: a fixed proposal)."""
    if q is None:
        rest = P.copy()
        if 0 <= x < len(P):
            rest[x] = 0.0
    else:
        rest = np.maximum(P - q, 0.0)
    total = rest.sum()
    return rest / total if total > 0 else rest


def stays(P, q, x, u):
    if not 0 <= x < len(P):
        return False
    return u * (1.0 if q is None else q[x]) < P[x]


def choose(P, u):
    """The first token whose running sum passes u times the whole; -1 if there is nothing to choose from."""
    total = P.sum()
    if not (total > 0 and np.isfinite(total)):
        return -1
    run = np.cumsum(P)
    hit = np.nonzero(run > u * run[-1])[0]
    return int(hit[0]) if len(hit) else int(np.nonzero(P > 0)[0][-1])


def verify_one(tokens, parent, p, q, u, u_next):
    """(rows that stay, next token) of one sequence; p, q: rows x vocab (q None: fixed)."""
    path, cur = [0], 0
    while True:
        P = np.asarray(p[cur], dtype=np.float64)
        Q = None if q is None else np.asarray(q[cur], dtype=np.float64)
        for j in range(cur + 1, len(tokens)):
            if int(parent[j]) != cur:
                continue
            if stays(P, Q, int(tokens[j]), float(u[j])):
                break
            P = left(P, Q, int(tokens[j]))
        else:
            if P.sum() == 0:
                P = np.asarray(p[cur], dtype=np.float64)
            return path, choose(P, float(u_next))
        cur = j
        path.append(j)


def verify(q_start, ctx, tokens, parent, p, u, u_next, q=None):
    rows, start, new_ctx, nxt = [], [0], [], []
    for s in range(len(ctx)):
        a, e = int(q_start[s]), int(q_start[s + 1])
        if a == e:
            path, t = [], -1
        else:
            path, t = verify_one(tokens[a:e], parent[a:e], p[a:e], None if q is None else q[a:e], u[a:e], u_next[s])
        rows += [a + j for j in path]
        start.append(len(rows))
        new_ctx.append(int(ctx[s]) + len(path))
        nxt.append(t)
    return rows + [-1] * (len(tokens) - len(rows)), start, new_ctx, nxt


def bits(mask, n):
    """The rows a mask (uint64 words) names, below n."""
    return [j for j in range(n) if j // 64 < len(mask) and int(mask[j // 64]) >> (j % 64) & 1]


def attend_tree(cache, batch, q, k, v, mask, scale, window=0, pos=None):
    """y, lse and the attention of |V|, as kv.attend: over the cached tokens
    (under a window: positions above pos - window) and the rows that the mask names."""
    n_tok, n_head, d = q.shape
    n_kv = cache["k"].shape[1]
    g = n_head // n_kv
    start, ctx = [int(x) for x in batch["q_start"]], [int(x) for x in batch["ctx"]]
    y, a, lse = np.zeros((n_tok, n_head, d)), np.zeros((n_tok, n_head, d)), np.full((n_tok, n_head), -np.inf)
    for s, c in enumerate(ctx):
        if c:
            ck, cv = (np.stack([kv.stored(cache, batch["table"][s], j, n) for j in range(c)]) for n in "kv")
        else:
            ck = cv = np.zeros((0, n_kv, d))
        for row in range(start[s], start[s + 1]):
            lo = min(c, max(0, max(int(pos[row]), c) - window + 1)) if window else 0
            take = [start[s] + j for j in bits(mask[row], start[s + 1] - start[s])]
            kk = np.concatenate([ck[lo:], k[take].astype(np.float64)]).transpose(1, 0, 2)
            vv = np.concatenate([cv[lo:], v[take].astype(np.float64)]).transpose(1, 0, 2)
            if kk.shape[1] == 0:
                continue
            x = np.einsum("hgd,hjd->hgj", q[row].astype(np.float64).reshape(n_kv, g, d), kk) * scale
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            l = e.sum(-1, keepdims=True)
            y[row] = (np.einsum("hgj,hjd->hgd", e, vv) / l).reshape(n_head, d)
            a[row] = (np.einsum("hgj,hjd->hgd", e, np.abs(vv)) / l).reshape(n_head, d)
            lse[row] = (m + np.log(l))[..., 0].reshape(n_head)
    return y, lse, a
