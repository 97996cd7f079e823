"""Rotary positions and the cache's rotating append on the GPU against the
float64 oracle (oracle/draft.py, oracle/kv.py).

A turned pair (a, b): cosine and sine are within 2^-22 (polynomials 2^-23,
the angle's last bit 2^-29), their products with the gain and with a and b and the
sum round to 2^-24 each: the fp32 result is within 2^-21 gain (|a| + |b|).
As fp16 it is rounded once more, by at most 2^-11 of it, or 2^-25 below the
normal range.  As a code of scale s: to half a step, s / 2 for int8, for e4m3
2^-4 of it and 2^-10 s below the normal range, with 2^-16 s for the quotient's rounding
at a tie.  A scale moves by 2^-21 gain (|a| + |b|) / QMAX and one rounding of the quotient.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O
from oracle import kv as K
from tests.test_gpu_kv import DEV, garbage_cache, host, host_batch, tables

pytestmark = pytest.mark.gpu


def gains(x, rot, layout, gain):
    """gain (|a| + |b|) at every dimension, 0 where nothing is turned."""
    a, b = O.pairs(layout, rot)
    out = np.zeros(x.shape)
    both = gain * (np.abs(x[..., a].astype(np.float64)) + np.abs(x[..., b].astype(np.float64)))
    out[..., a] = out[..., b] = both
    return out


def near(got, want, x, rot, layout, gain):
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -21 * gains(x, rot, layout, gain)
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= tol), (np.max(err / tol), np.argmax(err / tol))
    assert np.array_equal(got[..., rot:], x[..., rot:], equal_nan=True)


def rows(rng, n, heads, d, stride=None):
    """n rows inside wider ones."""
    wide = torch.from_numpy(rng.standard_normal((n, stride or heads * d)).astype(np.float16)).to(DEV)
    return wide[:, :heads * d].unflatten(1, (heads, d))


SHAPES = [(1, 1, 8, 8), (1, 1, 8, 2), (3, 5, 64, 64), (7, 12, 64, 32), (2, 3, 80, 20), (65, 2, 80, 80), (9, 4, 96, 24), (5, 71, 128, 128),
          (4, 9, 128, 96), (33, 7, 256, 256), (2, 40, 256, 18), (3, 2, 24, 6), (2, 3, 40, 40)]


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("n,heads,d,rot", SHAPES)
def test_rotate(layout, n, heads, d, rot):
    rng = np.random.default_rng(n * d + rot)
    x = rows(rng, n, heads, d, heads * d + 8 * (n % 3))
    pos = rng.integers(-(1 << 20), 1 << 20, n).astype(np.int32)
    pos[0] = 0 if n > 1 else 777777
    gain = 1.25 if rot % 4 else 1.0
    plan = R.rope(rot, layout=layout, gain=gain, device=DEV)
    freqs, _ = O.frequencies(rot)
    want = O.rotate(x.cpu().numpy(), pos, freqs, layout, gain)
    at = torch.from_numpy(pos).to(DEV)
    wide = torch.full((n, heads * d + 16), 7.0, dtype=torch.float16, device=DEV)
    out = R.rotate(x, at, plan, out=wide[:, :heads * d].unflatten(1, (heads, d)))
    fresh = R.rotate(x, at, plan)
    kept = x.cpu().numpy()
    near(out.cpu().numpy(), want, kept, rot, layout, gain)
    assert torch.equal(out, fresh) and torch.all(wide[:, heads * d:] == 7.0)
    assert R.rotate(x, at, plan, out=x) is x and torch.equal(x, fresh)


@pytest.mark.parametrize("layout,heads,d,rot", [("half", 71, 64, 64), ("half", 5, 128, 96), ("half", 18, 80, 20), ("pairs", 9, 96, 24),
                                                ("pairs", 40, 256, 256)])
def test_rotate_many_rows(layout, heads, d, rot):
    """Enough rows that four heads share a thread's angles, the heads no multiple of four."""
    units = (d // 8 if layout == "pairs" else rot // 16 + (d - rot) // 8 if rot % 16 == 0 else d // 2)
    n = (1 << 19) // (heads * units) + 3
    rng = np.random.default_rng(heads)
    x = rows(rng, n, heads, d)
    pos = rng.integers(0, 1 << 17, n).astype(np.int32)
    plan = R.rope(rot, base=5e5, layout=layout, scaling="yarn", factor=4.0, device=DEV)
    freqs, gain = O.frequencies(rot, 5e5, "yarn", 4.0)
    got = R.rotate(x, torch.from_numpy(pos).to(DEV), plan)
    near(got.cpu().numpy(), O.rotate(x.cpu().numpy(), pos, freqs, layout, gain), x.cpu().numpy(), rot, layout, gain)
    few = R.rotate(x[:2], torch.from_numpy(pos[:2]).to(DEV), plan)
    assert torch.equal(few, got[:2])


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("heads,d,rot", [(18, 80, 20), (30, 128, 64), (33, 40, 40), (7, 128, 120)])
def test_rotate_many_rows_either_layout(layout, heads, d, rot):
    """Shared angles at every width of a thread's share: 16 dimensions, eight, one pair; in place too."""
    n = (1 << 18) // (heads * (d // 16)) + 5
    rng = np.random.default_rng(d + rot)
    x = rows(rng, n, heads, d, heads * d + 8)
    pos = rng.integers(-(1 << 30), 1 << 30, n).astype(np.int32)
    plan = R.rope(rot, layout=layout, device=DEV)
    freqs, gain = O.frequencies(rot)
    kept, at = x.cpu().numpy(), torch.from_numpy(pos).to(DEV)
    got = R.rotate(x, at, plan)
    near(got.cpu().numpy(), O.rotate(kept, pos, freqs, layout, gain), kept, rot, layout, gain)
    assert torch.equal(R.rotate(x, at, plan, out=x), got)


def test_far_positions_are_exact():
    """Angles of whole eighths of a turn at positions up to the type's ends."""
    freqs = 2 * np.pi * np.array([0.25, 0.125, 0.5, 0.375])
    plan = R.rope(8, freqs=freqs, layout="half", device=DEV)
    plan["turns"] = torch.tensor([1 << 62, 1 << 61, -(1 << 63), 3 << 61], dtype=torch.int64, device=DEV)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 5, -(2 ** 29) + 3, 123456789], dtype=np.int32)
    x = rows(np.random.default_rng(0), len(pos), 2, 8)
    small = (pos.astype(np.int64) % 8).astype(np.int32)
    want = O.rotate(x.cpu().numpy(), small, freqs)
    near(R.rotate(x, torch.from_numpy(pos).to(DEV), plan).cpu().numpy(), want, x.cpu().numpy(), 8, "half", 1.0)


def test_what_is_not_turned_is_copied_bit_for_bit():
    for layout, rot, d in (("half", 32, 64), ("half", 6, 64), ("pairs", 12, 64)):
        x = torch.zeros(3, 2, d, dtype=torch.float16, device=DEV)
        x.view(torch.int16)[..., rot:] = torch.randint(-32768, 32767, (3, 2, d - rot), device=DEV).to(torch.int16)
        plan = R.rope(rot, layout=layout, device=DEV)
        y = R.rotate(x, torch.arange(3, dtype=torch.int32, device=DEV), plan)
        assert torch.equal(y.view(torch.int16)[..., rot:], x.view(torch.int16)[..., rot:]) and torch.all(y[..., :rot] == 0)


def test_nonfinite_values_stay_in_their_pair():
    x = torch.ones(1, 1, 64, dtype=torch.float16, device=DEV)
    x[0, 0, 3] = float("inf")
    x[0, 0, 40] = float("nan")
    y = R.rotate(x, torch.tensor([5], dtype=torch.int32, device=DEV), R.rope(64, device=DEV))
    bad = ~torch.isfinite(y[0, 0])
    assert sorted(torch.nonzero(bad)[:, 0].tolist()) == [3, 8, 35, 40]


# ---------------------------------------------------------------- the append

def codes_near(cache, before, batch, k, rope, freqs, layout, gain):
    """K of the batch's blocks: scales, new codes, older codes, and everything else untouched."""
    fmt, (n_pages, n_kv, page, d) = cache["fmt"], cache["k"].shape
    at, q = K.places(page, d)[0], K.QMAX[fmt]
    rot = 0 if rope is None else rope["rot"]
    blocks = {}
    for s, row, p in K.tokens(batch):
        if p >= 0:
            blocks.setdefault((s, p // page), []).append((p, row))
    want = {n: before[n].copy() for n in ("k", "k_scale")}
    for (s, blk), got in blocks.items():
        pid, first = int(batch["table"][s][blk]), min(p for p, _ in got) % page
        x0 = np.stack([k[row] for _, row in got])
        x = O.rotate(x0, [p for p, _ in got], freqs, layout, gain) if rope is not None else x0.astype(np.float64)
        slack = 2.0 ** -21 * gains(x0, rot, layout, gain)
        for h in range(n_kv):
            s0 = float(before["k_scale"][pid, h]) if first else 0.0
            s1 = float(cache["k_scale"][pid, h])
            true = max(s0, np.abs(x[:, h]).max() / q)
            assert abs(s1 - true) <= slack[:, h].max() / q + 2.0 ** -23 * true, (s1, true)
            flat = cache["k"][pid, h].reshape(-1)
            for (p, _), xt, sl in zip(got, x[:, h], slack[:, h]):
                v = K.decode(flat[at[p % page]], fmt) * s1
                half = 0.5 * s1 if fmt == "int8" else 2.0 ** -4 * np.abs(xt) + 2.0 ** -10 * s1
                err = np.abs(v - xt)
                assert np.all(err <= half + 2.0 ** -16 * s1 + sl), np.max(err - half)
            w = want["k"][pid, h].reshape(-1)
            for p, _ in got:
                w[at[p % page]] = flat[at[p % page]]
            if first and s1 > s0:
                r = np.float32(s0) / np.float32(s1)
                w[at[:first]] = K.encode(K.decode(w[at[:first]], fmt).astype(np.float32) * r, fmt)
            want["k_scale"][pid, h] = cache["k_scale"][pid, h]
    assert np.array_equal(K.decode(cache["k"], fmt), K.decode(want["k"], fmt), equal_nan=True)
    assert np.array_equal(cache["k_scale"], want["k_scale"], equal_nan=True)


STEPS = {
    "prompt": [([37, 16, 1], [37, 16, 1])],
    "tokens": [([20, 3], [20, 3]), ([1, 1], [21, 4]), ([1, 0], [22, 4]), ([13, 14], [35, 18])],
    "unused": [([3, 2, 1], [1, 0, 7]), ([1, 1, 1], [0, 1, 8])],
}
PLANS = [("half", 128, 128, 16, 2), ("half", 64, 128, 16, 3), ("half", 32, 80, 32, 2), ("half", 64, 80, 64, 1), ("half", 20, 80, 16, 2),
         ("half", 16, 16, 16, 2), ("half", 96, 96, 128, 1), ("half", 256, 256, 256, 1), ("half", 256, 256, 128, 1), ("pairs", 128, 128, 16, 2),
         ("pairs", 24, 96, 32, 2), ("pairs", 2, 64, 64, 2), ("pairs", 256, 256, 256, 1), ("half", 48, 48, 256, 1), ("half", 34, 64, 64, 2)]


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("steps", sorted(STEPS))
@pytest.mark.parametrize("layout,rot,d,page,n_kv", PLANS)
def test_append_rope(fmt, steps, layout, rot, d, page, n_kv):
    """Call after call: K near the turned values, V exactly the oracle's, queries as rotate turns them."""
    rng = np.random.default_rng(rot + d + page)
    plan_steps = STEPS[steps]
    most = [max(ctx[s] for _, ctx in plan_steps) for s in range(len(plan_steps[0][1]))]
    table, n_pages = tables(most, page, rng)
    table = [r or [0] for r in table]
    cache = R.kv_cache(n_pages, n_kv, d, page, fmt, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(rng.integers(0, 126, cache[n].shape).astype(np.uint8)))
        cache[n + "_scale"].fill_(3.0)
    heads = 3 * n_kv
    plan = R.rope(rot, layout=layout, scaling="linear", factor=2.0, gain=1.5, device=DEV)
    freqs = O.frequencies(rot, scaling="linear", factor=2.0)[0]
    for i, (new, ctx) in enumerate(plan_steps):
        tok = sum(new)
        gain = 2.0 ** i * np.exp(rng.standard_normal((tok, 1)))
        wide = torch.from_numpy((rng.standard_normal((tok, (heads + 2 * n_kv) * d)) * gain).astype(np.float16)).to(DEV)
        q, k, v = (t.unflatten(1, (-1, d)) for t in wide.split([heads * d, n_kv * d, n_kv * d], 1))
        batch = R.kv_batch(new, ctx, table, DEV)
        hb, before = host_batch(batch), host({n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in cache.items()})
        want = K.append(before, hb, k.cpu().numpy(), v.cpu().numpy())
        pos = torch.tensor([p for _, _, p in K.tokens(hb)], dtype=torch.int32, device=DEV)
        turned = R.rotate(q, pos, plan)
        got = R.kv_append_rope(cache, k, v, batch, plan, q=q)
        assert torch.equal(got, turned)
        after = host(cache)
        codes_near(after, before, hb, k.cpu().numpy(), plan, freqs, layout, 1.5)
        assert np.array_equal(K.decode(after["v"], fmt), K.decode(want["v"], fmt)) and np.array_equal(after["v_scale"], want["v_scale"])
        kept = k.clone()
        assert R.kv_append_rope(cache, k, v, batch, plan, q=q, q_out=q) is q   # in place, beside the keys
        assert torch.equal(q, turned) and torch.equal(k, kept)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("page,d", [(16, 128), (64, 80), (256, 256)])
def test_append_listed_rows(fmt, page, d):
    """rows without a plan: exactly the append of the gathered rows; the list's tail is not read."""
    rng = np.random.default_rng(page)
    n_kv, ctx = 2, [30, 7, 5]
    table, n_pages = tables(ctx, page, rng)
    cache = garbage_cache(n_pages, n_kv, d, page, fmt)
    src = torch.from_numpy(rng.standard_normal((2, 50, n_kv, d)).astype(np.float16)).to(DEV)
    first = R.kv_batch([25, 7], [25, 7], [table[0], table[1]], DEV)
    R.kv_append(cache, src[0, :32], src[1, :32], first)
    before = host({n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in cache.items()})
    batch = R.kv_batch([5, 0, 3], ctx, table, DEV)
    take = [4, 9, 11, 12, 49, 20, 0, 21]
    batch.update(n_tok=20, max_q=5)   # as verify leaves it: fewer rows than the bound
    lst = torch.tensor(take + [-1] * 12, dtype=torch.int32, device=DEV)
    R.kv_append_rope(cache, src[0], src[1], batch, rows=lst)
    k, v = (src[i].cpu().numpy()[take] for i in (0, 1))
    want = K.append(before, host_batch(batch), k, v)
    got = host(cache)
    for n in ("k", "v"):
        assert np.array_equal(K.decode(got[n], fmt), K.decode(want[n], fmt), equal_nan=True)
        assert np.array_equal(got[n + "_scale"], want[n + "_scale"], equal_nan=True)
    # the same with a plan: as if the gathered rows had come themselves
    plan = R.rope(d, device=DEV)
    a, b = ({n: (torch.from_numpy(t).to(DEV) if isinstance(t, np.ndarray) else t) for n, t in before.items()} for _ in range(2))
    R.kv_append_rope(a, src[0], src[1], batch, plan, rows=lst)
    plain = R.kv_batch([5, 0, 3], ctx, table, DEV)
    R.kv_append_rope(b, src[0][take].contiguous(), src[1][take].contiguous(), plain, plan)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))


def test_rows_that_do_not_exist_make_their_block_nan():
    cache = garbage_cache(3, 1, 64, 16, "int8")
    src = torch.ones(4, 1, 64, dtype=torch.float16, device=DEV)
    batch = R.kv_batch([2, 1], [2, 1], [[0], [1]], DEV)
    for bad in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        R.kv_append_rope(cache, src, src, batch, rows=torch.tensor([0, bad, 3], dtype=torch.int32, device=DEV))
        k, v = R.kv_read(cache, batch)
        assert torch.all(torch.isnan(k[:2])) and torch.all(torch.isnan(v[:2]))
        assert torch.all((k[2] - 1).abs() < 2.0 ** -8) and torch.all((v[2] - 1).abs() < 2.0 ** -8)


def test_nonfinite_keys_make_their_block_nan_and_no_other():
    cache = garbage_cache(4, 2, 64, 16, "fp8")
    k = torch.ones(20, 2, 64, dtype=torch.float16, device=DEV)
    v = k.clone()
    k[17, 1, 5] = float("inf")
    batch = R.kv_batch([20], [20], [[2, 0]], DEV)
    R.kv_append_rope(cache, k, v, batch, R.rope(64, device=DEV))
    kk, vv = R.kv_read(cache, batch)
    bad = torch.isnan(kk)
    assert torch.all(bad[16:, 1]) and not torch.any(bad[:16]) and not torch.any(bad[:, 0]) and torch.all((vv - 1).abs() < 2.0 ** -4)


def test_queries_of_no_sequence_are_left():
    """q_start that ends before n_tok: the rows behind it keep what they hold."""
    cache = garbage_cache(4, 2, 64, 16, "int8")
    x = torch.randn(9, 2, 64, device=DEV).half()
    q = torch.randn(9, 4, 64, device=DEV).half()
    batch = R.kv_batch([3, 2], [3, 2], [[0], [1]], DEV)
    batch.update(n_tok=9, max_q=3)
    out = torch.full_like(q, 5.0)
    plan = R.rope(64, device=DEV)
    R.kv_append_rope(cache, x, x, batch, plan, q=q, q_out=out)
    assert torch.all(out[5:] == 5.0)
    pos = torch.tensor([0, 1, 2, 0, 1], dtype=torch.int32, device=DEV)
    assert torch.equal(out[:5], R.rotate(q[:5], pos, plan))


@pytest.mark.parametrize("n,heads,n_kv,d,rot,layout", [(600, 64, 8, 128, 128, "half"), (700, 30, 2, 64, 34, "half"), (900, 40, 1, 128, 24, "pairs")])
def test_queries_of_long_prompts(n, heads, n_kv, d, rot, layout):
    """Enough rows that four heads share a thread's angles."""
    ctx = [n, n // 2 + 5]
    table, n_pages = tables(ctx, 16, np.random.default_rng(0))
    cache = garbage_cache(n_pages, n_kv, d, 16, "int8")
    tok = sum(ctx)
    q, k = torch.randn(tok, heads, d, device=DEV).half(), torch.randn(tok, n_kv, d, device=DEV).half()
    plan = R.rope(rot, layout=layout, device=DEV)
    got = R.kv_append_rope(cache, k, k, R.kv_batch(ctx, ctx, table, DEV), plan, q=q)
    pos = torch.cat([torch.arange(c, dtype=torch.int32, device=DEV) for c in ctx])
    assert torch.equal(got, R.rotate(q, pos, plan))


def test_another_stream_and_a_captured_graph():
    rng = np.random.default_rng(2)
    ctx = [20, 5]
    table, n_pages = tables([40, 40], 16, rng)
    plan = R.rope(64, device=DEV)
    q, k, v = (torch.from_numpy(rng.standard_normal((2, h, 64)).astype(np.float16)).to(DEV) for h in (4, 2, 2))
    old = torch.from_numpy(rng.standard_normal((25, 2, 64)).astype(np.float16)).to(DEV)
    caches = [garbage_cache(n_pages, 2, 64, 16, "int8") for _ in range(2)]
    for c in caches:
        for n in ("k", "v"):
            c[n].zero_()
        R.kv_append_rope(c, old, old, R.kv_batch(ctx, ctx, table, DEV), plan)
    batch = R.kv_batch([1, 1], [21, 6], table, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    R.kv_append_rope(caches[1], k, v, batch, plan, q=q, stream=side)   # warm, elsewhere
    torch.cuda.synchronize()
    R.kv_append_rope(caches[0], k, v, batch, plan, q=q)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.kv_append_rope(caches[1], k, v, batch, plan, q=q, q_out=out)
        turned = R.rotate(q, batch["ctx"], plan)
    for step in range(3):
        batch["ctx"].copy_(torch.tensor([22 + step, 7 + step], dtype=torch.int32))
        want = R.kv_append_rope(caches[0], k, v, batch, plan, q=q)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(turned, R.rotate(q, batch["ctx"], plan))
        for n in ("k", "v"):
            assert torch.equal(caches[0][n], caches[1][n])
