"""The 8-bit paged cache on the GPU against the float64 oracle (oracle/kv.py).

Codes and scales are compared exactly (a code as the number it stands for),
read values as fp16 of the oracle's.  Attention's bound follows from its
arithmetic.  With A the attention of |V| (the oracle's third result):
  output rounding     2^-11 |y|, and 2^-25 below fp16's normal range
  weights in fp16     2^-11 A      (not on every path, allowed on all)
  fp32 scores         an error e in x changes a weight by e: 2 e A for the
                      weight and the sum; e <= (d + 8) 2^-24 max sum|q_i k_i| scale,
                      which the inputs here keep under 2^-12: 2^-11 A
  exponentials, sums  under 2^-12 A
together under 2^-11 |y| + 1.25 2^-10 A + 2^-25.  lse: e and rounding, 2^-11 + 2^-21 |lse|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R
from oracle import kv as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def host(cache):
    return {n: (t.cpu().numpy() if isinstance(t, torch.Tensor) else t) for n, t in cache.items()}


def host_batch(batch):
    return {n: (t.cpu().numpy() if isinstance(t, torch.Tensor) else t) for n, t in batch.items()}


def tables(ctx, page, rng, spare=2):
    """Page ids in no order for sequences of these lengths, and the pool's size."""
    need = [-(-c // page) for c in ctx]
    ids = rng.permutation(sum(need) + spare)
    rows, at = [], 0
    for n in need:
        rows.append([int(i) for i in ids[at:at + n]])
        at += n
    return rows, sum(need) + spare


def garbage_cache(n_pages, n_kv, d, page, fmt):
    """Memory as an allocator may hand it out: NaN codes (fp8) and NaN scales everywhere."""
    c = R.kv_cache(n_pages, n_kv, d, page, fmt, DEV)
    for n in ("k", "v"):
        c[n].fill_(0xFF)
        c[n + "_scale"].fill_(float("nan"))
    return c


def filled(ctx, n_kv, d, page, fmt, seed=0, v_gain=None):
    """A cache whose sequences were appended whole, and its table."""
    rng = np.random.default_rng(seed)
    rows, n_pages = tables(ctx, page, rng)
    c = garbage_cache(n_pages, n_kv, d, page, fmt)
    tok = sum(ctx)
    k = torch.from_numpy(rng.standard_normal((tok, n_kv, d)).astype(np.float16)).to(DEV)
    v = rng.standard_normal((tok, n_kv, d))
    if v_gain is not None:
        v = v * v_gain(rng, tok)[:, None, None]
    v = torch.from_numpy(v.astype(np.float16)).to(DEV)
    live = [s for s, x in enumerate(ctx) if x]
    R.kv_append(c, k, v, R.kv_batch([ctx[s] for s in live], [ctx[s] for s in live], [rows[s] for s in live], DEV))
    return c, rows


def same_codes(got, want, touched=None):
    for n in ("k", "v"):
        g, w = O.decode(got[n], got["fmt"]), O.decode(want[n], got["fmt"])
        assert np.array_equal(g, w, equal_nan=True), f"{n}: {np.sum(g != w)} codes differ"
        assert np.array_equal(got[n + "_scale"], want[n + "_scale"], equal_nan=True), f"{n}_scale"


STEPS = {
    "prompt": [([37, 16, 1, 0], [37, 16, 1, 5])],
    "tokens": [([20, 3], [20, 3]), ([1, 1], [21, 4]), ([1, 1], [22, 5]), ([1, 0], [23, 5]), ([12, 14], [35, 19])],
    "unused": [([3, 2, 1], [1, 0, 7]), ([1, 1, 1], [0, 1, 8])],
}


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("page,d,n_kv", [(16, 128, 3), (16, 16, 1), (16, 256, 2), (32, 80, 2), (64, 64, 2), (64, 144, 1), (128, 128, 1),
                                         (256, 128, 1), (256, 256, 1)])
@pytest.mark.parametrize("steps", sorted(STEPS))
def test_append_exact(fmt, page, d, n_kv, steps):
    """Every byte of the pool and every scale, call after call, the older codes
    rounded again as the values grow; slots that are not written keep what they hold."""
    rng = np.random.default_rng(page + d)
    plan = STEPS[steps]
    most = [max(ctx[s] for _, ctx in plan) for s in range(len(plan[0][1]))]
    rows, n_pages = tables(most, page, rng)
    rows = [r or [0] for r in rows]
    cache = R.kv_cache(n_pages, n_kv, d, page, fmt, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(rng.integers(0, 126, cache[n].shape).astype(np.uint8)))
        cache[n + "_scale"].fill_(3.0)
    for i, (new, ctx) in enumerate(plan):
        tok = sum(new)
        gain = 2.0 ** i * np.exp(rng.standard_normal((tok, 1, 1)))
        # slices of one projection's rows: q, k and v side by side
        wide = np.zeros((tok, 3 * n_kv * d), np.float16)
        wide[:, n_kv * d:] = (rng.standard_normal((tok, 2, n_kv * d)) * gain).reshape(tok, -1)
        on = torch.from_numpy(wide).to(DEV)
        k, v = (on[:, j * n_kv * d:(j + 1) * n_kv * d].view(tok, n_kv, d) for j in (1, 2))
        batch = R.kv_batch(new, ctx, rows, DEV)
        want = O.append(host(cache), host_batch(batch), k.cpu().numpy(), v.cpu().numpy())
        R.kv_append(cache, k, v, batch)
        torch.cuda.synchronize()
        same_codes(host(cache), want)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_append_rounding_of_many_values(fmt):
    """The quotient's rounding over every finite fp16 number and many scales:
    blocks whose largest value is set, filled with all the numbers below it."""
    n_kv, d, page = 1, 256, 256
    every = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    rng = np.random.default_rng(1)
    tops = np.concatenate([every[[1, 2, 3, 0x3FF, 0x400, 0x7BFF]], rng.choice(every[1:], 40)])
    n = len(tops)
    x = np.zeros((n * page, n_kv, d), np.float16)
    for i, top in enumerate(tops):
        below = every[every <= top]
        vals = rng.choice(below, page * d) * rng.choice(np.array([-1, 1], np.float16), page * d)
        vals[0] = top
        x[i * page:(i + 1) * page, 0] = vals.reshape(page, d)
    cache = garbage_cache(n, n_kv, d, page, fmt)
    batch = R.kv_batch([n * page], [n * page], [list(range(n))], DEV)
    xd = torch.from_numpy(x).to(DEV)
    R.kv_append(cache, xd, xd, batch)
    torch.cuda.synchronize()
    got = host(cache)
    at = dict(zip("kv", O.places(page, d)))
    for i in range(n):
        s = np.float32(tops[i]) / np.float32(O.QMAX[fmt])
        want = O.decode(O.encode(x[i * page:(i + 1) * page, 0].astype(np.float32) / s, fmt), fmt)
        for m in ("k", "v"):
            assert got[m + "_scale"][i, 0] == s
            assert np.array_equal(O.decode(got[m][i, 0].reshape(-1)[at[m]], fmt), want), (m, float(tops[i]))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_append_zero_and_nonfinite(fmt):
    """Zero blocks have scale 0 and read as 0; infinity or NaN makes its own
    block, head and matrix NaN until the block is written from its start again."""
    n_kv, d, page = 2, 64, 16
    cache = garbage_cache(3, n_kv, d, page, fmt)
    rows = [[2, 0]]
    k = torch.zeros(20, n_kv, d, dtype=torch.float16, device=DEV)
    v = torch.ones_like(k)
    k[3, 1, 5], v[17, 0, 0] = float("inf"), float("nan")
    whole = R.kv_batch([20], [20], rows, DEV)
    steps = [(whole, k, v), (R.kv_batch([1], [21], rows, DEV), v[:1], v[:1]), (whole, v.nan_to_num(1.0), v.nan_to_num(1.0))]
    for batch, kk, vv in steps:
        kk, vv = kk.contiguous(), vv.contiguous()
        want = O.append(host(cache), host_batch(batch), kk.cpu().numpy(), vv.cpu().numpy())
        R.kv_append(cache, kk, vv, batch)
        torch.cuda.synchronize()
        same_codes(host(cache), want)
        gk, gv = R.kv_read(cache, batch)
        ok, ov = O.read(want, host_batch(batch))
        assert np.array_equal(gk.cpu().numpy(), ok.astype(np.float16), equal_nan=True)
        assert np.array_equal(gv.cpu().numpy(), ov.astype(np.float16), equal_nan=True)


def test_append_leaves_bad_pages_alone():
    """Page ids outside the pool are not written; others of the same call are."""
    cache = R.kv_cache(2, 1, 64, 16, "int8", DEV)
    for n in ("k", "v"):
        cache[n].fill_(9)
        cache[n + "_scale"].fill_(2.0)
    x = torch.randn(40, 1, 64, device=DEV).half()
    batch = R.kv_batch([40], [40], [[-1, 1, 2]], DEV)
    want = O.append(host(cache), host_batch(batch), x.cpu().numpy(), x.cpu().numpy())
    R.kv_append(cache, x, x, batch)
    gk, gv = R.kv_read(cache, batch)
    torch.cuda.synchronize()
    same_codes(host(cache), want)
    ok, _ = O.read(want, host_batch(batch))
    assert np.array_equal(gk.cpu().numpy(), ok.astype(np.float16), equal_nan=True)
    assert torch.isnan(gv[:16]).all() and not torch.isnan(gv[16:32]).any() and torch.isnan(gv[32:]).all()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("page,d,n_kv", [(16, 128, 2), (32, 80, 3), (64, 16, 1), (128, 256, 1)])
def test_read_exact(fmt, page, d, n_kv):
    """Whole sequences, their newest tokens from inside a page, one token, none,
    and rows before position 0."""
    ctx = [70, 16, 1, 0, 33]
    cache, rows = filled(ctx, n_kv, d, page, fmt, seed=3)
    H = host(cache)
    for new in (ctx[:3] + [2] + ctx[4:], [5, 1, 0, 1, 18], [75, 20, 1, 0, 33], [0, 0, 1, 0, 0]):
        batch = R.kv_batch(new, ctx, rows, DEV)
        k, v = R.kv_read(cache, batch)
        torch.cuda.synchronize()
        ok, ov = O.read(H, host_batch(batch))
        assert np.array_equal(k.cpu().numpy(), ok.astype(np.float16))
        assert np.array_equal(v.cpu().numpy(), ov.astype(np.float16))


def check_attend(cache, batch, q, scale=None, window=0, lse=True, **kw):
    d = q.shape[2]
    sc = d ** -0.5 if scale is None else scale
    got_lse = torch.full(q.shape[:2], 77.0, device=DEV) if lse else None
    y = R.kv_attend(cache, q, batch, scale=scale, window=window, lse=got_lse, **kw)
    torch.cuda.synchronize()
    want, want_lse, a = O.attend(host(cache), host_batch(batch), q.cpu().numpy(), sc, window)
    g = y.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(want)), "NaN in other places"
    ok = ~np.isnan(want)
    tol = 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * a + 2.0 ** -25
    worst = np.max((np.abs(g - want) / tol)[ok], initial=0.0)
    assert worst <= 1.0, f"{worst:.2f} times the bound"
    if lse:
        gl = got_lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(gl), np.isneginf(want_lse))
        f = np.isfinite(want_lse)
        assert np.array_equal(f | np.isneginf(want_lse), ~np.isnan(gl))
        assert np.all(np.abs(gl - want_lse)[f] <= 2.0 ** -11 + 2.0 ** -21 * np.abs(want_lse[f]))
    return y


def queries(n, heads, d, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, d, generator=g).half().to(DEV)


HEADS = [(1, 1), (4, 4), (8, 1), (15, 5), (16, 1), (71, 1), (6, 2)]


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv", HEADS)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 64), (80, 32), (16, 16), (256, 128), (208, 16), (128, 256)])
def test_attend_single_tokens(fmt, heads, n_kv, d, page):
    """One token of each sequence: lengths 0, 1, and around the granule, page and tile ends."""
    ctx = [1, 0, 15, 16, 17, 63, 64, 65, 130, 257]
    cache, rows = filled(ctx, n_kv, d, page, fmt, seed=d)
    check_attend(cache, R.kv_batch([1] * len(ctx), ctx, rows, DEV), queries(len(ctx), heads, d))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d,page", [(4, 4, 128, 16), (8, 1, 64, 32), (6, 2, 80, 16), (16, 1, 128, 64), (3, 1, 256, 16),
                                               (2, 2, 16, 16), (5, 5, 128, 32)])
@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("new", [[3, 1, 0, 5, 2], [9, 17, 1, 33, 4], [130, 1, 2, 64, 7], [40, 300, 0, 1, 129]])
def test_attend_rows(fmt, heads, n_kv, d, page, window, new):
    """Several rows of a sequence at once, decoding beside prompts, rows before
    position 0, windows that end inside tiles."""
    ctx = [131, 300, 1, 65, 140]
    cache, rows = filled(ctx, n_kv, d, page, fmt, seed=7)
    check_attend(cache, R.kv_batch(new, ctx, rows, DEV), queries(sum(new), heads, d), window=window)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,d", [(1, 1, 128), (8, 2, 64), (2, 1, 256)])
def test_attend_long_split(fmt, heads, n_kv, d):
    """Contexts long enough to be split over many workgroups and joined, beside short ones."""
    ctx = [9001, 40, 4096, 1]
    cache, rows = filled(ctx, n_kv, d, 64, fmt, seed=8)
    q = queries(4, heads, d)
    check_attend(cache, R.kv_batch([1, 1, 1, 1], ctx, rows, DEV), q)
    check_attend(cache, R.kv_batch([1, 1, 1, 1], ctx, rows, DEV), q, window=3000)
    check_attend(cache, R.kv_batch([3, 1, 40, 0], ctx, rows, DEV), queries(44, heads, d), window=5000)


def test_attend_prompt_split():
    """A few rows' worth of prompt over a long context: row tiles split over the context too."""
    ctx = [6000]
    cache, rows = filled(ctx, 1, 128, 16, "int8", seed=9)
    check_attend(cache, R.kv_batch([150], ctx, rows, DEV), queries(150, 1, 128))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_scales_far_apart(fmt, n):
    """Blocks whose values differ by 2^20, the large ones with the small weights
    and the other way round, and blocks of zeros."""
    def gain(rng, tok):
        return np.where(np.arange(tok) // 16 % 5 == 4, 0.0, 2.0 ** (np.arange(tok) // 16 % 3 * 10 - 14))
    ctx = [400]
    cache, rows = filled(ctx, 2, 64, 16, fmt, seed=10, v_gain=gain)
    batch = R.kv_batch([n], ctx, rows, DEV)
    check_attend(cache, batch, queries(n, 4, 64))
    check_attend(cache, batch, queries(n, 4, 64) * 8, scale=0.0625)


@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_only_zero_values_and_far_scores(n):
    """All V zero; and scores hundreds apart, so that nearly every weight underflows."""
    ctx = [300]
    cache, rows = filled(ctx, 1, 64, 16, "int8", seed=11, v_gain=lambda rng, tok: np.zeros(tok))
    batch = R.kv_batch([n], ctx, rows, DEV)
    y = check_attend(cache, batch, queries(n, 2, 64))
    assert not torch.any(y)
    cache, rows = filled(ctx, 1, 64, 16, "int8", seed=12, v_gain=lambda rng, tok: 2.0 ** rng.integers(-14, 10, tok))
    # whole numbers: the scores are exact in fp32 up to the block's scale
    q = torch.randint(-60, 61, (n, 2, 64), generator=torch.Generator().manual_seed(2)).half().to(DEV)
    check_attend(cache, R.kv_batch([n], ctx, rows, DEV), q * 0.25, scale=0.5)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_ignores_what_is_masked(fmt, n):
    """NaN codes and scales in the slots behind the context, in pages outside a
    window and in pages after a row's position change nothing, bit for bit."""
    ctx, page, d = [245], 16, 64
    cache, rows = filled(ctx, 2, d, page, fmt, seed=13)
    q = queries(n, 4, d)
    batch = R.kv_batch([n], ctx, rows, DEV)
    window = 40
    y0 = check_attend(cache, batch, q, window=window)
    first = ctx[0] - n - window + 1          # the first position that any row sees
    for s in rows[0][:max(0, first) // page]:
        for m in ("k", "v"):
            cache[m][s] = 0xFF
            cache[m + "_scale"][s] = float("nan")
    y1 = R.kv_attend(cache, q, batch, window=window)
    # the last page's slots behind the context were garbage from the start; other garbage there
    kp, vp = O.places(page, d)
    tail = ctx[0] % page
    last = rows[0][-1]
    for m, at in (("k", kp), ("v", vp)):
        flat = cache[m][last].view(2, -1)
        flat[:, torch.from_numpy(at[tail:].reshape(-1)).to(DEV)] = 0x7F
    y2 = R.kv_attend(cache, q, batch, window=window)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2)


@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_poisoned_block_reaches_only_its_readers(n):
    """A block with a NaN scale (and a page id outside the pool) makes NaN of
    the rows and heads that attend to it, and of no others."""
    ctx, page, d = [200, 50], 16, 64
    cache, rows = filled(ctx, 2, d, page, "int8", seed=14)
    blk = (200 - n // 2) // page
    cache["v_scale"][rows[0][blk], 1] = float("nan")
    q = queries(n + 1, 4, d)
    check_attend(cache, R.kv_batch([n, 1], ctx, rows, DEV), q, window=33, lse=False)
    rows[1][1] = 10 ** 6
    check_attend(cache, R.kv_batch([n, 1], ctx, rows, DEV), q, window=33, lse=False)
    rows[1][1] = -5
    check_attend(cache, R.kv_batch([n, 1], ctx, rows, DEV), q, window=2, lse=False)


@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_nonfinite_query_is_its_own(n):
    cache, rows = filled([120], 1, 64, 16, "int8", seed=15)
    q = queries(n, 3, 64)
    batch = R.kv_batch([n], [120], rows, DEV)
    y0 = R.kv_attend(cache, q, batch)
    q2 = q.clone()
    q2[n // 2, 1, 7] = float("nan")
    y1 = R.kv_attend(cache, q2, batch)
    q2[n // 2, 1, 7] = float("inf")
    y2 = R.kv_attend(cache, q2, batch)
    torch.cuda.synchronize()
    for y in (y1, y2):
        assert torch.isnan(y[n // 2, 1]).all()
        y[n // 2, 1] = y0[n // 2, 1]
        assert torch.equal(y, y0)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 1, 3], [70, 1, 20]])
def test_attend_repeats_bitwise_with_strided_queries_and_own_buffers(new):
    ctx = [3000, 17, 400]
    cache, rows = filled(ctx, 2, 128, 16, "int8", seed=16)
    batch = R.kv_batch(new, ctx, rows, DEV)
    tok = sum(new)
    wide = torch.randn(tok, 5, 4 * 128, device=DEV).half()
    q = wide[:, 1].view(tok, 4, 128)
    assert q.stride(0) == 5 * 512
    y0 = check_attend(cache, batch, q.contiguous())
    y = torch.full((tok, 4, 128), float("nan"), dtype=torch.float16, device=DEV)
    ws = R.kv_workspace(3, tok, max(new), 4, 2, 128, DEV)
    for _ in range(3):
        assert R.kv_attend(cache, q, batch, y=y, ws=ws) is y
        torch.cuda.synchronize()
        assert torch.equal(y, y0)


def test_attend_shares_a_workspace_with_the_other_calls():
    """One workspace through the FFN and attention calls of other shapes, in turn."""
    from synthetic import custom_config, make_layer, make_tokens
    cfg = custom_config("relu", 256, 1000, 64, mean=0.2, number=120)
    L = R.to_device(make_layer(cfg), DEV)
    x = make_tokens(cfg, 1).to(DEV)
    ctx = [5000, 100]
    cases = []
    for heads, d, n in ((8, 64, [1, 1]), (2, 128, [4, 60])):
        cache, rows = filled(ctx, 2, d, 16, "int8", seed=17)
        cases.append((cache, R.kv_batch(n, ctx, rows, DEV), queries(sum(n), heads, d)))
    want = [R.kv_attend(c, q, b) for c, b, q in cases]
    y, idx, cnt = R.decode(L, x)
    need = max([B.pi_workspace_size(B.PI_OP_DECODE, 1, cfg.d, cfg.r, cfg.ffn)]
               + [B.pi_kv_workspace_size(2, q.shape[0], b["max_q"], q.shape[1], 2, q.shape[2]) for _, b, q in cases])
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for (c, b, q), w in zip(cases, want):
            assert torch.equal(R.kv_attend(c, q, b, ws=ws), w)
            y2 = torch.empty_like(y)
            i2, c2 = torch.empty_like(idx), torch.empty_like(cnt)
            B.check(B.pi_ffn_decode(B.PI_FFN_RELU, x, 1, cfg.d, cfg.ffn, L["P1"], None, B.PI_ACT_RELU, L["P2"], L["b2"],
                                    cfg.r, 0.5, L["W_up"], L["b_up"], None, None, L["W_down"], i2, c2, y2, 0, ws,
                                    ws.numel()), "pi_ffn_decode")
            assert torch.equal(y, y2)


def test_other_stream():
    """The calls on a stream that is not the current one, as a torch stream and
    as a handle, with temporaries freed at once by the caller."""
    ctx = [2000, 33]
    cache, rows = filled(ctx, 2, 128, 16, "fp8", seed=18)
    batch = R.kv_batch([1, 1], ctx, rows, DEV)
    q = queries(2, 8, 128)
    want, (wk, wv) = R.kv_attend(cache, q, batch), R.kv_read(cache, batch)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for s in (st, st.cuda_stream):
        for _ in range(3):
            tmp = q.clone()
            torch.cuda.current_stream().synchronize()
            y = R.kv_attend(cache, tmp, batch, stream=s)
            del tmp
            torch.empty(2, 8, 128, dtype=torch.float16, device=DEV).fill_(float("nan"))
            k, v = R.kv_read(cache, batch, stream=s)
            R.kv_append(cache, wk, wv, batch, stream=s)
            st.synchronize()
            assert torch.equal(y, want) and torch.equal(k, wk) and torch.equal(v, wv)


def test_graph_replays_as_the_lengths_grow():
    """One decode step (append, then attention) captured once and replayed with
    the lengths advanced on the device, against the eager calls; eager work of
    the same kind on its own workspace in between."""
    page, n_kv, heads, d, fmt = 16, 2, 8, 64, "int8"
    start = [30, 700, 0]
    most = [x + 20 for x in start]
    rng = np.random.default_rng(19)
    rows, n_pages = tables(most, page, rng)
    caches = []
    for _ in range(2):
        c = garbage_cache(n_pages, n_kv, d, page, fmt)
        g = torch.Generator().manual_seed(3)
        pre = torch.randn(2, 730, n_kv, d, generator=g).half().to(DEV)
        R.kv_append(c, pre[0], pre[1], R.kv_batch(start[:2], start[:2], rows[:2], DEV))
        caches.append(c)
    eager = R.kv_batch([1, 1, 1], [x + 1 for x in start], rows, DEV)
    batch = R.kv_batch([1, 1, 1], [x + 1 for x in start], rows, DEV)
    k, v = (torch.zeros(3, n_kv, d, dtype=torch.float16, device=DEV) for _ in range(2))
    q = torch.zeros(3, heads, d, dtype=torch.float16, device=DEV)
    y = torch.empty(3, heads, d, dtype=torch.float16, device=DEV)
    ws = R.kv_workspace(3, 3, 1, heads, n_kv, d, DEV)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # once before the capture, on a cache that is written again below
        R.kv_attend(caches[0], q, batch, y=y, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        R.kv_append(caches[0], k, v, batch)
        R.kv_attend(caches[0], q, batch, y=y, ws=ws)
    for step in range(20):
        nk, nv, nq = (torch.randn(3, h, d, device=DEV).half() for h in (n_kv, n_kv, heads))
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        graph.replay()
        R.kv_append(caches[1], nk, nv, eager)
        want = R.kv_attend(caches[1], nq, eager)
        torch.cuda.synchronize()
        assert torch.equal(y, want), step
        batch["ctx"] += 1
        eager["ctx"] += 1
    for m in ("k", "v"):
        assert torch.equal(caches[0][m + "_scale"].nan_to_num(-1), caches[1][m + "_scale"].nan_to_num(-1))


@pytest.mark.parametrize("n", [1, 20, 90])
def test_offsets_beyond_32_bits(n):
    """A pool of more than 2^32 bytes a matrix, the sequence's pages at its end."""
    n_kv, d, page = 8, 128, 64
    n_pages = (1 << 32) // (n_kv * d * page) + 40
    cache = R.kv_cache(n_pages, n_kv, d, page, "int8", DEV)
    ctx = [150]
    rows = [[n_pages - 1, n_pages - 33, n_pages - 7]]
    assert rows[0][1] * n_kv * d * page > 1 << 32
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(150, n_kv, d, generator=g).half().to(DEV) for _ in range(2))
    R.kv_append(cache, k, v, R.kv_batch([150], ctx, rows, DEV))
    q = queries(n, 16, d)
    y = R.kv_attend(cache, q, R.kv_batch([n], ctx, rows, DEV))
    gk, gv = R.kv_read(cache, R.kv_batch([150], ctx, rows, DEV))
    small = {m: (cache[m][[n_pages - 1, n_pages - 33, n_pages - 7]] if isinstance(cache[m], torch.Tensor) else cache[m]) for m in cache}
    torch.cuda.synchronize()
    del cache
    want = R.kv_attend(small, q, R.kv_batch([n], ctx, [[0, 1, 2]], DEV))
    wk, wv = R.kv_read(small, R.kv_batch([150], ctx, [[0, 1, 2]], DEV))
    assert torch.equal(y, want) and torch.equal(gk, wk) and torch.equal(gv, wv)
    assert float((gk.float() - k.float()).abs().max()) < 0.05


def test_many_sequences():
    """More sequences than lanes of a wave, some with nothing to do."""
    rng = np.random.default_rng(20)
    ctx = [int(c) for c in rng.integers(0, 60, 200)]
    new = [int(min(c, x)) if c else x % 2 for c, x in zip(ctx, rng.integers(0, 4, 200))]
    cache, rows = filled(ctx, 1, 64, 16, "int8", seed=21)
    rows = [r or [0] for r in rows]
    batch = R.kv_batch(new, ctx, rows, DEV)
    check_attend(cache, batch, queries(sum(new), 2, 64))
    k, v = R.kv_read(cache, batch)
    ok, ov = O.read(host(cache), host_batch(batch))
    assert np.array_equal(k.cpu().numpy(), ok.astype(np.float16)) and np.array_equal(v.cpu().numpy(), ov.astype(np.float16))


def test_broken_lengths_stay_inside():
    """Lengths and row ranges beyond the arrays are clamped: nothing outside the
    table, the pool or the outputs is touched, and sound sequences are not affected."""
    ctx = [40, 33]
    cache, rows = filled(ctx, 1, 64, 16, "int8", seed=22)
    good = R.kv_batch([1, 1], ctx, rows, DEV)
    q = queries(2, 2, 64)
    want = R.kv_attend(cache, q, good)
    bad = dict(good)
    bad["ctx"] = torch.tensor([2 ** 31 - 1, 33], dtype=torch.int32, device=DEV)
    y = R.kv_attend(cache, q, bad)
    assert torch.equal(y[1], want[1])
    bad["ctx"] = torch.tensor([-2 ** 31, 33], dtype=torch.int32, device=DEV)
    y = R.kv_attend(cache, q, bad)
    assert torch.equal(y[1], want[1]) and not torch.any(y[0])
    bad = dict(good)
    bad["q_start"] = torch.tensor([-7, 1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y = R.kv_attend(cache, q, bad)
    k, v = R.kv_read(cache, bad)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("n", [1, 20, 90])
def test_attend_widest_windows(n):
    """A window as wide as the type is no window, also for rows before position 0."""
    ctx = [n // 2 + 1, 200, 0]
    cache, rows = filled(ctx, 2, 64, 16, "int8")
    batch, q = R.kv_batch([n, 1, n], ctx, [r or [0] for r in rows], DEV), queries(2 * n + 1, 8, 64)
    y0 = check_attend(cache, batch, q)
    for window in (2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1, 201):
        assert torch.equal(check_attend(cache, batch, q, window=window), y0)
