"""What the cache and attention operators are measured on.

A case is one call as a serving program makes it: the new tokens' keys and
values written into the 8-bit paged cache and read back ("write"), the cached
tokens of some sequences read back ("read"), or attention of the call's query
tokens over the cache ("attend").  Both forms of `run` take the same state: the
cache in the byte order of include/pi.h, the sequences' lengths and page table
on the device, and fp16 inputs.

The cache: pages of `page` tokens, one fp32 scale per page and kv head for K
and one for V; a value is code * scale, with codes of int8 (byte = code + 128)
or fp8 e4m3.  Sequence s holds ctx[s] tokens, the last n_s of them being the
call's own.
"""

import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}


# ---------------------------------------------------------------- the cases

def _case(name, op, fmt, heads, kv, d, page, seqs, q, ctx, **more):
    """seqs sequences; the first seqs - decoding of them bring q tokens and the others one, and their
    contexts go up to ctx (all ctx where ragged is false).  idle: further sequences with one token and
    no context at all (an unused slot of a serving batch)."""
    c = {"name": name, "op": op, "fmt": fmt, "heads": heads, "kv": kv, "d": d, "page": page, "seqs": seqs, "q": q,
         "ctx": ctx, "ragged": False, "decoding": 0, "idle": 0, "window": 0, "mix": 1}
    c.update(more)
    return c


def listed():
    return [
        # the newest token of one sequence, 56 heads of 128 (the OPT-30B-shaped layer's d 7168): latency
        _case("write-1x1", "write", "int8", 56, 56, 128, 16, 1, 1, 1000),
        # a decode step of a serving batch, 8 kv heads of 128 (the LLaMA2-70B-shaped layer), ragged
        _case("write-64x1", "write", "fp8", 64, 8, 128, 64, 64, 1, 4096, ragged=True, mix=2),
        # prompts of a batch being admitted
        _case("write-8x2048", "write", "int8", 64, 8, 128, 16, 8, 2048, 2048),
        # one short conversation read back (moved to another place or another format)
        _case("read-1x777", "read", "fp8", 128, 8, 64, 16, 1, 777, 777),
        # a batch's whole caches read back
        _case("read-32x4096", "read", "int8", 64, 8, 128, 32, 32, 4096, 4096, ragged=True, mix=3),
        # one sequence's token shortly after a 128-token prompt: the smallest call, latency
        _case("attend-1x128", "attend", "int8", 56, 56, 128, 16, 1, 1, 128),
        # a decode step of 32 ragged sequences, 8 query heads a kv head (the LLaMA2-70B-shaped layer)
        _case("attend-32x4096", "attend", "int8", 64, 8, 128, 16, 32, 1, 4096, ragged=True, idle=1, mix=4),
        # one long document, 16 query heads of 64 a kv head (the Falcon-40B-shaped layer)
        _case("attend-1x131072", "attend", "fp8", 128, 8, 64, 64, 1, 1, 131072),
        # a decode step of 64 ragged sequences with a kv head per query head (the OPT-66B-shaped layer)
        _case("attend-64x2048", "attend", "int8", 72, 72, 128, 32, 64, 1, 2048, ragged=True, mix=5),
        # four proposed tokens a sequence checked at once, under a sliding window
        _case("attend-16x4of8192", "attend", "fp8", 64, 8, 128, 16, 16, 4, 8192, ragged=True, window=4097, mix=6),
        # a whole 2048-token prompt (the OPT-30B-shaped layer)
        _case("attend-prompt2048", "attend", "int8", 56, 56, 128, 16, 1, 2048, 2048),
        # a prompt's next 509 tokens beside seven sequences that decode
        _case("attend-mixed509", "attend", "int8", 64, 8, 128, 16, 8, 509, 4095, ragged=True, decoding=7, mix=7),
    ]


_HEADS = [(56, 56), (64, 8), (128, 8), (72, 72), (32, 32), (40, 8), (28, 4), (12, 12), (15, 5), (71, 1), (16, 2), (20, 20)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "attend"])
        heads, kv = rng.choice(_HEADS)
        c = _case("", op, rng.choice(["int8", "fp8"]), heads, kv, rng.choice([64, 64, 80, 96, 128, 128, 128, 256]),
                  rng.choice([16, 32, 64, 128]), 1, 1, 1, ragged=rng.random() < 0.7, mix=rng.randrange(1 << 20))
        c["seqs"] = _log(rng, 1, 64)
        c["ctx"] = _log(rng, 1, 131072)
        kind = rng.choice(["step", "step", "few", "prompt"])
        if op == "read":
            c["q"] = c["ctx"]
        elif kind == "few":
            c["q"] = min(c["ctx"], rng.randint(2, 9))
        elif kind == "prompt":
            c["q"] = _log(rng, 1, min(c["ctx"], 4096))
            c["decoding"] = rng.randrange(c["seqs"]) if rng.random() < 0.5 else 0
        if op == "attend" and rng.random() < 0.25:
            c["window"] = _log(rng, 1, c["ctx"])
        if op == "attend" and rng.random() < 0.2:
            c["idle"] = rng.randint(1, 3)
        w = work(c)
        n = c["seqs"] + c["idle"]
        pool = n * c["ctx"] * kv * c["d"] * 2
        scores = n * c["heads"] * c["q"] * c["ctx"] if op == "attend" else 0
        # no more than the largest listed cases: bytes and operations, the pool, and the padded plain form's scores
        sizes = list(c.values()) + [heads * c["d"], kv * c["d"]] + [x for of in _lens(c) for x in of]
        if w["bytes"] < 1.0e9 and w["flops"] < 6e10 and pool < 2.4e9 and scores < 5e8 and 3072 not in sizes:
            del c["name"]
            return c


def _lens(c):
    """[(new tokens, context)] of the sequences: the case's alone, not the seed's."""
    rng = random.Random(c["mix"])
    out = []
    for s in range(c["seqs"]):
        ctx = c["ctx"] if s == 0 or not c["ragged"] else max(1, int(c["ctx"] * rng.uniform(0.2, 1.0)))
        n = 1 if s >= c["seqs"] - c["decoding"] else min(c["q"], ctx)
        if c["op"] == "read":
            n = ctx
        out.append((n, ctx))
    return out + [(1, 0)] * c["idle"]


def _pages(ctx, page):
    return -(-ctx // page)


def _open(n, ctx, page):
    """First token of the block that the first of the n newest tokens falls into."""
    return (ctx - n) // page * page


def work(c):
    lens, h, kv, d, page = _lens(c), c["heads"], c["kv"], c["d"], c["page"]
    tok = sum(n for n, _ in lens)
    if c["op"] == "read":  # codes in, fp16 out, K and V
        return {"bytes": tok * kv * d * 2 * (1 + 2) + 8 * kv * sum(_pages(x, page) for _, x in lens), "flops": 2 * tok * kv * d}
    if c["op"] == "write":
        back = sum(x - _open(n, x, page) for n, x in lens)  # the open blocks are read back
        blocks = sum(_pages(x - _open(n, x, page), page) for n, x in lens)
        return {"bytes": 2 * kv * d * (3 * tok + 3 * back) + 16 * kv * blocks, "flops": 2 * kv * d * (3 * tok + back)}
    pairs, seen, scales = 0, 0, 0
    for n, x in lens:
        w = c["window"] or x + 1
        first = max(0, x - n - w + 1)  # first position any of the rows attends to
        if x:
            seen += x - first
            scales += _pages(x, page) - first // page
            under = max(0, min(n, w - (x - n)))  # rows that see less than a whole window, from x - n + 1 keys on
            pairs += under * (2 * (x - n) + under + 1) // 2 + (n - under) * w
    return {"bytes": 2 * kv * d * seen + 8 * kv * scales + 4 * tok * h * d, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------- inputs

def _to_cache_order(k, v):
    """Bytes of K and V, [pages, kv, page, d] each, in the cache's order."""
    p, h, n, d = k.shape
    k = k.view(p, h, n // 4, 4, d // 16, 16).permute(0, 1, 2, 4, 3, 5).reshape(p, h, n, d)
    v = v.view(p, h, n // 16, 16, d).permute(0, 1, 2, 4, 3).reshape(p, h, n, d)
    return k.contiguous(), v.contiguous()


def _from_cache_order(k, v):
    """The same bytes as [..., pages, kv, page, d] again, for any leading axes."""
    *a, h, n, d = k.shape
    k = k.reshape(*a, h, n // 4, d // 16, 4, 16).transpose(-3, -2).reshape(*a, h, n, d)
    v = v.reshape(*a, h, n // 16, d, 16).transpose(-2, -1).reshape(*a, h, n, d)
    return k, v


def _encode(x, fmt):
    """Rounded to the format's codes, as bytes; x is within +-QMAX."""
    if fmt == "int8":
        return (torch.round(x) + 128).to(torch.uint8)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(b, fmt):
    return b.float() - 128 if fmt == "int8" else b.view(torch.float8_e4m3fn).float()


def _normal(shape, g, dev):
    return torch.randn(shape, generator=g, device=dev)


def _keys(shape, g, dev, lead):
    """Keys with a few strong channels, as trained models have them; values are plain normal."""
    x = _normal(shape, g, dev)
    return x * (1.0 + 3.0 * (torch.rand(lead + (shape[-1],), generator=g, device=dev) < 0.04)).float()


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    lens, page, kv, d, fmt = _lens(c), c["page"], c["kv"], c["d"], c["fmt"]
    used = [_pages(x, page) for _, x in lens]
    n_pages = sum(used) + 3
    # every page quantised by its own largest value, as the cache holds it
    pools, scales = [], []
    for of in (_keys((n_pages, kv, page, d), g, dev, (1, kv, 1)), _normal((n_pages, kv, page, d), g, dev)):
        s = of.abs().amax(dim=(2, 3)) / QMAX[fmt]
        pools.append(_encode((of / s[:, :, None, None]).clamp(-QMAX[fmt], QMAX[fmt]), fmt))
        scales.append(s)
        del of
    k, v = _to_cache_order(*pools)
    # the pages in no order; entries past a sequence's last page hold nothing
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    width, rows = max(1, max(used)), []
    for n in used:
        rows.append(order[:n] + [-1] * (width - n))
        order = order[n:]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def batch(counts):
        at = [0]
        for n in counts:
            at.append(at[-1] + n)
        return {"q_start": ints(at), "ctx": ints([x for _, x in lens]), "table": ints(rows), "n_tok": at[-1], "max_q": max(counts)}

    st = {"op": c["op"], "window": c["window"], "cache": {"k": k, "v": v, "k_scale": scales[0], "v_scale": scales[1], "fmt": fmt},
          "batch": batch([n for n, _ in lens])}
    tok = st["batch"]["n_tok"]
    if c["op"] == "attend":
        st["q"] = _normal((tok, c["heads"], d), g, dev).half()
    elif c["op"] == "write":
        st["k_new"] = _keys((tok, kv, d), g, dev, (kv,)).half()
        st["v_new"] = _normal((tok, kv, d), g, dev).half()
        st["back"] = batch([x - _open(n, x, page) for n, x in lens])
    return st


# ---------------------------------------------------------------- the plain forms

def _rows(batch):
    """Per token of the call: its sequence and its position."""
    start = batch["q_start"].long()
    t = torch.arange(batch["n_tok"], device=start.device)
    s = (t[:, None] >= start[None, 1:]).sum(1)
    return s, batch["ctx"].long()[s] - start[s + 1] + t


def _read(cache, batch):
    s, pos = _rows(batch)
    page = cache["k"].shape[2]
    at = pos.clamp(min=0)
    ids = batch["table"].long()[s, at // page].clamp(min=0)
    k, v = _from_cache_order(cache["k"], cache["v"])
    gone = (pos < 0)[:, None, None]
    out = []
    for codes, scale in ((k, cache["k_scale"]), (v, cache["v_scale"])):
        x = _decode(codes[ids, :, at % page], cache["fmt"]) * scale[ids][:, :, None]
        out.append(x.masked_fill(gone, 0.0).half())
    return {"k": out[0], "v": out[1]}


def _write(cache, batch, k_new, v_new):
    fmt, page, kv, d = cache["fmt"], cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    start, ctx, dev = batch["q_start"].long(), batch["ctx"].long(), k_new.device
    n = start[1:] - start[:-1]
    # the blocks that get new tokens: [sequences, blocks], and their slots' tokens: [blocks, page]
    first = (ctx - n) // page
    blocks = first[:, None] + torch.arange((batch["max_q"] + page - 2) // page + 1, device=dev)
    live = (blocks * page < ctx[:, None]) & (n > 0)[:, None]
    seq = torch.arange(len(ctx), device=dev)[:, None].expand_as(blocks)[live]
    blocks = blocks[live]
    ids = batch["table"].long()[seq, blocks]
    slot = blocks[:, None] * page + torch.arange(page, device=dev)
    new = (slot >= (ctx - n)[seq][:, None]) & (slot < ctx[seq][:, None])
    old = slot < (ctx - n)[seq][:, None]
    token = (start[seq + 1] - ctx[seq])[:, None] + slot
    k, v = _from_cache_order(cache["k"][ids], cache["v"][ids])
    done = []
    for codes, scale, x in ((k, cache["k_scale"], k_new), (v, cache["v_scale"], v_new)):
        x = x[token.clamp(0, batch["n_tok"] - 1)].permute(0, 2, 1, 3).float()  # [blocks, kv, page, d]
        here, there = new[:, None, :, None], old[:, None, :, None]
        s0 = torch.where(old.any(1)[:, None], scale[ids], 0.0)
        s = torch.maximum(s0, x.abs().masked_fill(~here, 0.0).amax(dim=(2, 3)) / QMAX[fmt])
        by = s[:, :, None, None]
        fresh = torch.where(by > 0, x / by, 0.0).clamp(-QMAX[fmt], QMAX[fmt])
        kept = _decode(codes, fmt) * torch.where(s > 0, s0 / s, 1.0)[:, :, None, None]
        codes = torch.where(here, _encode(fresh, fmt), torch.where(there & (s > s0)[:, :, None, None], _encode(kept, fmt), codes))
        scale[ids] = s
        done.append(codes)
    cache["k"][ids], cache["v"][ids] = _to_cache_order(*done)


def _attend(cache, batch, q, window):
    fmt, page, kv, d = cache["fmt"], cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    heads, most = q.shape[1], batch["max_q"]
    start, ctx, dev = batch["q_start"].long(), batch["ctx"].long(), q.device
    n = start[1:] - start[:-1]
    ids = batch["table"].long().clamp(min=0)  # [sequences, pages]
    k, v = _from_cache_order(cache["k"][ids], cache["v"][ids])

    def values(codes, scale):  # [sequences, kv, tokens, d]
        x = _decode(codes, fmt) * scale[ids][..., None, None]
        return x.transpose(1, 2).reshape(len(ctx), kv, -1, d)

    # the queries as [sequences, kv, tokens * heads of a kv head, d], padded to the longest
    i = torch.arange(most, device=dev)
    at = (start[:-1, None] + i).clamp(max=batch["n_tok"] - 1)
    rows = q[at].float().view(len(ctx), most, kv, heads // kv, d).transpose(1, 2).reshape(len(ctx), kv, -1, d)
    x = torch.matmul(rows, values(k, cache["k_scale"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    pos = ((ctx - n)[:, None] + i)[:, :, None]
    key = torch.arange(x.shape[-1], device=dev)
    seen = (key <= pos) & (key > pos - window if window else key >= 0)
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, heads // kv, -1).reshape(len(ctx), 1, -1, x.shape[-1])
    x = x.masked_fill(~seen, float("-inf"))
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    total = e.sum(-1, keepdim=True)
    y = torch.matmul(e, values(v, cache["v_scale"])) / torch.where(total > 0, total, 1.0)
    y = y.view(len(ctx), kv, most, heads // kv, d).transpose(1, 2).reshape(len(ctx), most, heads, d)
    s, p = _rows(batch)
    return y[s, p - (ctx - n)[s]].half()


def run(state):
    op, cache, batch = state["op"], state["cache"], state["batch"]
    if own:
        from activation_sparse_predictor_amd import runtime as R

        if op == "attend":
            return R.kv_attend(cache, state["q"], batch, window=state["window"])
        if op == "write":
            R.kv_append(cache, state["k_new"], state["v_new"], batch)
            batch = state["back"]
        k, v = R.kv_read(cache, batch)
        return {"k": k, "v": v}
    if op == "attend":
        return _attend(cache, batch, state["q"], state["window"])
    if op == "write":
        _write(cache, batch, state["k_new"], state["v_new"])
        batch = state["back"]
    return _read(cache, batch)


# ---------------------------------------------------------------- 64 bits

_E4M3 = [(-1.0 if b & 128 else 1.0) * ((b & 7) / 8.0 * 2.0 ** -6 if not b & 120 else (1 + (b & 7) / 8.0) * 2.0 ** ((b >> 3 & 15) - 7)) for b in range(256)]


def _exact_codes(b, fmt):
    """Bytes to code values in 64 bits, by the formats' definitions."""
    if fmt == "int8":
        return b.double() - 128.0
    return torch.tensor(_E4M3, dtype=torch.float64, device=b.device)[b.long()]


def _exact_round(x, fmt):
    """To the nearest code, ties to even."""
    if fmt == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_sequence(st, s, k_scale, v_scale):
    """K and V codes and scales of sequence s's tokens: [tokens, kv, d] and [tokens, kv]."""
    cache, page = st["cache"], st["cache"]["k"].shape[2]
    x = int(st["batch"]["ctx"][s])
    ids = st["batch"]["table"][s, : _pages(x, page)].long()
    t = torch.arange(x, device=ids.device)
    kv, d = cache["k"].shape[1], cache["k"].shape[3]
    j = torch.arange(d, device=ids.device)
    tk, out = t % page, []
    where = ((tk // 4 * 4 * d + tk % 4 * 16)[:, None] + j // 16 * 64 + j % 16, (tk // 16 * 16 * d + tk % 16)[:, None] + j * 16)
    for name, place, scale in (("k", where[0], k_scale), ("v", where[1], v_scale)):
        flat = cache[name].view(-1, kv, page * d)[ids[t // page]]  # [tokens, kv, page * d] would be large: gathered head by head below
        out += [torch.stack([flat[:, h].gather(1, place) for h in range(kv)], 1), scale[ids[t // page]]]
        del flat
    return out


def exact(case, seed):
    c, fmt, page = case, case["fmt"], case["page"]
    kv, d, lens = c["kv"], c["d"], _lens(c)
    st = prepare(case, seed)
    k_scale, v_scale = (st["cache"][n].double() for n in ("k_scale", "v_scale"))
    out, at = [], 0
    for s, (n, x) in enumerate(lens):
        if c["op"] == "attend" and x == 0:
            out.append(torch.zeros(n, c["heads"], d, dtype=torch.float64, device="cuda"))
            at += n
            continue
        seq = []
        # pieces of whole pages, so that a page's bytes are not gathered for all tokens at once
        part = max(page, (1 << 28) // (kv * page * d) // page * page)
        full = {"ctx": st["batch"]["ctx"], "table": st["batch"]["table"]}
        for lo in range(0, x, part):
            piece = {"cache": st["cache"], "batch": {"ctx": torch.clamp(full["ctx"] - lo, max=part), "table": full["table"][:, lo // page:]}}
            seq.append(_exact_sequence(piece, s, k_scale, v_scale))
        kc, ks, vc, vs = (torch.cat([p[i] for p in seq]) for i in range(4))
        kc, vc = _exact_codes(kc, fmt), _exact_codes(vc, fmt)
        if c["op"] == "attend":
            kx, vx = (kc * ks[:, :, None]).permute(1, 2, 0), (vc * vs[:, :, None]).transpose(0, 1)  # [kv, d, x], [kv, x, d]
            q = st["q"][at : at + n].double().view(n, kv, -1, d).transpose(0, 1)  # [kv, n, group, d]
            pos = x - n + torch.arange(n, device=q.device)
            key = torch.arange(x, device=q.device)
            far = (key[None] > pos[:, None]) | ((key[None] <= pos[:, None] - c["window"]) if c["window"] else False)
            ys = []
            for h in range(kv):
                z = (q[h].reshape(-1, d) @ kx[h]).view(n, -1, x) / math.sqrt(d)
                p = torch.softmax(z.masked_fill(far[:, None], -math.inf), -1)
                ys.append((p.view(-1, x) @ vx[h]).view(n, -1, d))
            out.append(torch.stack(ys, 1).reshape(n, c["heads"], d))
        elif c["op"] == "read":
            out.append((kc * ks[:, :, None], vc * vs[:, :, None]))
        else:
            back = []
            for codes, scale, new in ((kc, ks, st["k_new"]), (vc, vs, st["v_new"])):
                new = new[at : at + n].double()
                for b in range(_open(n, x, page), x, page):  # block by block, as the definition says it
                    a = max(b, x - n)
                    fresh = new[a - (x - n) : b + page - (x - n)]
                    s0 = scale[b] if a > b else torch.zeros(kv, dtype=torch.float64, device=scale.device)
                    s1 = torch.maximum(s0, fresh.abs().amax((0, 2)) / QMAX[fmt])
                    safe = torch.where(s1 > 0, s1, 1.0)
                    older = codes[b:a]
                    older = torch.where((s1 > s0)[None, :, None], _exact_round(older * (s0 / safe)[None, :, None], fmt), older)
                    fresh = _exact_round(fresh / safe[None, :, None], fmt)
                    back.append(torch.cat([older, fresh]) * s1[None, :, None])
            half = len(back) // 2
            out.append((torch.cat(back[:half]), torch.cat(back[half:])))
        at += n
    if c["op"] == "attend":
        return torch.cat(out)
    return {"k": torch.cat([o[0] for o in out]), "v": torch.cat([o[1] for o in out])}
