"""What the operators of a speculative decoding step are measured on.

A case is one call as a serving program makes it: heads turned by rotary
positions ("rotate"), new keys and values written into the 8-bit paged cache
with the rotation on the way ("append"; the written blocks are read back),
attention of a tree of drafted tokens over the cache ("tree"), or the decision
which drafted tokens stay ("verify").  Both forms of `run` take the same state:
the cache in the byte order of include/pi.h, lengths, page table, masks and
parents on the device, fp16 rows, fp32 probabilities.

A rotary plan is a layout ("half": dimensions i and i + rot / 2 form a pair,
"pairs": 2 i and 2 i + 1), the number of dimensions it turns, a gain, and for
each pair the angle's advance per position: in 64 bits for the plain form, and
in units of 2^-64 turns as the library takes it.
"""

import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}


# ---------------------------------------------------------------- the cases

def _rotate(name, heads, d, rot, tokens, far, layout="half", scaling="none", factor=1.0):
    return {"name": name, "op": "rotate", "heads": heads, "d": d, "rot": rot, "tokens": tokens, "far": far, "layout": layout,
            "scaling": scaling, "factor": factor}


def _append(name, fmt, heads, kv, d, page, seqs, q, ctx, rot, layout="half", scaling="none", factor=1.0, ragged=False, nodes=0,
            mix=1):
    """seqs sequences of up to ctx tokens, the last up to q of them new.  nodes: the new tokens are accepted ones among that many
    drafted rows a sequence, already turned, and are named by a list of rows; no queries then."""
    return {"name": name, "op": "append", "fmt": fmt, "heads": heads, "kv": kv, "d": d, "page": page, "seqs": seqs, "q": q,
            "ctx": ctx, "rot": rot, "layout": layout, "scaling": scaling, "factor": factor, "ragged": ragged, "nodes": nodes,
            "mix": mix}


def _tree(name, fmt, heads, kv, d, page, seqs, nodes, ctx, ragged=False, window=0, mix=1):
    return {"name": name, "op": "tree", "fmt": fmt, "heads": heads, "kv": kv, "d": d, "page": page, "seqs": seqs, "nodes": nodes,
            "ctx": ctx, "ragged": ragged, "window": window, "mix": mix}


def _verify(name, seqs, nodes, vocab, drafts, chain=False, ragged=False, mix=1):
    """nodes rows a sequence, the first of them the newest known token.  drafts: "drawn" from the draft's probabilities, or
    "fixed" (a table's or a search's proposals, which have none)."""
    return {"name": name, "op": "verify", "seqs": seqs, "nodes": nodes, "vocab": vocab, "drafts": drafts, "chain": chain,
            "ragged": ragged, "mix": mix}


def listed():
    return [
        # the query heads of one token, 56 heads of 128 (the OPT-30B-shaped layer's d 7168): latency
        _rotate("rotate-1x56", 56, 128, 128, 1, 4000),
        # queries and keys of a 2048-token prompt in one call (the LLaMA2-70B-shaped layer: 64 + 8 heads), a context stretched by 8
        _rotate("rotate-2048x72", 72, 128, 128, 2048, 262144, scaling="yarn", factor=8.0),
        # a decode step's one token of one sequence (the OPT-30B-shaped layer): latency
        _append("append-1x1", "int8", 56, 56, 128, 16, 1, 1, 1000, 128),
        # a decode step of a serving batch, 8 kv heads (the LLaMA2-70B-shaped layer), ragged
        _append("append-64x1", "fp8", 64, 8, 128, 64, 64, 1, 4096, 128, scaling="linear", factor=4.0, ragged=True, mix=2),
        # prompts of a batch being admitted
        _append("append-4x2048", "int8", 64, 8, 128, 16, 4, 2048, 2048, 128),
        # the accepted ones of 16 drafted tokens of 48 sequences
        _append("append-accepted48", "int8", 64, 8, 128, 16, 48, 6, 3000, 128, ragged=True, nodes=16, mix=3),
        # a small tree shortly after a short prompt, one sequence (the OPT-30B-shaped layer): latency
        _tree("tree-1x8of128", "int8", 56, 56, 128, 16, 1, 8, 128),
        # 16 ragged sequences of 16 drafted tokens (the LLaMA2-70B-shaped layer: 128 rows a kv head)
        _tree("tree-16x16of8192", "fp8", 64, 8, 128, 16, 16, 16, 8192, ragged=True, mix=4),
        # a wide tree over long ragged contexts under a sliding window, 16 query heads of 64 a kv head (the Falcon-40B-shaped layer)
        _tree("tree-6x63of6000", "int8", 128, 8, 64, 32, 6, 63, 6000, ragged=True, window=4097, mix=5),
        # one sequence's chain of four proposals: latency
        _verify("verify-1x5", 1, 5, 32000, "drawn", chain=True),
        # trees of 16 of 48 sequences, siblings drawn from one distribution
        _verify("verify-48x16", 48, 16, 50257, "drawn", ragged=True, mix=6),
        # a table's proposals, which have no probabilities, over a large vocabulary
        _verify("verify-16x32", 16, 32, 128000, "fixed", ragged=True, mix=7),
    ]


_HEADS = [(56, 56), (64, 8), (128, 8), (72, 72), (32, 32), (40, 8), (28, 4), (12, 12), (15, 5), (71, 1), (16, 2), (20, 20)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_rope(rng, d):
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    rot = d if rng.random() < 0.6 else 2 * rng.randint(2, d // 2)
    return {"rot": rot, "layout": rng.choice(["half", "half", "pairs"]), "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])}


def draw(rng):
    while True:
        op = rng.choice(["rotate", "append", "append", "tree", "tree", "tree", "verify", "verify"])
        heads, kv = rng.choice(_HEADS)
        d = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
        ctx, page, seqs = _log(rng, 1, 32768), rng.choice([16, 32, 64, 128]), _log(rng, 1, 64)
        ragged, mix = rng.random() < 0.7, rng.randrange(1 << 20)
        if op == "rotate":
            c = _rotate("", heads + kv, d, d, _log(rng, 1, 8192), _log(rng, 16, 1 << 20))
            c.update(_draw_rope(rng, d))
            scores = 0
        elif op == "append":
            nodes = rng.choice([0, 0, 8, 16, 33])
            new = min(ctx, rng.choice([1, rng.randint(2, 9), _log(rng, 1, 4096)]) if not nodes else rng.randint(1, 7))
            c = _append("", rng.choice(["int8", "fp8"]), heads, kv, d, page, seqs, new, ctx, d, ragged=ragged, nodes=nodes, mix=mix)
            c.update(_draw_rope(rng, d))
            scores = 0
        elif op == "tree":
            c = _tree("", rng.choice(["int8", "fp8"]), heads, kv, d, page, seqs, _log(rng, 1, 200), ctx, ragged=ragged, mix=mix)
            if rng.random() < 0.25:
                c["window"] = _log(rng, 1, ctx)
            scores = seqs * heads * c["nodes"] * (ctx + c["nodes"])
        else:
            c = _verify("", seqs, _log(rng, 1, 48), _log(rng, 100, 131072), rng.choice(["drawn", "fixed"]),
                        chain=rng.random() < 0.4, ragged=ragged, mix=mix)
            scores = seqs * c["nodes"] * c["vocab"] * 8
        w = work(c)
        pool = seqs * ctx * kv * d * 2 if op in ("append", "tree") else 0
        # no more than the largest listed cases, and what the plain form and the inputs take
        if w["bytes"] < 2.0e8 and w["flops"] < 3e10 and pool < 1.2e9 and scores < 4e8:
            del c["name"]
            return c


def _pages(ctx, page):
    return -(-ctx // page)


def _open(n, ctx, page):
    """First token of the block that the first of the n newest tokens falls into."""
    return (ctx - n) // page * page


def _lens(c):
    """[(rows of the call, context)] of the sequences: the case's alone, not the seed's."""
    rng = random.Random(c["mix"])
    out = []
    for s in range(c["seqs"]):
        whole = s == 0 or not c["ragged"]
        if c["op"] == "verify":
            out.append((c["nodes"] if whole else rng.randint(1, c["nodes"]), 100 + 7 * s))
            continue
        ctx = c["ctx"] if whole else max(1, int(c["ctx"] * rng.uniform(0.2, 1.0)))
        if c["op"] == "tree":
            out.append((c["nodes"] if whole else max(1, int(c["nodes"] * rng.uniform(0.4, 1.0))), ctx))
        else:
            n = min(c["q"], ctx)
            out.append((rng.randint(1, n) if c["nodes"] else n, ctx))
    return out


def _parents(c):
    """Per sequence, each row's parent (-1: none): row 0 is the known token, the others hang below an earlier one."""
    rng = random.Random(c["mix"] + 1)
    out = []
    for n, _ in _lens(c):
        chain = c.get("chain", False)
        out.append([-1] + [j - 1 if chain else max(0, j - 1 - int(rng.expovariate(0.4))) for j in range(1, n)])
    return out


def work(c):
    if c["op"] == "rotate":
        n = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 4 * n + 4 * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    lens = _lens(c)
    if c["op"] == "verify":
        # of a sequence: the last accepted row's probabilities, and an element or two a drafted token
        rows = 2 if c["drafts"] == "drawn" else 1
        tok = sum(n for n, _ in lens)
        return {"bytes": 4 * rows * c["vocab"] * len(lens) + (20 + 4 * rows) * tok, "flops": 3 * c["vocab"] * len(lens)}
    h, kv, d, page = c["heads"], c["kv"], c["d"], c["page"]
    tok = sum(n for n, _ in lens)
    if c["op"] == "append":
        back = sum(x - _open(n, x, page) for n, x in lens)  # the open blocks are read back
        blocks = sum(_pages(x - _open(n, x, page), page) for n, x in lens)
        turned = 0 if c["nodes"] else 4 * tok * h * d
        return {"bytes": 2 * kv * d * (3 * tok + 3 * back) + 16 * kv * blocks + turned,
                "flops": 2 * kv * d * (3 * tok + back) + (0 if c["nodes"] else 3 * tok * (h + kv) * c["rot"])}
    pairs, seen, scales = 0, 0, 0
    depths, masks = _ancestors(c)
    for (n, x), dep, mask in zip(lens, depths, masks):
        w = c["window"] or x + n + 1
        first = max(0, x + min(dep) - w + 1)
        seen += x - first if first < x else 0
        scales += _pages(x, page) - first // page if first < x else 0
        pairs += sum(max(0, x - max(0, x + t - w + 1)) + bin(m).count("1") for t, m in zip(dep, mask))
    return {"bytes": 2 * kv * d * seen + 8 * kv * scales + 4 * tok * h * d + 4 * tok * kv * d + 8 * tok, "flops": 4 * d * h * pairs}


def _ancestors(c):
    """Per sequence and row: its depth, and the rows it attends to (itself and those above it) as bits."""
    depths, masks = [], []
    for parent in _parents(c):
        dep, mask = [], []
        for j, p in enumerate(parent):
            dep.append(0 if p < 0 else dep[p] + 1)
            mask.append((0 if p < 0 else mask[p]) | 1 << j)
        depths.append(dep)
        masks.append(mask)
    return depths, masks


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


def _frequencies(c):
    """Radians a position advances each pair by, and the gain, in 64 bits."""
    half, base, f = c["rot"] // 2, 10000.0, c["factor"]
    if c["scaling"] == "ntk" and c["rot"] > 2:
        base *= f ** (c["rot"] / (c["rot"] - 2.0))
    out = [base ** (-2.0 * i / c["rot"]) for i in range(half)]
    gain = 1.0
    if c["scaling"] == "linear":
        out = [x / f for x in out]
    if c["scaling"] == "yarn":
        gain = 0.1 * math.log(f) + 1.0
        blend = []
        for x in out:  # a pair that turns often over the trained length keeps its frequency, one that hardly turns is stretched
            keep = min(1.0, max(0.0, (4096 * x / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
            blend.append((1.0 - keep) * x / f + keep * x)
        out = blend
    return out, gain


def _rope(c, dev):
    freqs, gain = _frequencies(c)
    turns = []
    for x in freqs:
        t = int(x / (2 * math.pi) % 1.0 * 2 ** 64)
        turns.append(t - (1 << 64) if t >> 63 else t)
    return ({"layout": c["layout"], "rot": c["rot"], "gain": gain, "turns": torch.tensor(turns, dtype=torch.int64, device=dev)},
            torch.tensor(freqs, dtype=torch.float64, device=dev))


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    st = {"op": c["op"]}
    if c["op"] in ("rotate", "append"):
        st["rope"], st["freqs"] = _rope(c, dev)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if c["op"] == "rotate":
        n = c["tokens"]
        # a batch's tokens: runs of neighbouring positions
        start = torch.randint(0, c["far"], (n // 64 + 1,), generator=g, device=dev)
        st["pos"] = (start[:, None] + torch.arange(64, device=dev)).flatten()[:n].to(torch.int32).contiguous()
        st["x"] = _normal((n, c["heads"], c["d"]), g, dev).half()
        return st
    lens = _lens(c)

    def batch(counts):
        at = [0]
        for n in counts:
            at.append(at[-1] + n)
        return {"q_start": ints(at), "ctx": ints([x for _, x in lens]), "n_tok": at[-1], "max_q": max(counts)}

    if c["op"] == "verify":
        st["batch"] = batch([n for n, _ in lens])
        tok, vocab = st["batch"]["n_tok"], c["vocab"]
        parents = _parents(c)
        st["parent"] = ints([p for seq in parents for p in seq])
        # the target's next-token distributions, and a draft model's that is nearly as sure of the same tokens
        z = _normal((tok, vocab), g, dev) * 2.5
        st["p"] = torch.softmax(z, 1)
        st["q"] = torch.softmax(z * 0.8 + _normal((tok, vocab), g, dev), 1) if c["drafts"] == "drawn" else None
        first, above = 0, []
        for seq in parents:
            above += [first + max(p, 0) for p in seq]
            first += len(seq)
        above = torch.tensor(above, device=dev)
        if c["drafts"] == "drawn":  # each drawn from the draft's distribution at its parent
            cum = torch.cumsum(st["q"].double(), 1)
            at = torch.rand((tok, 1), generator=g, device=dev, dtype=torch.float64) * cum[above, -1:]
            st["tokens"] = (cum[above] <= at).sum(1).clamp(max=vocab - 1).to(torch.int32)
        else:  # siblings are the target's likeliest tokens in another order
            order = torch.topk(z, min(vocab, 8), 1).indices
            pick = torch.randint(0, order.shape[1], (tok,), generator=g, device=dev)
            st["tokens"] = order[above, pick].to(torch.int32)
        st["u"] = torch.rand((tok,), generator=g, device=dev)
        st["u_next"] = torch.rand((len(lens),), generator=g, device=dev)
        return st

    page, kv, d, fmt = c["page"], c["kv"], c["d"], c["fmt"]
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
    st["cache"] = {"k": k, "v": v, "k_scale": scales[0], "v_scale": scales[1], "fmt": fmt}
    # the pages in no order; entries past a sequence's last page hold nothing
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    width, rows = max(1, max(used)), []
    for n in used:
        rows.append(order[:n] + [-1] * (width - n))
        order = order[n:]
    table = ints(rows)
    st["batch"] = {**batch([n for n, _ in lens]), "table": table}
    tok = st["batch"]["n_tok"]
    if c["op"] == "append":
        src = c["nodes"] * c["seqs"] if c["nodes"] else tok
        if c["nodes"]:  # ascending rows of each sequence's drafted ones, the first always
            rng, taken = random.Random(int(seed) * 31 + c["mix"]), []
            for s, (n, _) in enumerate(lens):
                taken += [s * c["nodes"]] + [s * c["nodes"] + r for r in sorted(rng.sample(range(1, c["nodes"]), n - 1))]
            st["rows"] = ints(taken)
        else:
            st["query"] = _normal((tok, c["heads"], d), g, dev).half()
        st["k_new"] = _keys((src, kv, d), g, dev, (kv,)).half()
        st["v_new"] = _normal((src, kv, d), g, dev).half()
        st["back"] = {**batch([x - _open(n, x, page) for n, x in lens]), "table": table}
        return st
    depths, masks = _ancestors(c)
    st["window"] = c["window"]
    words = (c["nodes"] + 63) // 64
    bits = [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for seq in masks for m in seq]
    st["mask"] = torch.tensor([[b - (1 << 64) if b >> 63 else b for b in row] for row in bits], dtype=torch.int64, device=dev)
    st["pos"] = ints([x + t for (_, x), dep in zip(lens, depths) for t in dep])
    st["query"] = _normal((tok, c["heads"], d), g, dev).half()
    st["k_new"] = _keys((tok, kv, d), g, dev, (kv,)).half()
    st["v_new"] = _normal((tok, kv, d), g, dev).half()
    return st


# ---------------------------------------------------------------- the plain forms

def _turn(x, pos, rope, freqs):
    """Rows x [tokens, heads, d] turned by their positions, in fp32; the angles in 64 bits."""
    rot = rope["rot"]
    a = pos.double()[:, None, None] * freqs
    cos, sin = (torch.cos(a) * rope["gain"]).float(), (torch.sin(a) * rope["gain"]).float()
    x = x.float()
    t = x[..., :rot]
    if rope["layout"] == "half":
        one, two = t[..., : rot // 2], t[..., rot // 2 :]
        t = torch.cat([one * cos - two * sin, two * cos + one * sin], -1)
    else:
        one, two = t[..., ::2], t[..., 1::2]
        t = torch.stack([one * cos - two * sin, two * cos + one * sin], -1).flatten(-2)
    return torch.cat([t, x[..., rot:]], -1)


def _rows(batch):
    """Per token of the call: its sequence and its position."""
    start = batch["q_start"].long()
    t = torch.arange(batch["n_tok"], device=start.device)
    s = (t[:, None] >= start[None, 1:]).sum(1)
    return s, batch["ctx"].long()[s] - start[s + 1] + t


def _read(cache, batch):
    s, pos = _rows(batch)
    page = cache["k"].shape[2]
    ids = batch["table"].long()[s, pos // page]
    k, v = _from_cache_order(cache["k"], cache["v"])
    out = []
    for codes, scale in ((k, cache["k_scale"]), (v, cache["v_scale"])):
        out.append((_decode(codes[ids, :, pos % page], cache["fmt"]) * scale[ids][:, :, None]).half())
    return {"k": out[0], "v": out[1]}


def _write(cache, batch, k_new, v_new):
    """k_new and v_new: the batch's tokens in fp32."""
    fmt, page = cache["fmt"], cache["k"].shape[2]
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
        x = x[token.clamp(0, batch["n_tok"] - 1)].permute(0, 2, 1, 3)  # [blocks, kv, page, d]
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


def _attend_tree(st):
    cache, batch, q = st["cache"], st["batch"], st["query"]
    fmt, kv, d = cache["fmt"], cache["k"].shape[1], cache["k"].shape[3]
    heads, most = q.shape[1], batch["max_q"]
    start, ctx, dev = batch["q_start"].long(), batch["ctx"].long(), q.device
    n, seqs = start[1:] - start[:-1], batch["ctx"].shape[0]
    ids = batch["table"].long().clamp(min=0)  # [sequences, pages]
    k, v = _from_cache_order(cache["k"][ids], cache["v"][ids])
    i = torch.arange(most, device=dev)
    at = (start[:-1, None] + i).clamp(max=batch["n_tok"] - 1)  # the padded rows of the sequences

    def values(codes, scale, new):  # [sequences, kv, cached and drafted tokens, d]
        x = _decode(codes, fmt) * scale[ids][..., None, None]
        return torch.cat([x.transpose(1, 2).reshape(seqs, kv, -1, d), new[at].float().transpose(1, 2)], 2)

    rows = q[at].float().view(seqs, most, kv, heads // kv, d).transpose(1, 2).reshape(seqs, kv, -1, d)
    ks = values(k, cache["k_scale"], st["k_new"]).transpose(-1, -2).contiguous()
    x = torch.matmul(rows, ks) * (1.0 / math.sqrt(d))
    del ks, k
    cached = torch.arange(x.shape[-1] - most, device=dev)
    seen = (cached < ctx[:, None, None]).expand(-1, most, -1)
    if st["window"]:
        seen = seen & (cached > (st["pos"].long()[at] - st["window"])[:, :, None])
    bits = st["mask"][at][:, :, i // 64] >> (i % 64) & 1  # [sequences, rows, drafted]
    seen = torch.cat([seen, (bits > 0) & (i < n[:, None, None])], 2)
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, heads // kv, -1).reshape(seqs, 1, -1, x.shape[-1])
    x = x.masked_fill_(~seen, float("-inf"))
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    del x
    total = e.sum(-1, keepdim=True)
    y = torch.matmul(e, values(v, cache["v_scale"], st["v_new"])) / torch.where(total > 0, total, 1.0)
    y = y.view(seqs, kv, most, heads // kv, d).transpose(1, 2).reshape(seqs, most, heads, d)
    s = (torch.arange(batch["n_tok"], device=dev)[:, None] >= start[None, 1:]).sum(1)
    return y[s, torch.arange(batch["n_tok"], device=dev) - start[s]].half()


def _decide(st):
    """The walk from each sequence's first row down to where no child is accepted, all sequences abreast and row by row: a child
    lies behind its parent.  In 64 bits: what is left of a distribution decides between neighbouring tokens."""
    batch, p, q = st["batch"], st["p"], st["q"]
    start, ctx, dev = batch["q_start"].long(), batch["ctx"].long(), p.device
    n, seqs, vocab = start[1:] - start[:-1], batch["ctx"].shape[0], p.shape[1]
    cur = start[:-1].clone()
    left = p[cur].double()          # what the children rejected so far leave of the row's distribution
    draft = q[cur].double() if q is not None else None
    mass = torch.ones(seqs, dtype=torch.float64, device=dev)
    taken = torch.zeros(batch["n_tok"], dtype=torch.bool, device=dev)
    taken[cur] = True
    for j in range(1, batch["max_q"]):
        row = (start[:-1] + j).clamp(max=batch["n_tok"] - 1)
        child = (j < n) & (st["parent"].long()[row] + start[:-1] == cur)
        token = st["tokens"].long()[row][:, None]
        of = left.gather(1, token)[:, 0]
        by = draft.gather(1, token)[:, 0] if q is not None else 1.0
        good = child & (st["u"][row].double() * by * mass < of)
        bad = child & ~good
        if q is not None:
            rest = (left - mass[:, None] * draft).clamp(min=0)
        else:
            rest = left.scatter(1, token, 0.0)
        here = p[row].double()
        left = torch.where(good[:, None], here, torch.where(bad[:, None], rest, left))
        mass = torch.where(good, 1.0, torch.where(bad, rest.sum(1) if q is not None else mass - of, mass))
        if q is not None:
            draft = torch.where(good[:, None], q[row].double(), draft)
        cur = torch.where(good, row, cur)
        taken[row[good]] = True
    left = torch.where(left.sum(1, keepdim=True) > 0, left, p[cur].double())
    cum = torch.cumsum(left, 1)
    token = (cum <= st["u_next"].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=vocab - 1)
    seq = (torch.arange(batch["n_tok"], device=dev)[:, None] >= start[None, 1:]).sum(1)
    count = torch.zeros(seqs, dtype=torch.int64, device=dev).index_add_(0, seq, taken.long())
    rows = torch.full((batch["n_tok"],), -1, dtype=torch.int32, device=dev)
    found = torch.nonzero(taken)[:, 0]
    rows[: found.shape[0]] = found.to(torch.int32)
    at = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    return {"rows": rows, "q_start": at.to(torch.int32), "ctx": (ctx + count).to(torch.int32), "next": token.to(torch.int32)}


def run(state):
    st, op = state, state["op"]
    if own:
        from activation_sparse_predictor_amd import runtime as R

        if op == "rotate":
            return R.rotate(st["x"], st["pos"], st["rope"])
        if op == "append":
            rows = st.get("rows")
            if rows is None:
                query = R.kv_append_rope(st["cache"], st["k_new"], st["v_new"], st["batch"], st["rope"], q=st["query"])
            else:
                query = R.kv_append_rope(st["cache"], st["k_new"], st["v_new"], st["batch"], rows=rows)
            k, v = R.kv_read(st["cache"], st["back"])
            return {"k": k, "v": v} if query is None else {"q": query, "k": k, "v": v}
        if op == "tree":
            return R.kv_attend_tree(st["cache"], st["query"], st["k_new"], st["v_new"], st["batch"], st["mask"],
                                    pos=st["pos"] if st["window"] else None, window=st["window"])
        return R.verify(st["batch"], st["tokens"], st["parent"], st["p"], st["u"], st["u_next"], q=st["q"])
    if op == "rotate":
        return _turn(st["x"], st["pos"], st["rope"], st["freqs"]).half()
    if op == "append":
        rows = st.get("rows")
        if rows is None:
            pos = _rows(st["batch"])[1]
            _write(st["cache"], st["batch"], _turn(st["k_new"], pos, st["rope"], st["freqs"]), st["v_new"].float())
            return {"q": _turn(st["query"], pos, st["rope"], st["freqs"]).half(), **_read(st["cache"], st["back"])}
        _write(st["cache"], st["batch"], st["k_new"][rows.long()].float(), st["v_new"][rows.long()].float())
        return _read(st["cache"], st["back"])
    return _attend_tree(st) if op == "tree" else _decide(st)


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


def _exact_turn(c, x, pos):
    """Each pair as one complex number times gain e^(i pos f)."""
    freqs, gain = _frequencies(c)
    rot, half = c["rot"], c["rot"] // 2
    by = torch.polar(torch.tensor(gain, dtype=torch.float64, device=x.device),
                     pos.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device=x.device))[:, None]
    i = torch.arange(half, device=x.device)
    one, two = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    y = x.double().clone()
    z = torch.complex(y[..., one], y[..., two]) * by
    y[..., one], y[..., two] = z.real, z.imag
    assert y.shape[-1] >= rot
    return y


def _exact_sequence(cache, table, s, x):
    """K and V codes and scales of the first x tokens of sequence s, head by head: [x, kv, d] and [x, kv]."""
    page, kv, d = cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    t = torch.arange(x, device=table.device)
    ids = table[s].long()[t // page]
    j = torch.arange(d, device=table.device)
    tk, out = t % page, []
    where = ((tk // 4 * 4 * d + tk % 4 * 16)[:, None] + j // 16 * 64 + j % 16, (tk // 16 * 16 * d + tk % 16)[:, None] + j * 16)
    for name, place in (("k", where[0]), ("v", where[1])):
        flat = cache[name].view(-1, kv * page * d)
        out += [torch.stack([flat[ids[:, None], h * page * d + place] for h in range(kv)], 1), cache[name + "_scale"].double()[ids]]
    return out


def _exact_verify(c, st):
    """One sequence after the other, the definition as it is written."""
    host = {k: st[k].cpu() for k in ("tokens", "parent", "u", "u_next")}
    rows, count, nexts, first = [], [], [], 0
    for s, (n, _) in enumerate(_lens(c)):
        cur, path = 0, [0]
        while True:
            dist = st["p"][first + cur].double()
            draft = st["q"][first + cur].double() if st["q"] is not None else None
            accepted = None
            for j in range(1, n):
                if int(host["parent"][first + j]) != cur:
                    continue
                x = int(host["tokens"][first + j])
                one = torch.zeros_like(dist)
                one[x] = 1.0
                by = draft if draft is not None else one
                if float(host["u"][first + j]) * float(by[x]) < float(dist[x]):
                    accepted = j
                    break
                # what a rejection leaves: max(p - q, 0), and for a fixed proposal p without it, brought to mass one
                rest = (dist - by).clamp(min=0) if draft is not None else dist * (1.0 - one)
                mass = rest.sum() if draft is not None else 1.0 - dist[x]
                if not float(rest.sum()) > 0:  # nothing left: the row's own distribution decides
                    dist = st["p"][first + cur].double()
                    break
                dist = rest / mass
            if accepted is None:
                break
            cur = accepted
            path.append(cur)
        cum = torch.cumsum(dist, 0)
        nexts.append(min(int((cum <= float(host["u_next"][s]) * cum[-1]).sum()), c["vocab"] - 1))
        rows += [first + r for r in path]
        count.append(len(path))
        first += n
    at = [0]
    for x in count:
        at.append(at[-1] + x)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    return {"rows": ints(rows + [-1] * (first - len(rows))), "q_start": ints(at),
            "ctx": ints([x + k for (_, x), k in zip(_lens(c), count)]), "next": ints(nexts)}


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "rotate":
        return _exact_turn(c, st["x"], st["pos"])
    if c["op"] == "verify":
        return _exact_verify(c, st)
    lens, fmt, page, kv, d = _lens(c), c["fmt"], c["page"], c["kv"], c["d"]
    out, turned, at = [], [], 0
    for s, (n, x) in enumerate(lens):
        if c["op"] == "tree":
            kc, ks, vc, vs = _exact_sequence(st["cache"], st["batch"]["table"], s, x)
            key = torch.cat([(_exact_codes(kc, fmt) * ks[:, :, None]), st["k_new"][at : at + n].double()]).permute(1, 2, 0).contiguous()
            val = torch.cat([(_exact_codes(vc, fmt) * vs[:, :, None]), st["v_new"][at : at + n].double()]).transpose(0, 1).contiguous()
            q = st["query"][at : at + n].double().view(n, kv, -1, d).transpose(0, 1)
            far = torch.ones(n, x + n, dtype=torch.bool, device="cuda")
            for r, parent in enumerate(_parents(c)[s]):  # a row sees what its parent sees of the drafted rows, and itself
                if parent >= 0:
                    far[r, x:] = far[parent, x:]
                far[r, x + r] = False
                p = int(st["pos"][at + r])
                far[r, max(0, p - c["window"] + 1) if c["window"] else 0 : x] = False
            ys = []
            for h in range(kv):
                z = (q[h].reshape(-1, d) @ key[h]).view(n, -1, x + n) / math.sqrt(d)
                w = torch.softmax(z.masked_fill(far[:, None], -math.inf), -1)
                ys.append((w.view(-1, x + n) @ val[h]).view(n, -1, d))
            out.append(torch.stack(ys, 1).reshape(n, c["heads"], d))
            at += n
            continue
        pos = torch.arange(x - n, x, device="cuda")
        if c["nodes"]:
            take = st["rows"][at : at + n].long()
            k_new, v_new = st["k_new"][take].double(), st["v_new"][take].double()
        else:
            k_new, v_new = _exact_turn(c, st["k_new"][at : at + n], pos), st["v_new"][at : at + n].double()
            turned.append(_exact_turn(c, st["query"][at : at + n], pos))
        b0 = _open(n, x, page)
        kc, ks, vc, vs = _exact_sequence(st["cache"], st["batch"]["table"][:, b0 // page :], s, x - b0)
        back = []
        for codes, scale, new in ((_exact_codes(kc, fmt), ks, k_new), (_exact_codes(vc, fmt), vs, v_new)):
            for b in range(b0, x, page):  # block by block, as the definition says it
                a = max(b, x - n)
                fresh = new[a - (x - n) : b + page - (x - n)]
                s0 = scale[b - b0] if a > b else torch.zeros(kv, dtype=torch.float64, device=scale.device)
                s1 = torch.maximum(s0, fresh.abs().amax((0, 2)) / QMAX[fmt])
                safe = torch.where(s1 > 0, s1, 1.0)
                older = codes[b - b0 : a - b0]
                older = torch.where((s1 > s0)[None, :, None], _exact_round(older * (s0 / safe)[None, :, None], fmt), older)
                back.append(torch.cat([older, _exact_round(fresh / safe[None, :, None], fmt)]) * s1[None, :, None])
        half = len(back) // 2
        out.append((torch.cat(back[:half]), torch.cat(back[half:])))
        at += n
    if c["op"] == "tree":
        return torch.cat(out)
    done = {"k": torch.cat([o[0] for o in out]), "v": torch.cat([o[1] for o in out])}
    return done if c["nodes"] else {"q": torch.cat(turned), **done}
