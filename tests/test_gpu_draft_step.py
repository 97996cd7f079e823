"""The operators of a speculative decoding step together, as a serving loop
calls them: the example's layer against the oracles, stage by stage, and the
whole step captured and replayed without the host in between."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from activation_sparse_predictor_amd import runtime as R
from examples.decode_layer import Layer, drafting
from oracle import draft as O
from oracle import kv as K
from synthetic import CONFIGS, make_tokens
from tests.test_gpu_kv import DEV, garbage_cache, host, host_batch, tables
from tests.test_gpu_rope import near

pytestmark = pytest.mark.gpu


def tree_of(n, rng):
    return [-1] + [max(0, j - 1 - int(rng.exponential(1.5))) for j in range(1, n)]


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("heads,n_kv,rot,layout", [(4, 4, 64, "half"), (4, 2, 32, "half"), (16, 1, 16, "pairs")])
def test_layer_drafts(fmt, heads, n_kv, rot, layout):
    """Prompts with rotary positions, then trees of which the verified rows are cached.  Compared: turned queries and
    keys, attention over cache and tree on what the layer holds (test_gpu_kv.py's bound), verify's whole numbers,
    and the cache after the accepted rows, code for code."""
    cfg = CONFIGS["c1"]
    plan = R.rope(rot, layout=layout, device=DEV)
    freqs, _ = O.frequencies(rot)
    layer = Layer(cfg, heads, n_kv, 64, 3, fmt, rope=plan)
    d, rng = layer.d, np.random.default_rng(heads)
    layer.step(make_tokens(cfg, 12).to(DEV), [5, 1, 6])
    assert layer.lengths == [5, 1, 6]
    vocab = 211
    for counts in ([6, 1, 9], [1, 7, 3]):
        parents = [tree_of(n, rng) for n in counts]
        tok = sum(counts)
        x = make_tokens(cfg, tok).to(DEV)
        before = list(layer.lengths)
        y = layer.tree_step(x, parents)
        assert y.shape == x.shape and layer.lengths == before
        k, v, batch, parent = layer.drafted
        t = R.kv_tree(parents, DEV)
        pos = np.repeat(before, counts) + t["depth"].cpu().numpy()
        qkv = (x @ layer.w_qkv.t()).cpu().numpy()
        q0, k0, v0 = (a.reshape(tok, -1, d) for a in np.split(qkv, [heads * d, (heads + n_kv) * d], 1))
        near(k.cpu().numpy(), O.rotate(k0, pos, freqs, layout), k0, rot, layout, 1.0)
        assert np.array_equal(v.cpu().numpy(), v0)
        q = R.rotate(torch.from_numpy(q0).to(DEV), torch.from_numpy(pos.astype(np.int32)).to(DEV), plan)
        a = R.kv_attend_tree(layer.cache, q, k, v, batch, t["mask"])
        was = host({n: c.clone() if isinstance(c, torch.Tensor) else c for n, c in layer.cache.items()})
        want, _, bound = O.attend_tree(was, host_batch(batch), q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(),
                                       t["mask"].cpu().numpy().view(np.uint64), d ** -0.5)
        assert np.all(np.abs(a.cpu().numpy() - want) <= 2.0 ** -11 * np.abs(want) + 1.25 * 2.0 ** -10 * bound + 2.0 ** -25)
        mid = x + a.view(tok, -1) @ layer.w_o.t()
        assert torch.equal(y, layer.ffn_rows(mid))
        p = torch.softmax(torch.from_numpy(rng.standard_normal((tok, vocab)).astype(np.float32)).to(DEV) * 3, 1)
        q_draft = torch.softmax(p.log() * 0.5, 1)
        tokens = torch.from_numpy(rng.integers(0, vocab, tok).astype(np.int32)).to(DEV)
        tokens[1::2] = p.argmax(1).int()[torch.from_numpy(np.maximum(parent.cpu().numpy(), 0)).to(DEV) + torch.repeat_interleave(
            batch["q_start"][:-1], torch.tensor(counts, device=DEV))][1::2]
        u, u_next = (torch.from_numpy(rng.random(n, dtype=np.float32)).to(DEV) for n in (tok, 3))
        kept = layer.keep(tokens, p, u, u_next, q=q_draft)
        rows, start, ctx, nxt = O.verify(host_batch(batch)["q_start"], before, tokens.tolist(), parent.tolist(), p.cpu().numpy(),
                                         u.tolist(), u_next.tolist(), q_draft.cpu().numpy())
        assert kept["rows"].tolist() == rows and kept["q_start"].tolist() == start and kept["next"].tolist() == nxt
        assert layer.lengths == ctx
        stay = rows[:start[-1]]
        after = K.append(was, {"q_start": start, "ctx": ctx, "table": layer.table}, k.cpu().numpy()[stay], v.cpu().numpy()[stay])
        got = host(layer.cache)
        for s in range(3):
            for pg in layer.table[s][:-(-ctx[s] // 16)]:
                for n in ("k", "v"):
                    used = min(16, ctx[s] - layer.table[s].index(pg) * 16)
                    at = K.places(16, d)["kv".index(n)][:used]
                    for h in range(n_kv):
                        assert np.array_equal(K.decode(got[n][pg, h].reshape(-1)[at], fmt), K.decode(after[n][pg, h].reshape(-1)[at], fmt))
                    assert np.array_equal(got[n + "_scale"][pg], after[n + "_scale"][pg])


def test_the_example_drafts():
    cfg = CONFIGS["c1"]
    layer = Layer(cfg, 4, 2, 200, 3, "int8", rope=R.rope(cfg.d // 4))
    layer.step(make_tokens(cfg, 9).to(DEV), [3, 3, 3])
    drafting(layer, cfg, 3, 6, 5)
    assert all(3 + 5 <= n <= 3 + 5 * 7 for n in layer.lengths)


def test_a_whole_step_replayed():
    """rotate, kv_attend_tree, verify and kv_append_rope in one graph: the lengths that verify leaves on the device
    are the next step's, with no copy to the host between the replays."""
    seqs, n, heads, n_kv, d, vocab, page = 3, 7, 8, 2, 64, 500, 16
    rng = np.random.default_rng(5)
    start = [30, 700, 1]
    table, n_pages = tables([x + 80 for x in start], page, rng)
    plan = R.rope(d, device=DEV)
    tree = R.kv_tree([[-1, 0, 0, 1, 1, 2, 4]] * seqs, DEV)
    caches = []
    for _ in range(2):
        c = garbage_cache(n_pages, n_kv, d, page, "int8")
        for m in ("k", "v"):
            c[m].zero_()
        old = torch.from_numpy(np.random.default_rng(6).standard_normal((sum(start), n_kv, d)).astype(np.float16)).to(DEV)
        R.kv_append_rope(c, old, old, R.kv_batch(start, start, table, DEV), plan)
        caches.append(c)
    of = torch.arange(seqs, device=DEV).repeat_interleave(n)

    def step(cache, batch, s):
        pos = (batch["ctx"][of] + tree["depth"]).int()
        q, k = R.rotate(s["q"], pos, plan), R.rotate(s["k"], pos, plan)
        y = R.kv_attend_tree(cache, q, k, s["v"], batch, tree["mask"], pos=pos, window=300)
        kept = R.verify(batch, s["tokens"], tree["parent"], s["p"], s["u"], s["u_next"], q=s["draft"])
        R.kv_append_rope(cache, k, s["v"], {**batch, **kept}, rows=kept["rows"])
        batch["ctx"].copy_(kept["ctx"])
        return y, kept["rows"], kept["next"]

    def inputs(seed):
        r = np.random.default_rng(seed)
        p = torch.softmax(torch.from_numpy(r.standard_normal((seqs * n, vocab)).astype(np.float32)) * 3, 1)
        out = {"q": r.standard_normal((seqs * n, heads, d)).astype(np.float16), "k": r.standard_normal((seqs * n, n_kv, d)).astype(np.float16),
               "v": r.standard_normal((seqs * n, n_kv, d)).astype(np.float16), "u": r.random(seqs * n, dtype=np.float32),
               "u_next": r.random(seqs, dtype=np.float32)}
        out = {m: torch.from_numpy(a).to(DEV) for m, a in out.items()}
        tokens = p.argmax(1)[torch.clamp(tree["parent"].cpu().long(), min=0) + of.cpu() * n].int()
        return {**out, "p": p.to(DEV), "draft": torch.softmax(p.log() * 0.8, 1).to(DEV), "tokens": tokens.to(DEV)}

    fixed = inputs(0)
    batches = [R.kv_batch([n] * seqs, start, table, DEV) for _ in range(2)]
    step(caches[0], dict(batches[0], ctx=batches[0]["ctx"].clone()), fixed)   # once before the capture ...
    step(caches[1], dict(batches[1], ctx=batches[1]["ctx"].clone()), fixed)   # ... on both caches
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0], batches[0], fixed)
    grown = 0
    for turn in range(1, 9):
        new = inputs(turn)
        for m, t in new.items():
            fixed[m].copy_(t)
        graph.replay()
        want = step(caches[1], batches[1], new)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn
        assert torch.equal(batches[0]["ctx"], batches[1]["ctx"])
    grown = batches[0]["ctx"].tolist()
    assert all(a + 8 <= b <= a + 8 * 4 for a, b in zip(start, grown)) and sum(grown) > sum(start) + 8 * seqs
    for m in ("k", "v"):
        assert torch.equal(caches[0][m + "_scale"].nan_to_num(-1), caches[1][m + "_scale"].nan_to_num(-1))
        assert torch.equal(caches[0][m], caches[1][m])
