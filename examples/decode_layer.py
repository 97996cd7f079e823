"""One decoder layer at work: attention over the 8-bit paged cache and the
neuron-aware FFN, a batch of prompts first and then single tokens, or with
--draft trees of drafted tokens of which the verified ones stay.

    python examples/decode_layer.py [--config c1] [--heads 4] [--kv 4] [--fmt int8] [--rope] [--draft 8]

Per step and layer (x: tokens x d, fp16):
    q, k, v = W_q x, W_k x, W_v x            torch products (one matrix, so q, k and v are slices of one output)
    kv_append; a = kv_attend                 quantise k and v into the cache, attend over it
                                             (kv_append_rope where positions are rotary: q and k turned in the same launch)
    x = x + W_o a
    x = x + FFN(x)                           the predicted neurons only (pi_ffn_decode)
A step with drafted tokens:
    q, k turned (rotate); a = kv_attend_tree the drafted rows see the cache and their ancestors, and are not cached
    x as above; verify                       which rows stay, by the target's probabilities
    kv_append_rope(rows=...)                 those, by verify's lists
"""

from __future__ import annotations

import argparse
import os
import sys
import time
from typing import Optional

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from activation_sparse_predictor_amd import runtime as R  # noqa: E402
from synthetic import CONFIGS, make_layer, make_tokens  # noqa: E402


class Layer:
    """Weights and cache of one layer, and the sequences that the cache holds."""

    def __init__(self, cfg, heads: int, n_kv: int, max_tokens: int, seqs: int, fmt: str = "int8", page: int = 16,
                 device="cuda", seed: int = 0, rope: Optional[dict] = None):
        self.cfg, self.heads, self.n_kv, self.d = cfg, heads, n_kv, cfg.d // heads
        g = torch.Generator(device=device).manual_seed(seed)

        def rows(n, m):
            return (torch.randn(n, m, generator=g, device=device) / m ** 0.5).half()

        self.w_qkv = rows((heads + 2 * n_kv) * self.d, cfg.d)
        self.w_o = rows(cfg.d, cfg.d)
        self.ffn = make_layer(cfg, device=device)
        self.page, self.pages = page, -(-max_tokens // page)
        self.cache = R.kv_cache(seqs * self.pages, n_kv, self.d, page, fmt, device)
        # a sequence's pages: here simply its share of the pool
        self.table = [list(range(s * self.pages, (s + 1) * self.pages)) for s in range(seqs)]
        self.lengths = [0] * seqs
        self.rope = rope      # a plan of R.rope, for the heads' first rope["rot"] dimensions
        self.drafted = None   # of the last tree_step: keys, values, batch

    def batch(self, new) -> dict:
        """The next new[s] tokens of each sequence."""
        lengths = [x + n for x, n in zip(self.lengths, new)]
        if max(lengths) > self.pages * self.page:   # the library would clamp the length and write over the newest tokens
            raise ValueError(f"a sequence of {max(lengths)} tokens; its pages hold {self.pages * self.page}")
        self.lengths = lengths
        return R.kv_batch(new, self.lengths, self.table, self.w_o.device)

    def attention(self, x: torch.Tensor, batch: dict) -> torch.Tensor:
        n, h, kv, d = x.shape[0], self.heads, self.n_kv, self.d
        qkv = x @ self.w_qkv.t()
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([h * d, kv * d, kv * d], 1))
        if self.rope is None:
            R.kv_append(self.cache, k, v, batch)
        else:
            q = R.kv_append_rope(self.cache, k, v, batch, self.rope, q=q)
        return R.kv_attend(self.cache, q, batch).view(n, h * d) @ self.w_o.t()

    def step(self, x: torch.Tensor, new) -> torch.Tensor:
        """x: the new tokens of all sequences, one after the other (tokens x d fp16)."""
        return self.ffn_rows(x + self.attention(x, self.batch(new)))

    def tree_step(self, x: torch.Tensor, parents) -> torch.Tensor:
        """x: each sequence's newest token and the ones drafted below it, parents[s] their parents in
        the sequence (-1 for the first).  Nothing is cached until `keep`."""
        n, h, kv, d = x.shape[0], self.heads, self.n_kv, self.d
        counts = [len(p) for p in parents]
        if max(c + m for c, m in zip(self.lengths, counts)) > self.pages * self.page:
            raise ValueError(f"more tokens than a sequence's pages hold, {self.pages * self.page}")
        batch, tree = R.kv_batch(counts, self.lengths, self.table, x.device), R.kv_tree(parents, x.device)
        qkv = x @ self.w_qkv.t()
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([h * d, kv * d, kv * d], 1))
        if self.rope is not None:   # q and k lie side by side: one call turns both in place
            pos = torch.tensor([c for c, m in zip(self.lengths, counts) for _ in range(m)], dtype=torch.int32, device=x.device)
            qk = qkv[:, :(h + kv) * d].unflatten(1, (-1, d))
            R.rotate(qk, pos + tree["depth"], self.rope, out=qk)
        self.drafted = k, v, batch, tree["parent"]
        a = R.kv_attend_tree(self.cache, q, k, v, batch, tree["mask"]).view(n, h * d) @ self.w_o.t()
        return self.ffn_rows(x + a)

    def keep(self, tokens: torch.Tensor, p: torch.Tensor, u: torch.Tensor, u_next: torch.Tensor,
             q: Optional[torch.Tensor] = None) -> dict:
        """Verifies the last tree_step's tokens and caches those that stay.  Returns verify's results."""
        k, v, batch, parent = self.drafted
        kept = R.verify(batch, tokens, parent, p, u, u_next, q=q)
        R.kv_append_rope(self.cache, k, v, {**batch, **kept}, rows=kept["rows"])
        self.lengths = kept["ctx"].tolist()
        return kept

    def ffn_rows(self, x: torch.Tensor) -> torch.Tensor:
        out = []
        for part in x.split(128):   # the FFN takes up to 256 tokens a call
            y, _, _ = R.decode(self.ffn, part.contiguous())
            out.append(part + y.half())
        return torch.cat(out)


def drafting(layer: Layer, cfg, seqs: int, drafts: int, steps: int, vocab: int = 1000) -> None:
    """Steps with drafted tokens: a random embedding, which is the output layer too, and proposals from a random table."""
    g = torch.Generator(device="cuda").manual_seed(1)
    embed = (torch.randn(vocab, cfg.d, generator=g, device="cuda") / cfg.d ** 0.5).half()
    table = torch.randint(0, vocab, (vocab, 2), generator=g, device="cuda")
    newest = torch.randint(0, vocab, (seqs,), generator=g, device="cuda")
    parents = [-1] + [max(0, (j - 1) // 2) for j in range(1, drafts + 1)]   # two proposals a token
    total = 0
    for _ in range(steps):
        rows = [newest]
        for j in range(1, drafts + 1):
            rows.append(table[rows[parents[j]], j % 2])
        tokens = torch.stack(rows, 1).flatten()
        y = layer.tree_step(embed[tokens] * 30.0, [parents] * seqs)
        p = torch.softmax((y @ embed.t()).float(), 1)
        u, u_next = (torch.rand(n, generator=g, device="cuda") for n in (len(tokens), seqs))
        kept = layer.keep(tokens.int(), p, u, u_next)
        total += int(kept["q_start"][-1])
        newest = kept["next"].long()
    print(f"{cfg.workload}: {seqs} sequences, {steps} steps with {drafts} drafted tokens: {total / steps / seqs:.2f} tokens a step stayed, "
          f"lengths {min(layer.lengths)} to {max(layer.lengths)}")


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="c1", choices=sorted(CONFIGS))
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--kv", type=int, default=4)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--fmt", default="int8", choices=["int8", "fp8"])
    ap.add_argument("--rope", action="store_true", help="rotary positions")
    ap.add_argument("--draft", type=int, default=0, help="drafted tokens of a step and sequence, verified against random targets")
    a = ap.parse_args()
    cfg = CONFIGS[a.config]
    rope = R.rope(cfg.d // a.heads) if a.rope else None
    layer = Layer(cfg, a.heads, a.kv, a.prompt + a.tokens * (1 + a.draft), a.seqs, a.fmt, rope=rope)
    x = make_tokens(cfg, a.seqs * a.prompt, device="cuda")
    x = layer.step(x, [a.prompt] * a.seqs).view(a.seqs, a.prompt, cfg.d)[:, -1].contiguous()
    if a.draft:
        return drafting(layer, cfg, a.seqs, a.draft, a.tokens)
    for i in range(a.tokens):
        if i == a.tokens // 2:   # the first half warms the libraries up
            torch.cuda.synchronize()
            t = time.perf_counter()
        x = layer.step(x, [1] * a.seqs)
        x = x / x.float().square().mean(1, keepdim=True).sqrt().half()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / (a.tokens - a.tokens // 2) * 1e6
    print(f"{cfg.workload}: {a.seqs} sequences of {layer.lengths[0]} tokens, {a.heads} heads of {layer.d} ({a.kv} kv), "
          f"{a.fmt} cache: {us:.0f} us a step, |x| max {float(x.abs().max()):.3f}")


if __name__ == "__main__":
    main()
