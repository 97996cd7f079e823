"""One decoder layer at work: attention over the 8-bit paged cache and the
neuron-aware FFN, a batch of prompts first and then single tokens.

    python examples/decode_layer.py [--config c1] [--heads 4] [--kv 4] [--fmt int8]

Per step and layer (x: tokens x d, fp16):
    q, k, v = W_q x, W_k x, W_v x            torch products (one matrix, so q, k and v are slices of one output)
    kv_append; a = kv_attend                 quantise k and v into the cache, attend over it
    x = x + W_o a
    x = x + FFN(x)                           the predicted neurons only (pi_ffn_decode)
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from activation_sparse_predictor_amd import runtime as R  # noqa: E402
from synthetic import CONFIGS, make_layer, make_tokens  # noqa: E402


class Layer:
    """Weights and cache of one layer, and the sequences that the cache holds."""

    def __init__(self, cfg, heads: int, n_kv: int, max_tokens: int, seqs: int, fmt: str = "int8", page: int = 16,
                 device="cuda", seed: int = 0):
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
        R.kv_append(self.cache, k, v, batch)
        return R.kv_attend(self.cache, q, batch).view(n, h * d) @ self.w_o.t()

    def step(self, x: torch.Tensor, new) -> torch.Tensor:
        """x: the new tokens of all sequences, one after the other (tokens x d fp16)."""
        x = x + self.attention(x, self.batch(new))
        out = []
        for part in x.split(128):   # the FFN takes up to 256 tokens a call
            y, _, _ = R.decode(self.ffn, part.contiguous())
            out.append(part + y.half())
        return torch.cat(out)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="c1", choices=sorted(CONFIGS))
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--kv", type=int, default=4)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--fmt", default="int8", choices=["int8", "fp8"])
    a = ap.parse_args()
    cfg = CONFIGS[a.config]
    layer = Layer(cfg, a.heads, a.kv, a.prompt + a.tokens, a.seqs, a.fmt)
    x = make_tokens(cfg, a.seqs * a.prompt, device="cuda")
    x = layer.step(x, [a.prompt] * a.seqs).view(a.seqs, a.prompt, cfg.d)[:, -1].contiguous()
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
