"""A verify step of speculative decoding over packed weights, with the calls in
the order an engine makes them: the q/k/v projections of the drafted rows as one
grouped verify call, rotary positions and the append to the paged cache, the
attention of the rows over that cache, the output projection, the head, and
sampling, which accepts the drafted prefix that the samples agree with.

The model is one small attention layer with random weights.  Run it on a GB300:

    python examples/verify_step.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import few_row_packed_gb300 as lbv  # noqa: E402
import synth  # noqa: E402


class Layer:
    """Attention with Q4_0 projections, and a 2-bit output head."""

    def __init__(self, hidden=512, heads=8, kv_heads=2, head_dim=64, vocab=2000, pages=64,
                 page_size=16, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, head_dim
        self.vocab = vocab
        q, kv = heads * head_dim, kv_heads * head_dim
        self.qkv = lbv.Group(lbv.FMT_Q4_0, 32, lbv.F16, [(hidden, q), (hidden, kv), (hidden, kv)])
        self.out = lbv.Plan(lbv.FMT_Q4_0, q, hidden, 32, lbv.F16)
        self.head = lbv.Plan(lbv.FMT_AFFINE2, hidden, vocab, 64, lbv.F16)
        shapes = [(lbv.FMT_Q4_0, synth.Q4_0, hidden, q, 32), (lbv.FMT_Q4_0, synth.Q4_0, hidden, kv, 32),
                  (lbv.FMT_Q4_0, synth.Q4_0, hidden, kv, 32), (lbv.FMT_Q4_0, synth.Q4_0, q, hidden, 32),
                  (lbv.FMT_AFFINE2, synth.AFFINE2, hidden, vocab, 64)]
        self.weights = []
        for i, (fmt, name, k, n, group) in enumerate(shapes):
            parts, _ = synth.gen_matrix(synth.Matrix(f"w{i}", name, k, n, group, "f16", sigma_scale=0.01),
                                        [seed, i], rows=1)
            self.weights.append(torch.from_numpy(lbv.pack(fmt, parts, k, n, group)).cuda())
        rng = np.random.default_rng(seed)
        self.embedding = torch.from_numpy(rng.standard_normal((vocab, hidden)).astype(np.float16)).cuda()
        cache = (pages, page_size, kv_heads, head_dim)
        self.cache = lbv.KVCache(torch.zeros(cache, dtype=torch.float16, device="cuda"),
                                 torch.zeros(cache, dtype=torch.float16, device="cuda"))
        self.rope = lbv.Rope(lbv.rope_frequencies(head_dim))
        self.table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)[None].cuda()
        probe = lbv.Batch(*self._counts(1, 1), self.table, 8)
        self.workspace = torch.zeros(lbv.attend_workspace_bytes(self.cache, probe, heads),
                                     dtype=torch.uint8, device="cuda")

    @staticmethod
    def _counts(n, context):
        return (torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                torch.tensor([context], dtype=torch.int32, device="cuda"))

    def logits(self, tokens, context):
        """Logits of up to 8 new tokens after `context` cached ones; their keys and
        values enter the cache."""
        n = len(tokens)
        x = self.embedding[torch.tensor(tokens, device="cuda")].contiguous()
        rows = [torch.empty((n, h, self.dim), dtype=torch.float32, device="cuda")
                for h in (self.heads, self.kv_heads, self.kv_heads)]
        lbv.verify_grouped(self.qkv, [(x, n, w, y) for w, y in zip(self.weights, rows)])
        batch = lbv.Batch(*self._counts(n, context + n), self.table, n)
        q = torch.empty((n, self.heads, self.dim), dtype=torch.float16, device="cuda")
        lbv.rope_append(self.rope, batch, self.cache, *rows, q)
        attended = torch.empty_like(q)
        lbv.attend(self.cache, batch, q, attended, self.dim ** -0.5, workspace=self.workspace)
        y = torch.empty((n, self.hidden), dtype=torch.float32, device="cuda")
        lbv.verify_gemm(self.out, attended, n, self.weights[3], y)
        x = x.float() + y
        x = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).half()
        z = torch.empty((n, self.vocab), dtype=torch.float32, device="cuda")
        lbv.verify_gemm(self.head, x, n, self.weights[4], z)
        return z

    def verify(self, last, drafts, context, u, **rules):
        """One step: the last accepted token and the drafts after it go through the
        layer together; returns the tokens it settles (a drafted prefix that the
        samples agree with, and one more)."""
        z = self.logits([last, *drafts], context)
        token = torch.empty(z.shape[0], dtype=torch.int32, device="cuda")
        lbv.sample(z, u[:z.shape[0]], token, **rules)
        sampled = token.tolist()
        same = 0
        while same < len(drafts) and drafts[same] == sampled[same]:
            same += 1
        return sampled[:same + 1]


def main():
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens, steps = [1], 0
    rules = {"temperature": torch.full((8,), 0.8, device="cuda"),
             "top_p": torch.full((8,), 0.9, device="cuda"),
             "top_k": torch.full((8,), 50, dtype=torch.int32, device="cuda")}
    guess = {}                  # drafts: what followed this token the last time
    while len(tokens) < 100:
        drafts, t = [], tokens[-1]
        while len(drafts) < 7 and t in guess:
            t = guess[t]
            drafts.append(t)
        u = torch.rand(8, generator=g, device="cuda")
        settled = layer.verify(tokens[-1], drafts, len(tokens) - 1, u, **rules)
        for a, b in zip([tokens[-1], *settled], settled):
            guess[a] = b
        tokens += settled
        steps += 1
    lbv.attend_status(layer.workspace)
    print(f"{len(tokens) - 1} tokens in {steps} steps:", tokens)


if __name__ == "__main__":
    main()
