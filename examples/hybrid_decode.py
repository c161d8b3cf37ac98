"""Speculative decoding of a small hybrid stack with this library's calls.

The stack has three recurrent layers to one attention layer, random weights
and a bigram table as the draft model.  One step, for N requests at once:

  1. the draft model proposes K tokens after each request's last one;
  2. the stack runs over the last token and the drafts: every recurrent layer
     by kda_decode_verify (its state is only read), every attention layer by
     kda_cache_append and kda_cache_attend;
  3. kda_draft_accept decides how many drafts each request keeps and draws the
     token after them;
  4. kda_decode_commit advances the recurrent states by what was kept, and the
     caches' lens advance by the same counts (rows of dropped drafts are
     written again by the next step).

Run:  python examples/hybrid_decode.py [--requests 8] [--drafts 4] [--steps 16]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_recurrence_fwd_gb300 import (  # noqa: E402
    PagedCache, binding, kda_cache_append, kda_cache_attend, kda_draft_accept)


class HybridStack:
    """layers: "r" (recurrent, H heads of 128) or "a" (attention, H heads on
    H_kv key heads of 128, rotated by position, pages of 16 tokens)."""

    def __init__(self, requests, layers="rrra", H=4, H_kv=2, vocabulary=1000, max_tokens=512, page=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers, self.H, self.H_kv, self.V, self.N = layers, H, H_kv, vocabulary, requests
        self.width = 128 * H

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(rows)

        self.embedding = torch.randn((vocabulary, self.width), generator=g, device="cuda")
        self.draft = torch.softmax(2 * torch.randn((vocabulary, vocabulary), generator=g, device="cuda"), -1)
        self.head = 2 * weight(self.width, vocabulary)
        self.inv_freq = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        pages = max_tokens // page
        table = torch.randperm(requests * pages, generator=g, device="cuda").to(torch.int32).view(requests, pages)
        self.weights, self.held = [], []  # what a layer keeps of each request: states, or a paged cache
        for kind in layers:
            out = weight(self.width, self.width)
            if kind == "r":
                self.weights.append((weight(self.width, self.width * 4 + H), out))
                self.held.append(torch.zeros((requests, H, 128, 128), device="cuda"))
            else:
                self.weights.append((weight(self.width, 128 * (H + 2 * H_kv)), out))
                pools = [torch.empty((requests * pages, page, H_kv, 128), dtype=torch.bfloat16, device="cuda")
                         for _ in range(2)]
                self.held.append(PagedCache(*pools, table, self.lens))

    def forward(self, tokens):
        """Probabilities [N, K, V] after each of tokens [N, K], and what commit() needs."""
        N, K = tokens.shape
        x = self.embedding[tokens.long()]
        inputs = []
        for kind, (w_in, w_out), held in zip(self.layers, self.weights, self.held):
            y = torch.nn.functional.rms_norm(x, (self.width,)) @ w_in
            if kind == "r":
                q, k, v, decay = (t.unflatten(-1, (self.H, 128)) for t in y[..., :4 * self.width].split(self.width, -1))
                parts = [torch.nn.functional.normalize(q, dim=-1), torch.nn.functional.normalize(k, dim=-1), v,
                         -5 * torch.sigmoid(decay), torch.sigmoid(y[..., 4 * self.width:])]
                parts = [t.to(torch.bfloat16).contiguous() for t in parts]
                out = binding.kda_decode_verify(*parts, held)
                inputs.append(parts)
            else:
                q, k, v = y.to(torch.bfloat16).split([128 * self.H, 128 * self.H_kv, 128 * self.H_kv], -1)
                q, k, v = (t.unflatten(-1, (-1, 128)) for t in (q, k, v))  # slices of the projection, not copies
                q = kda_cache_append(k, v, held, q=q, inv_freq=self.inv_freq)
                out = kda_cache_attend(q, held)
                inputs.append(None)
            x = x + out.float().flatten(-2) @ w_out
        return torch.softmax(torch.nn.functional.rms_norm(x, (self.width,)) @ self.head, -1), inputs

    def commit(self, inputs, counts):
        """Keep the first counts[n] of the tokens that forward() ran over."""
        for held, parts in zip(self.held, inputs):
            if parts is not None:
                binding.kda_decode_commit(*parts, held, counts)
        self.lens.add_(counts)

    def step(self, last, K, generator):
        """One speculative step from each request's last token [N].  Returns
        (counts [N], tokens [N, K + 1], the new last tokens)."""
        drafts, probs, at = [], [], last.long()
        for _ in range(K):
            probs.append(self.draft[at])
            at = torch.multinomial(probs[-1], 1, generator=generator)[:, 0]
            drafts.append(at)
        drafts = torch.stack(drafts, 1).to(torch.int32)
        target, inputs = self.forward(torch.cat([last[:, None].to(torch.int32), drafts], 1))
        uniform = torch.rand((self.N, K + 1), generator=generator, device="cuda")
        counts, tokens = kda_draft_accept(drafts, torch.stack(probs, 1), target, uniform)
        self.commit(inputs, counts)
        return counts, tokens, tokens.gather(1, (counts - 1).long()[:, None])[:, 0]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    stack = HybridStack(a.requests, max_tokens=16 * ((a.steps + 1) * (a.drafts + 1) // 16 + 2))
    generator = torch.Generator(device="cuda").manual_seed(1)
    last = torch.arange(a.requests, device="cuda", dtype=torch.int32)
    gained = torch.zeros((), dtype=torch.int64, device="cuda")
    _, _, last = stack.step(last, a.drafts, generator)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.steps):
        counts, _, last = stack.step(last, a.drafts, generator)
        gained += counts.sum()
    n = int(gained)
    spent = time.perf_counter() - began
    print(f"{a.requests} requests, {a.steps} steps of {a.drafts} drafts: {n / a.steps / a.requests:.2f} tokens a step "
          f"and request, {n / spent:.0f} tokens/s; device status {binding.kda_last_device_status()}")


if __name__ == "__main__":
    main()
