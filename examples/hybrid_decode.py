"""Speculative decoding of a small hybrid stack with this library's calls.

The stack mixes recurrent layers ("r": the gated delta rule, "l": linear
attention with a decay per head) and attention layers ("a"), by default three
recurrent ones to one of attention, with random weights and a bigram table as
the draft model.  One step, for N requests at once:

  1. the draft model proposes K tokens after each request's last one;
  2. the stack runs over the last token and the drafts: every recurrent layer
     by kda_decode_verify or kda_linear_verify (its state is only read), every
     attention layer by kda_cache_append and kda_cache_attend; with a
     temperature or a penalty for what has been said, the logits go through
     kda_logits_probs;
  3. kda_draft_accept decides how many drafts each request keeps and draws the
     token after them;
  4. kda_decode_commit and kda_linear_commit advance the recurrent states by
     what was kept, and the caches' lens advance by the same counts (rows of dropped drafts are
     written again by the next step).

Run:  python examples/hybrid_decode.py [--requests 8] [--drafts 4] [--steps 16]
          [--layers rrra] [--temperature 1] [--repetition 1]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_recurrence_fwd_gb300 import (  # noqa: E402
    PagedCache, binding, kda_cache_append, kda_cache_attend, kda_draft_accept, kda_linear_commit, kda_linear_verify,
    kda_logits_probs)


class HybridStack:
    """layers: "r" or "l" (recurrent, H heads of 128) or "a" (attention, H heads
    on H_kv key heads of 128, rotated by position, pages of 16 tokens).
    temperature and repetition (kda_logits_probs) may be given together."""

    def __init__(self, requests, layers="rrra", H=4, H_kv=2, vocabulary=1000, max_tokens=512, page=16, seed=0,
                 temperature=None, repetition=None):
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
        self.rules = None
        if temperature is not None or repetition is not None:
            # what each request has said: the tokens before position lens, and the last one
            self.said = torch.full((requests, max_tokens + 1), -1, dtype=torch.int32, device="cuda")
            each = [torch.full((requests,), 1.0 if x is None else x, device="cuda") for x in (temperature, repetition)]
            self.rules = {"temperature": each[0], "repetition": each[1]}
        pages = max_tokens // page
        table = torch.randperm(requests * pages, generator=g, device="cuda").to(torch.int32).view(requests, pages)
        self.weights, self.held = [], []  # what a layer keeps of each request: states, or a paged cache
        for kind in layers:
            out = weight(self.width, self.width)
            if kind == "r":
                self.weights.append((weight(self.width, self.width * 4 + H), out))
                self.held.append(torch.zeros((requests, H, 128, 128), device="cuda"))
            elif kind == "l":
                self.weights.append((weight(self.width, self.width * 3 + H), out))
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
            elif kind == "l":
                q, k, v = (t.unflatten(-1, (self.H, 128)) for t in y[..., :3 * self.width].split(self.width, -1))
                parts = [torch.nn.functional.normalize(q, dim=-1), torch.nn.functional.normalize(k, dim=-1), v,
                         -torch.nn.functional.softplus(y[..., 3 * self.width:])]
                parts = [t.to(torch.bfloat16).contiguous() for t in parts]
                out = kda_linear_verify(*parts, held)
                inputs.append(parts)
            else:
                q, k, v = y.to(torch.bfloat16).split([128 * self.H, 128 * self.H_kv, 128 * self.H_kv], -1)
                q, k, v = (t.unflatten(-1, (-1, 128)) for t in (q, k, v))  # slices of the projection, not copies
                q = kda_cache_append(k, v, held, q=q, inv_freq=self.inv_freq)
                out = kda_cache_attend(q, held)
                inputs.append(None)
            x = x + out.float().flatten(-2) @ w_out
        logits = torch.nn.functional.rms_norm(x, (self.width,)) @ self.head
        if self.rules is None:
            return torch.softmax(logits, -1), inputs
        # the first of the tokens is said, the others are drafts that are said if the rows after them count
        self.said.scatter_(1, self.lens.long()[:, None], tokens[:, :1].to(torch.int32))
        return kda_logits_probs(logits, tokens=self.said, lens=self.lens + 1, drafts=tokens[:, 1:].to(torch.int32).contiguous(),
                                **self.rules), inputs

    def commit(self, inputs, counts):
        """Keep the first counts[n] of the tokens that forward() ran over."""
        for kind, held, parts in zip(self.layers, self.held, inputs):
            if kind == "r":
                binding.kda_decode_commit(*parts, held, counts)
            elif kind == "l":
                kda_linear_commit(*parts[1:], held, counts)
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
        if self.rules is not None:  # what was gained, behind the last token; what was not (-1) is written over
            at = self.lens.long()[:, None] + 1 + torch.arange(K + 1, device="cuda")
            self.said.scatter_(1, at.clamp(max=self.said.shape[1] - 1), tokens)
        self.commit(inputs, counts)
        return counts, tokens, tokens.gather(1, (counts - 1).long()[:, None])[:, 0]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--layers", default="rrra")
    ap.add_argument("--temperature", type=float)
    ap.add_argument("--repetition", type=float)
    a = ap.parse_args()
    stack = HybridStack(a.requests, a.layers, max_tokens=16 * ((a.steps + 1) * (a.drafts + 1) // 16 + 2),
                        temperature=a.temperature, repetition=a.repetition)
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
