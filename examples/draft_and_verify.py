"""Serving with drafted tokens on a compressed, metered KV cache.

A stack of attention layers with random weights stands in for a model.  Prompts of different lengths
arrive in chunks; then every step drafts a few tokens for each sequence, checks them all at once
(chunk attention over the cache), keeps the accepted ones and drops the rest; the last token of each
sequence is decoded with the meters.  Everything between the projections is the library's:

  witcert_rope                 positions of the queries
  witcert_write_rope_ragged    keys and values into the cache, positions on the way
  attend                       the new tokens' attention over the compressed cache
  witcert_truncate             rejected drafts leave
  decode                       one token, with its error meters

Run on a GB300: python examples/draft_and_verify.py [--scheme int8_dither] [--steps 16] [--draft 4]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kv_cache_quantization_witcert_gb300 as wc  # noqa: E402

HQ, HKV, D = 28, 4, 128           # Qwen2.5-7B's attention


class Stack:
    """n_layers of x + Wo attention(Wqkv x); the cache holds one request batch."""

    def __init__(self, n_layers, batch, max_tokens, scheme, steps, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda a, b: (torch.randn(a, b, generator=g, device="cuda") * a ** -0.5).bfloat16()
        self.layers = [(w(HQ * D, (HQ + 2 * HKV) * D), w(HQ * D, HQ * D)) for _ in range(n_layers)]
        # pages for the whole batch; a sequence's share follows its length
        self.cache = wc.Cache(n_layers, HQ, HKV, batch, max_tokens, scheme, seed=seed, total_steps=steps,
                              max_pages=batch * ((max_tokens + 15) // 16))
        self.rope = wc.Rope(D, base=1e6)
        self.batch = batch
        self.len = [0] * batch

    def project(self, layer, x, positions):
        """Rotated queries, and keys and values as the cache's writers take them (keys unrotated)."""
        qkv = x @ self.layers[layer][0]
        q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
        k, v = (t.contiguous().unflatten(1, (HKV, D)) for t in (qkv[:, HQ * D:(HQ + HKV) * D], qkv[:, (HQ + HKV) * D:]))
        return wc.witcert_rope(self.rope, positions, q), k, v

    def positions(self, n):
        return torch.cat([torch.arange(a, a + m) for a, m in zip(self.len, n)]).cuda()

    def chunk(self, x, n):
        """n[i] new tokens of sequence i, packed in x [sum n, HQ * D]: their outputs, causal over the cache."""
        at = self.positions(n)
        for layer, (_, out) in enumerate(self.layers):
            q, k, v = self.project(layer, x, at)
            self.cache.witcert_write_rope_ragged(layer, k, v, n, self.rope)
            x = x + self.cache.attend(layer, q, n).flatten(1) @ out
        self.len = [a + m for a, m in zip(self.len, n)]
        return x

    def keep(self, lengths):
        """Drop what lies beyond lengths[i] in every layer."""
        self.cache.witcert_truncate(-1, lengths)
        self.len = [min(a, b) for a, b in zip(self.len, lengths)]

    def decode(self, x, delta_req=1e-2):
        """One token a sequence, with each layer's Tier A meters."""
        at, meters = self.positions([1] * self.batch), []
        for layer, (_, out) in enumerate(self.layers):
            q, k, v = self.project(layer, x, at)
            self.cache.witcert_write_rope_ragged(layer, k, v, [1] * self.batch, self.rope)
            o, m = self.cache.decode(layer, q, delta_req)
            meters.append(m["meter_a"])
            x = x + o.bfloat16().flatten(1) @ out
        self.len = [a + 1 for a in self.len]
        return x, torch.stack(meters)


def serve(scheme="int8_dither", n_layers=4, prompts=(700, 37, 1500, 260), steps=8, draft=4, chunk=512, seed=0):
    """Returns the last outputs, their meters and the largest difference between a token's output as a
    checked draft and as a single decode."""
    g = torch.Generator().manual_seed(seed)
    B = len(prompts)
    stack = Stack(n_layers, B, max(prompts) + steps * draft + 2, scheme, steps, seed)
    token = lambda n: torch.randn(n, HQ * D, generator=g).bfloat16().cuda()
    left = list(prompts)
    while any(left):                                       # prompts, up to `chunk` tokens a call
        n = [min(chunk, m) for m in left]
        stack.chunk(token(sum(n)), n)
        left = [a - b for a, b in zip(left, n)]
    for _ in range(steps):                                 # KIVI2 cannot reopen a finished block: it keeps all
        n = [draft] * B
        before = list(stack.len)
        stack.chunk(token(B * draft), n)
        if scheme != "kivi2":
            taken = torch.randint(1, draft + 1, (B,), generator=g).tolist()
            stack.keep([a + t for a, t in zip(before, taken)])
    x = token(B)                                           # the same tokens, as drafts and as a decode
    before = list(stack.len)
    checked = stack.chunk(x, [1] * B)
    if scheme == "kivi2" and any((a + 1) % 16 == 0 for a in before):
        return checked, None, 0.0
    stack.keep(before)
    out, meters = stack.decode(x)
    return out, meters, (out.float() - checked.float()).abs().max().item()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--scheme", default="int8_dither", choices=[s for s in wc.SCHEMES if s != "blackbox"])
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--draft", type=int, default=4)
    a = p.parse_args()
    serve(a.scheme, steps=1, draft=a.draft)                # warm-up
    torch.cuda.synchronize()
    t = time.perf_counter()
    _, meters, diff = serve(a.scheme, steps=a.steps, draft=a.draft)
    torch.cuda.synchronize()
    tail = "" if meters is None else f", Tier A meters up to {meters.max().item():.3g}"
    print(f"{a.scheme}: {a.steps} steps of {a.draft} drafted tokens in {time.perf_counter() - t:.3f} s; "
          f"draft against decode {diff:.3g}{tail}")


if __name__ == "__main__":
    main()
