"""The n best continuations of one prompt, with their log probabilities.

A toy target (two layers of softmax attention with normed queries and keys, the first with a sliding window
and first tokens that stay visible, W4A16 projections, int8 lm_head, random weights) reads a prompt once.
Its n most likely next tokens begin n continuations: sequences forked from the prompt's, which share its
pages and, in the layer that sees everything, its attention.  They are decoded greedily side by side; each
step scores the tokens that it takes, and the continuations are ranked by the sum.

    python examples/continuations.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verify_w4a16_gb300 import inputs, w4v  # noqa: E402

H, V, LAYERS, Q_HEADS, KV_HEADS, D, PAGE, WINDOW, SINKS = 256, 1024, 2, 8, 2, 64, 16, 40, 4


class Target:
    def __init__(self, seed: int, device="cuda"):
        E, _, W8, s8 = inputs.toy_model_arrays(seed, V=V, H=H, layers=LAYERS)
        dev = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
        lin = lambda n, k, tag, i: (dev(w4v.pack_int4(inputs.w4_codes(seed, n, k, tag, i))),  # noqa: E731
                                    dev(inputs.w4_scales(seed, n, k, tag, i)), n)
        self.E, self.W8, self.s8 = dev(E), dev(W8), dev(s8)
        self.qkv = [lin((Q_HEADS + 2 * KV_HEADS) * D, H, "qkv", i) for i in range(LAYERS)]
        self.out = [lin(H, Q_HEADS * D, "attn-out", i) for i in range(LAYERS)]
        g = torch.Generator().manual_seed(seed)
        weight = lambda: (torch.randn(D, generator=g) * 0.2).half().to(device)  # noqa: E731
        self.norm = [w4v.HeadNorm(weight(), weight(), zero_centred=True) for _ in range(LAYERS)]
        self.rope = w4v.Rope(D, device=device)

    def logits(self, tokens, cache, offsets, rows=None):
        """Logits after new tokens that the cache has pages for already (of `rows` of them)."""
        h = self.E[tokens].float()
        for i in range(LAYERS):
            k_cache, v_cache = cache.pool[2 * i], cache.pool[2 * i + 1]
            at = (k_cache, v_cache, cache.table, cache.lengths, offsets)
            packed, scales, n = self.qkv[i]
            q, k, v = w4v.w4a16_gemm(rms(h), packed, scales, n).unflatten(1, (-1, D)).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q = w4v.norm_rope_append(q, k, v, *at, self.rope, self.norm[i])
            if i == 0:
                o = w4v.paged_attn(q, *at, window=WINDOW, sinks=SINKS)
            else:
                o = w4v.paged_attn_shared(q, *at, cache.groups, cache.prefix)
            packed, scales, n = self.out[i]
            h = h + w4v.w4a16_gemm(o.flatten(1), packed, scales, n).float()
        x = rms(h if rows is None else h[rows])
        logits = torch.empty((x.shape[0], V), dtype=torch.float32, device=x.device)
        w4v.w8_lmhead_argmax(x, self.W8, self.s8, logits=logits)
        return logits


def rms(x):
    return (x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()).half()


class Cache:
    """Pages of both layers; the sequences from 0 to n - 1 are one group whose prefix is the prompt."""

    def __init__(self, sequences: int, pages: int, device="cuda"):
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.pool = torch.zeros((2 * LAYERS, pages, KV_HEADS, PAGE, D), dtype=torch.float16, device=device)
        self.refs, self.table, self.lengths, self.prefix = i32(pages), i32(sequences, pages) - 1, i32(sequences), i32(1)
        self.groups = torch.tensor([0, sequences], dtype=torch.int32, device=device)

    def extend(self, new):
        if int(w4v.kv_extend(self.pool, self.refs, self.table, self.lengths, self.lengths + new)):
            raise RuntimeError("the cache is full")


def main(seed: int = 7, count: int = 16, n: int = 8):
    """(sum of log probabilities, tokens, their log probabilities) of n continuations of `count` tokens, best first."""
    w4v.init()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    target, cache = Target(seed), Cache(n, pages=16 + 4 * n)
    prompt = torch.tensor([int(t) for t in inputs.random_tokens(seed, 100, V)], device="cuda")
    size = len(prompt)
    cache.extend(i32([size] + [0] * (n - 1)))
    first = target.logits(prompt, cache, i32([0] + [size] * n), rows=[size - 1])
    _, _, ids, logprobs = w4v.token_logprobs(first, top=n)
    if int(w4v.kv_fork(cache.pool, cache.refs, cache.table, cache.lengths, i32([0] * (n - 1)), i32(list(range(1, n))))):
        raise RuntimeError("the cache is full")
    cache.prefix.fill_(size)
    tokens, scores, offsets = [ids[0]], [logprobs[0]], torch.arange(n + 1, device="cuda").int()
    for _ in range(count - 1):
        cache.extend(torch.ones_like(cache.lengths))
        logits = target.logits(tokens[-1].long(), cache, offsets)
        _, _, ids, logprobs = w4v.token_logprobs(logits, top=1)
        tokens.append(ids[:, 0])
        scores.append(logprobs[:, 0])
    assert w4v.get_status() == w4v.OK
    tokens, scores = torch.stack(tokens, 1).tolist(), torch.stack(scores, 1).double().tolist()
    ranked = sorted(((sum(s), t, s) for s, t in zip(scores, tokens)), key=lambda r: -r[0])
    for total, t, _ in ranked[:3]:
        print("%8.3f  %s" % (total, t))
    return ranked


if __name__ == "__main__":
    main()
