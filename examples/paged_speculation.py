"""Greedy speculative decoding over a paged key/value cache, two sequences that share a prompt.

A toy target (two layers of softmax attention and W4A16 MLP, int8 lm_head, random weights) runs as a
server would run it: the prompt goes through in chunks, the second sequence is forked from the first
(full pages shared), every step drafts by prompt lookup, verifies K + 1 positions of both sequences in
one pass and gives back the pages of rejected drafts, and the cache is compacted on the way.  All of
it stays on the GPU but the loop itself.  With batch invariance in the projections, the lm_head and the
attention, the tokens are exactly those of decoding one token at a time, which is what main() checks.

    python examples/paged_speculation.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verify_w4a16_gb300 import inputs, w4v  # noqa: E402

H, V, LAYERS, Q_HEADS, KV_HEADS, D, PAGE = 256, 1024, 2, 8, 2, 64, 16


class Target:
    """Weights on the device; positions are scaled for a context longer than the base's."""

    def __init__(self, seed: int, device="cuda"):
        E, mlp, W8, s8 = inputs.toy_model_arrays(seed, V=V, H=H, layers=LAYERS)
        dev = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
        lin = lambda n, k, tag, i: (dev(w4v.pack_int4(inputs.w4_codes(seed, n, k, tag, i))),  # noqa: E731
                                    dev(inputs.w4_scales(seed, n, k, tag, i)), n)
        self.E, self.W8, self.s8 = dev(E), dev(W8), dev(s8)
        self.qkv = [lin((Q_HEADS + 2 * KV_HEADS) * D, H, "qkv", i) for i in range(LAYERS)]
        self.out = [lin(H, Q_HEADS * D, "attn-out", i) for i in range(LAYERS)]
        self.mlp = [((dev(w4v.pack_int4(a)), dev(b), a.shape[0]), (dev(w4v.pack_int4(c)), dev(d), c.shape[0]))
                    for a, b, c, d in mlp]
        self.rope = w4v.Rope(D, scaling=("yarn", 4.0, 64.0), device=device)

    def project(self, x, w):
        packed, scales, n = w
        return w4v.w4a16_gemm(x, packed, scales, n, batch_invariant=True)

    def hidden(self, tokens, cache, offsets):
        """Last hidden rows (fp16) of new tokens that the cache has pages for already."""
        h = self.E[tokens].double()
        for i in range(LAYERS):
            k_cache, v_cache = cache.pool[2 * i], cache.pool[2 * i + 1]
            rows = self.project(rms(h), self.qkv[i]).unflatten(1, (-1, D))
            q, k, v = rows.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q = w4v.rope_append(q, k, v, k_cache, v_cache, cache.table, cache.lengths, offsets, self.rope)
            o = w4v.paged_attn(q, k_cache, v_cache, cache.table, cache.lengths, offsets, batch_invariant=True)
            h = h + self.project(o.flatten(1), self.out[i]).double()
            gate, up = self.project(rms(h), self.mlp[i][0]).double().chunk(2, 1)
            h = h + self.project((torch.nn.functional.silu(gate) * up).half(), self.mlp[i][1]).double()
        return rms(h)


def rms(x):
    return (x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()).half()


class Cache:
    """Pages of all layers ([2 layers][pages][KV_HEADS][PAGE][D]: plane 2i is layer i's k, 2i + 1 its v)."""

    def __init__(self, sequences: int, pages: int, device="cuda"):
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.pool = torch.zeros((2 * LAYERS, pages, KV_HEADS, PAGE, D), dtype=torch.float16, device=device)
        self.refs, self.table, self.lengths = i32(pages), i32(sequences, pages) - 1, i32(sequences)
        self.short, self.ws = i32(1), w4v.workspace(w4v.kv_workspace_bytes(pages, sequences), device)

    def extend(self, new):
        w4v.kv_extend(self.pool, self.refs, self.table, self.lengths, self.lengths + new, self.short, self.ws)
        if int(self.short):
            raise RuntimeError("the cache is short of %d pages" % int(self.short))

    def truncate(self, lengths):
        w4v.kv_truncate(self.refs, self.table, self.lengths, lengths, PAGE)

    def fork(self, parent: int, child: int):
        at = lambda x: torch.tensor([x], dtype=torch.int32, device=self.refs.device)  # noqa: E731
        w4v.kv_fork(self.pool, self.refs, self.table, self.lengths, at(parent), at(child), self.short, self.ws)
        assert int(self.short) == 0

    def compact(self):
        w4v.kv_compact(self.pool, self.refs, self.table, self.lengths, ws=self.ws)


def offsets_of(counts):
    c = torch.tensor([0, *counts], dtype=torch.int32, device="cuda")
    return c.cumsum(0, dtype=torch.int32), c[1:]


def prefill(target, cache, prompt, chunk=48):
    """All of the prompt but its last token, into sequence 0, in chunks."""
    for at in range(0, len(prompt) - 1, chunk):
        piece = prompt[at:min(at + chunk, len(prompt) - 1)]
        offsets, new = offsets_of([len(piece)] + [0] * (cache.table.shape[0] - 1))
        cache.extend(new)
        target.hidden(torch.tensor(piece, device="cuda"), cache, offsets)


def decode(target, prompt, firsts, count, K):
    """`count` tokens after prompt + [first] for each of `firsts`, K drafted tokens a step (K = 0: plain
    greedy decoding).  Returns (tokens of every sequence, steps)."""
    B = len(firsts)
    cache = Cache(B, pages=64)
    prefill(target, cache, prompt + [0])
    for b in range(1, B):
        cache.fork(0, b)
    context = [prompt + [f] for f in firsts]
    ld, steps = len(prompt) + count + 2 * K + 8, 0
    while min(len(c) for c in context) < len(prompt) + 1 + count:
        lengths = torch.tensor([len(c) for c in context], dtype=torch.int32, device="cuda")
        rows = torch.zeros((B, ld), dtype=torch.int32)
        for b, c in enumerate(context):
            rows[b, :len(c)] = torch.tensor(c, dtype=torch.int32)
        rows = rows.cuda()
        drafts = w4v.ngram_draft(rows, lengths, 1, 3, K)[0] if K else torch.zeros((B, 0), dtype=torch.int32, device="cuda")
        last = rows.gather(1, lengths[:, None].long() - 1)
        block = torch.cat([last, drafts.clamp(min=0)], 1)              # a sentinel is fed as token 0
        offsets, new = offsets_of([K + 1] * B)
        cache.extend(new)
        hidden = target.hidden(block.flatten().long(), cache, offsets)
        _, accepted, emitted = w4v.w8_lmhead_argmax_accept(hidden, target.W8, target.s8, drafts, batch_invariant=True)
        cache.truncate(cache.lengths - K + accepted)                   # keeps the last token and the accepted drafts
        if steps % 3 == 1:
            cache.compact()
        for b, (n, toks) in enumerate(zip(accepted.tolist(), emitted.tolist())):
            context[b] += toks[:n + 1]
        steps += 1
    assert w4v.get_status() == w4v.OK
    return [c[len(prompt) + 1:len(prompt) + 1 + count] for c in context], steps


def main(seed: int = 7, count: int = 40, K: int = 15):
    w4v.init()
    target = Target(seed)
    prompt = [int(t) for t in inputs.random_tokens(seed, 25, V)] * 4   # repeats: something to look up
    firsts = [prompt[0], 3]
    plain = [decode(target, prompt, [f], count, 0)[0][0] for f in firsts]
    tokens, steps = decode(target, prompt, firsts, count, K)
    print("%d tokens of each of %d sequences in %d verify steps; as decoded one by one: %s"
          % (count, len(firsts), steps, tokens == plain))
    return tokens, plain, steps


if __name__ == "__main__":
    got, want, _ = main()
    sys.exit(got != want)
