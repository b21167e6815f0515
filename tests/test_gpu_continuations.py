"""What continuations of one prompt run together: heads normed, rotated and appended, pages forked, extended,
rolled back and moved, attention over the shared prefix and over a window with first tokens, scores of the
lm_head's tokens.  Every step is held to the oracle on what the step before has left on the GPU."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged, scores
from paged_helpers import attention_bounds, cache
from test_gpu_streams import MODES, on_side_stream

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, V, H = 8, 2, 128, 16, 2048, 256


class Step:
    """One layer's tensors of a fixed size, so that a step can be captured."""

    def __init__(self, w, gpu, C, T, pages):
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=gpu)  # noqa: E731
        r = np.random.default_rng(1)
        self.w, self.C, self.n = w, C, C * T
        self.pool = torch.zeros((2, pages, HKV, PAGE, D), dtype=torch.float16, device=gpu)
        self.refs, self.table, self.lengths, self.short = i32(pages), i32(C, pages) - 1, i32(C), i32(1)
        self.offsets = (torch.arange(C + 1, device=gpu) * T).int()
        self.groups, self.prefix = torch.tensor([0, C], dtype=torch.int32, device=gpu), i32(1)
        self.rows = torch.empty((self.n, (HQ + 2 * HKV) * D), dtype=torch.float16, device=gpu)
        self.q = torch.empty((self.n, HQ, D), dtype=torch.float16, device=gpu)
        self.full, self.near = torch.empty_like(self.q), torch.empty_like(self.q)
        self.lse = torch.empty((self.n, HQ), device=gpu)
        self.ws = w.workspace(max(w.paged_attn_shared_workspace_bytes(self.n, C, 1, HQ, HKV, D),
                                  w.paged_attn_workspace_bytes(self.n, C, HQ, HKV, D, pages * PAGE)))
        self.kv_ws = w.workspace(w.kv_workspace_bytes(pages, C))
        half = lambda *s: to_dev((r.standard_normal(s) * 0.3).astype(np.float16), gpu)  # noqa: E731
        self.rope, self.norm = w.Rope(64), w.HeadNorm(half(D), half(D), zero_centred=True)
        self.W8 = to_dev(r.integers(-127, 128, (V, H)).astype(np.int8), gpu)
        self.s8 = to_dev((r.random(V) * 0.002 + 0.001).astype(np.float16), gpu)
        self.x = torch.empty((self.n, H), dtype=torch.float16, device=gpu)
        self.logits, self.best = torch.empty((self.n, V), device=gpu), i32(self.n)
        self.lm_ws = w.workspace(w.w8_lmhead_argmax_workspace_bytes(self.n, V))
        self.out = (torch.empty(self.n, device=gpu), torch.empty(self.n, device=gpu),
                    torch.empty((self.n, 5), dtype=torch.int32, device=gpu), torch.empty((self.n, 5), device=gpu))

    def cache(self):
        return self.pool[0], self.pool[1], self.table, self.lengths, self.offsets

    def extend(self, new):
        self.w.kv_extend(self.pool, self.refs, self.table, self.lengths, self.lengths + new, self.short, self.kv_ws)
        assert int(self.short) == 0

    def run(self, stream=None):
        w = self.w
        q, k, v = self.rows.unflatten(1, (-1, D)).split([HQ, HKV, HKV], 1)
        w.norm_rope_append(q, k, v, *self.cache(), self.rope, self.norm, q_out=self.q, stream=stream)
        w.paged_attn_shared(self.q, *self.cache(), self.groups, self.prefix, out=self.full, lse=self.lse, ws=self.ws,
                            stream=stream)
        w.paged_attn(self.q, *self.cache(), window=50, sinks=20, out=self.near, ws=self.ws, stream=stream)
        w.w8_lmhead_argmax(self.x, self.W8, self.s8, out=self.best, logits=self.logits, ws=self.lm_ws, stream=stream)
        w.token_logprobs(self.logits, self.best, top=5, temperature=0.7, out=self.out, stream=stream)

    def check(self, before):
        """before: the pool as the step found it."""
        host = lambda t: t.cpu().numpy()  # noqa: E731
        table, lengths, offsets = host(self.table), host(self.lengths), host(self.offsets)
        rows = host(self.rows).reshape(self.n, -1, D)
        f, mul = paged.frequencies(64)
        places = paged.token_places(lengths, offsets)
        pos = np.array([p for _, p in places])
        wq, wk = (host(x).astype(np.float64) for x in (self.norm.q_weight, self.norm.k_weight))
        pool = before.copy()
        for x, want, got in ((rows[:, :HQ], wq, host(self.q)), (rows[:, HQ:HQ + HKV], wk, None)):
            n = paged.head_norm(x, want, 1e-6, 1.0)
            y = paged.rotate(n, pos, f, mul, False)
            tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -15 * np.abs(n).max(-1, keepdims=True) + 2.0 ** -25   # see test_gpu_norm_rope
            if got is None:
                got = np.stack([host(self.pool)[0, table[b, p // PAGE], :, p % PAGE] for b, p in places])
                for t, (b, p) in enumerate(places):
                    pool[0, table[b, p // PAGE], :, p % PAGE] = got[t]
                    pool[1, table[b, p // PAGE], :, p % PAGE] = rows[t, HQ + HKV:]
            assert np.all(np.abs(got - y) <= tol)
        assert np.array_equal(host(self.pool), pool)                     # nothing else was written
        c = dict(q=host(self.q), k=pool[0], v=pool[1], table=table, lengths=lengths, offsets=offsets)
        for got, window, sinks in ((self.full, 0, 0), (self.near, 50, 20)):
            ref = paged.attention(c["q"], c["k"], c["v"], table, lengths, offsets, D ** -0.5, window, sinks)
            bo, bl = attention_bounds(c, ref)
            assert np.all(np.abs(host(got) - ref[0]) <= bo)
            if window == 0:
                assert np.all(np.abs(host(self.lse) - ref[1]) <= bl)
        logits, best = host(self.logits), host(self.best)
        lp, entropy, ids, tops = (host(t) for t in self.out)
        for r in range(self.n):
            want = scores.row(logits[r], [best[r]], 5, 0.7)
            per, eh = scores.bounds(logits[r], 0.7)
            high = logits[r].max()
            near = lambda a, b, x: abs(a - b) <= per + 2.0 ** -21 * abs(float(x) - high) / 0.7  # noqa: E731
            assert near(lp[r], want[0][0], logits[r, best[r]]) and abs(entropy[r] - want[1]) <= eh
            assert ids[r].tolist() == want[2] and ids[r, 0] == best[r]
            assert all(near(a, b, logits[r, i]) for a, b, i in zip(tops[r], want[3], ids[r]))


@pytest.mark.parametrize("captured", [False, True])
def test_continuations_of_one_prompt(w4v_mod, gpu, captured):
    w, rng = w4v_mod, np.random.default_rng(2)
    C, T, prompt, pages = 6, 3, 150, 80
    s = Step(w, gpu, C, T, pages)
    i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).to(gpu)  # noqa: E731
    half = lambda *shape: to_dev(rng.standard_normal(shape).astype(np.float16), gpu)  # noqa: E731
    # the prompt into sequence 0, which the others are forked from
    w.kv_extend(s.pool, s.refs, s.table, s.lengths, i32([prompt] + [0] * (C - 1)), s.short, s.kv_ws)
    q, k, v = half(prompt, HQ, D), half(prompt, HKV, D), half(prompt, HKV, D)
    w.norm_rope_append(q, k, v, s.pool[0], s.pool[1], s.table, s.lengths, i32([0] + [prompt] * C), s.rope, s.norm)
    w.kv_fork(s.pool, s.refs, s.table, s.lengths, i32([0] * (C - 1)), i32(range(1, C)), s.short, s.kv_ws)
    assert int(s.short) == 0 and s.lengths.tolist() == [prompt] * C
    assert torch.equal(s.table[0, :prompt // PAGE], s.table[5, :prompt // PAGE])
    s.prefix.fill_(prompt)
    graph, stream = None, torch.cuda.Stream()
    for step in range(5):
        s.extend(torch.full((C,), T, dtype=torch.int32, device=gpu))
        s.rows.copy_(half(*s.rows.shape))
        s.x.copy_(half(*s.x.shape))
        before = s.pool.cpu().numpy()
        if not captured:
            s.run()
        elif graph is None:
            s.run()                                       # (first calls set kernels up; the step itself is written again)
            s.pool.copy_(to_dev(before, gpu))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.run()
            graph.replay()
        else:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        assert w.get_status() == w.OK
        s.check(before)
        kept = s.lengths - i32(rng.integers(0, T + 1, C))                # some of the step's tokens are rejected
        w.kv_truncate(s.refs, s.table, s.lengths, kept, PAGE)
        if step == 1:                                                    # two end; sequence 0, the prefix's holder, goes on
            w.kv_truncate(s.refs, s.table, s.lengths, i32([9999, 0, 9999, 9999, 0, 9999]), PAGE)
        if step == 2:
            w.kv_compact(s.pool, s.refs, s.table, s.lengths, ws=s.kv_ws)
        if step == 3:                                                    # it ends too: the group begins behind it
            w.kv_truncate(s.refs, s.table, s.lengths, i32([0] + [9999] * (C - 1)), PAGE)
            s.groups.copy_(i32([2, C]))


@MODES
def test_workspaces_and_results_on_a_stream_of_their_own(w4v_mod, gpu, raw, late):
    """What the binding allocates for these calls belongs to their stream, as for the others."""
    w, rng = w4v_mod, np.random.default_rng(3)
    c = cache(rng, [16, 1], [3000, 500], 4, 2, 64, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    at = [d[x] for x in ("k", "v", "table", "lengths", "offsets")]
    groups, prefix = torch.tensor([0, 1, 2], dtype=torch.int32, device=gpu), torch.tensor([2000, 400], dtype=torch.int32, device=gpu)
    kn, vn = (d[x][:17, :, 0].contiguous() for x in "kv")
    rope, norm = w.Rope(64), w.HeadNorm()
    x, t = torch.randn((17, 30000), device=gpu), torch.zeros(17, dtype=torch.int32, device=gpu)
    nq = c["q"].nbytes
    for call, sizes in ((lambda s: [w.norm_rope_append(d["q"], kn, vn, *at, rope, norm, stream=s)], (nq,)),
                        (lambda s: [w.paged_attn(d["q"], *at, window=700, sinks=9, stream=s)],
                         (w.paged_attn_workspace_bytes(17, 2, 4, 2, 64, d["table"].shape[1] * 16), nq)),
                        (lambda s: [w.paged_attn_shared(d["q"], *at, groups, prefix, stream=s)],
                         (w.paged_attn_shared_workspace_bytes(17, 2, 2, 4, 2, 64), nq)),
                        (lambda s: list(w.token_logprobs(x, t, top=5, stream=s)), (4 * 17, 4 * 17 * 5))):
        want = [y.clone() for y in call(None)]
        torch.cuda.synchronize()
        got = on_side_stream(call, raw, late, sizes)
        assert w.get_status() == w.OK
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_two_calls_at_once(w4v_mod, gpu):
    """The same operators on two streams, each with a workspace of its own, while the other runs."""
    w, rng = w4v_mod, np.random.default_rng(4)
    c = cache(rng, [16] * 6, [9000, 700, 5000, 40, 3000, 16], 8, 2, 128, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    at = [d[x] for x in ("k", "v", "table", "lengths", "offsets")]
    groups, prefix = (torch.tensor(v, dtype=torch.int32, device=gpu) for v in ([0, 1, 2, 3, 4, 5, 6], [8000, 600, 4000, 0, 2000, 0]))
    x, t = torch.randn((96, 50001), device=gpu), torch.zeros(96, dtype=torch.int32, device=gpu)

    def both():
        return [w.paged_attn_shared(d["q"], *at, groups, prefix), w.paged_attn(d["q"], *at, window=500, sinks=130),
                *w.token_logprobs(x, t, top=20)]
    want = [y.clone() for y in both()]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, got):
            with torch.cuda.stream(s):
                g.append(both())
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    for results in got[0] + got[1]:
        assert all(torch.equal(a, b) for a, b in zip(want, results))


def test_the_example_ranks_its_continuations(w4v_mod, gpu):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "continuations.py")
    spec = importlib.util.spec_from_file_location("continuations", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    ranked = example.main(seed=7, count=12, n=5)
    assert len(ranked) == 5 and all(len(tokens) == 12 for _, tokens, _ in ranked)
    assert [r[0] for r in ranked] == sorted((r[0] for r in ranked), reverse=True)
    for total, tokens, each in ranked:
        assert np.isclose(total, sum(each)) and max(each) <= 0 and len(each) == 12
        assert all(0 <= t < example.V for t in tokens)
    assert len({tokens[0] for _, tokens, _ in ranked}) == 5
