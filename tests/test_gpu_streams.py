"""Calls with `stream=`: what the binding allocates for them belongs to that stream, so nothing of another
stream's work, before or after, meets the call.  The other (current) stream is kept busy meanwhile, and
memory of the sizes in question is handed round on it."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import attention_bounds, cache

pytestmark = pytest.mark.gpu

BUSY = 100_000_000                                     # clock cycles: some 50 ms


def on_side_stream(call, raw, late, sizes=()):
    """call(stream) with the current stream busy before it (late: with the side stream busy instead,
    and blocks of `sizes` bytes filled on the current one while the call is still waiting)."""
    s = torch.cuda.Stream()
    for n in sizes:                                    # what the allocator holds for the current stream is not zero
        torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    if late:
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
    else:
        torch.cuda._sleep(BUSY)
    got = call(s.cuda_stream if raw else s)
    held = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes] if late else []
    s.synchronize()
    first = [x.clone() for x in got]
    torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)
    del held
    return got


MODES = pytest.mark.parametrize("raw,late", [(False, False), (True, False), (False, True), (True, True)])


@MODES
def test_short_and_workspace_of_the_page_calls(w4v_mod, gpu, raw, late):
    w = w4v_mod
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=gpu)  # noqa: E731
    pool = torch.zeros((2, 6, 1, 16, 64), dtype=torch.float16, device=gpu)
    refs, table, lengths = i32(*[0] * 6), torch.full((3, 8), -1, dtype=torch.int32, device=gpu), i32(0, 0, 0)
    sizes = (w.kv_workspace_bytes(6, 3), 4)
    call = lambda f, *a, **kw: on_side_stream(lambda s: [f(pool, refs, table, lengths, *a, stream=s, **kw)], raw, late,  # noqa: E731
                                              sizes)
    want, more = i32(40, 20, 0), i32(40, 20, 32)
    assert int(call(w.kv_extend, want)[0]) == 0 and lengths.tolist() == [40, 20, 0]
    assert int(call(w.kv_extend, more)[0]) == 1 and lengths.tolist() == [40, 20, 0]          # two wanted, one free
    parents, children = i32(0), i32(2)
    assert int(call(w.kv_fork, parents, i32(1))[0]) == -1
    assert int(call(w.kv_fork, parents, children)[0]) == 0 and refs.tolist() == [2, 2, 1, 1, 1, 1]
    w.kv_truncate(refs, table, lengths, i32(0, 20, 0), 16)
    on_side_stream(lambda s: w.kv_compact(pool, refs, table, lengths, stream=s), raw, late, sizes)
    assert refs.tolist() == [1, 1, 0, 0, 0, 0] and sorted(table[1, :2].tolist()) == [0, 1]


@MODES
@pytest.mark.parametrize("invariant", [False, True])
def test_workspace_and_result_of_attention(w4v_mod, gpu, raw, late, invariant):
    w, rng = w4v_mod, np.random.default_rng(1)
    c = cache(rng, [16, 1], [3000, 500], 4, 2, 64, 16)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], 0.125)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    sizes = (w.paged_attn_workspace_bytes(17, 2, 4, 2, 64, d["table"].shape[1] * 16, invariant), c["q"].nbytes)
    got, = on_side_stream(lambda s: [w.paged_attn(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"],
                                                  batch_invariant=invariant, stream=s)], raw, late, sizes)
    assert w.get_status() == w.OK
    assert np.all(np.abs(got.cpu().numpy() - ref[0]) <= attention_bounds(c, ref)[0])
    rope = w.Rope(64)
    kn, vn = (d[x][:17, :, 0].contiguous() for x in "kv")
    append = lambda s: [w.rope_append(d["q"], kn, vn, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope,  # noqa: E731
                                      stream=s)]
    want, = append(None)
    q, = on_side_stream(append, raw, late, (c["q"].nbytes,))
    assert torch.equal(q, want)


@MODES
def test_workspaces_and_results_of_the_verify_step(w4v_mod, gpu, raw, late):
    w, r = w4v_mod, np.random.default_rng(2)
    N, K, M = 512, 1024, 16
    Bq = to_dev(w.pack_int4(r.integers(0, 16, (N, K)).astype(np.uint8)), gpu)
    sc = to_dev((r.random((K // 128, N)) * 0.01).astype(np.float16), gpu)
    X = to_dev(r.standard_normal((M, K)).astype(np.float16), gpu)
    W8 = to_dev(r.integers(-127, 128, (4096, K)).astype(np.int8), gpu)
    s8 = to_dev((r.random(4096) * 0.01).astype(np.float16), gpu)
    draft = to_dev(r.integers(0, 4096, (1, M - 1)).astype(np.int32), gpu)
    ctx, length = to_dev(r.integers(0, 5, (2, 3000)).astype(np.int32), gpu), to_dev(np.array([3000, 77], np.int32), gpu)
    C = torch.empty((M, N), dtype=torch.float16, device=gpu)
    ws = (w.w4a16_workspace_bytes(M, N, K), w.w8_lmhead_argmax_workspace_bytes(M, 4096))

    def grouped(s):
        return w.GroupedGemm([(X, Bq, sc, None, C)], stream=s)(stream=s)
    target = w.w8_lmhead_argmax(X, W8, s8).view(1, M)
    for call, sizes in ((lambda s: [w.w4a16_gemm(X, Bq, sc, N, stream=s)], (ws[0], 2 * M * N)), (grouped, (ws[0],)),
                        (lambda s: [w.w8_lmhead_argmax(X, W8, s8, stream=s)], (ws[1], 4 * M)),
                        (lambda s: w.w8_lmhead_argmax_accept(X, W8, s8, draft, stream=s), (ws[1], 4 * M)),
                        (lambda s: w.spec_accept(target, draft, stream=s), (4 * M, 4)),
                        (lambda s: w.ngram_draft(ctx, length, 1, 3, 15, stream=s), (120, 8, 48))):
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        got = on_side_stream(call, raw, late, sizes)
        assert w.get_status() == w.OK
        for a, b in zip(want, got):
            assert torch.equal(a, b)
