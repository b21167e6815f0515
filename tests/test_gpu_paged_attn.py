"""paged_attn on the GPU against the oracle (double precision), at the sizes,
masks and layouts where it can go wrong.  Bounds: paged_helpers."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import attention_bounds, cache

pytestmark = pytest.mark.gpu


def run(w, gpu, c, scale=None, window=0, lse=True, invariant=False, ws=None):
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    n, Hq, _ = c["q"].shape
    L = torch.full((n, Hq), 7.0, dtype=torch.float32, device=gpu) if lse else None
    out = torch.full(c["q"].shape, 9.0, dtype=torch.float16, device=gpu)
    o = w.paged_attn(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"], scale=scale, window=window,
                     out=out, lse=L, batch_invariant=invariant, ws=ws)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    return o.cpu().numpy(), L.cpu().numpy() if lse else None


def check(w, gpu, c, scale=None, window=0, invariant=False):
    s = c["q"].shape[2] ** -0.5 if scale is None else scale
    got, lse = run(w, gpu, c, scale, window, invariant=invariant)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], s, window)
    (o, l, _, _), (bo, bl) = ref, attention_bounds(c, ref)
    err = np.abs(got.astype(np.float64) - o)
    assert np.all(err <= bo), (float(np.max(err / bo)), np.unravel_index(np.argmax(err / bo), err.shape))
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(lse), ~fin)
    assert np.all(np.abs(lse[fin] - l[fin]) <= bl[fin]), float(np.max(np.abs(lse[fin] - l[fin]) / bl[fin]))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
def test_lengths_around_tiles_and_pages(w4v_mod, gpu, D, page):
    """One and several new tokens over lengths around every edge of a page and of 128 keys."""
    rng = np.random.default_rng([D, page])
    lengths = [1, 2, 7, 8, 9, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 400]
    check(w4v_mod, gpu, cache(rng, [1 + i % 3 if n > 3 else 1 for i, n in enumerate(lengths)], lengths, 8, 2, D, page))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (10, 2), (21, 3), (8, 1), (66, 1), (128, 1), (40, 2)])
def test_head_groups(w4v_mod, gpu, Hq, Hkv):
    """Groups that divide 128 rows and groups that do not, tiles of one token and of many."""
    rng = np.random.default_rng([Hq, Hkv])
    check(w4v_mod, gpu, cache(rng, [3, 0, 40, 1], [90, 50, 300, 1], Hq, Hkv, 64, 16))
    check(w4v_mod, gpu, cache(rng, [16], [150], Hq, Hkv, 128, 32))


@pytest.mark.parametrize("D,page", [(64, 8), (128, 16), (256, 256)])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000])
def test_windows(w4v_mod, gpu, D, page, window):
    rng = np.random.default_rng([D, window])
    check(w4v_mod, gpu, cache(rng, [1, 30, 150], [300, 290, 420], 4, 2, D, page), window=window)


@pytest.mark.parametrize("stale", [np.nan, np.inf, -np.inf, 65504.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_lies_past_a_sequence_is_never_used(w4v_mod, gpu, stale, D):
    rng = np.random.default_rng(5)
    check(w4v_mod, gpu, cache(rng, [1, 5, 0, 17, 1], [3, 130, 40, 257, 128], 6, 2, D, 32, stale=stale))


def test_rows_that_see_nothing(w4v_mod, gpu):
    """More new tokens than cached ones: the first rows sit before position 0; length 0: all of them."""
    rng = np.random.default_rng(6)
    c = cache(rng, [4, 3, 200, 2], [10, 3, 200, 4], 4, 2, 128, 16)
    c["lengths"] = np.array([2, 0, 130, -5], np.int32)
    got, lse = run(w4v_mod, gpu, c)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], [2, 0, 130, 0], c["offsets"], 128 ** -0.5)
    o, l = ref[:2]
    assert np.all(got[~np.isfinite(l)] == 0) and np.array_equal(np.isneginf(lse), ~np.isfinite(l))
    assert np.all(np.abs(got - o) <= attention_bounds(c, ref)[0])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_contexts_split_over_the_gpu(w4v_mod, gpu, D):
    rng = np.random.default_rng(7)
    check(w4v_mod, gpu, cache(rng, [16], [20011], 4, 1, D, 16))
    check(w4v_mod, gpu, cache(rng, [1, 21, 1], [9000, 5003, 17], 4, 2, D, 64))


def test_a_chunk_of_a_prompt(w4v_mod, gpu):
    rng = np.random.default_rng(8)
    check(w4v_mod, gpu, cache(rng, [700, 129], [1500, 129], 3, 1, 128, 16))
    check(w4v_mod, gpu, cache(rng, [300], [1000], 8, 2, 256, 64))
    check(w4v_mod, gpu, cache(rng, [520], [520], 2, 2, 64, 8))


@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_scores_from_equal_to_one_hot(w4v_mod, gpu, spread):
    """Rising scores force the running maximum up again and again; equal ones never."""
    rng = np.random.default_rng(9)
    c = cache(rng, [3], [1300], 2, 1, 64, 16)
    c["q"][:] = 0
    c["q"][:, :, 0] = 8.0
    ramp = (np.arange(c["table"].shape[1] * 16) / 1300.0 * spread).astype(np.float16)
    for p in range(-(-1300 // 16)):
        c["k"][c["table"][0, p], 0, :, 0] = ramp[16 * p:16 * p + 16]
    check(w4v_mod, gpu, c, scale=0.25)


def test_many_sequences(w4v_mod, gpu):
    rng = np.random.default_rng(10)
    n = rng.integers(0, 4, 700)
    check(w4v_mod, gpu, cache(rng, n, n + rng.integers(0, 40, 700), 2, 1, 64, 8))


def test_strided_rows_and_another_stream(w4v_mod, gpu):
    """q as a slice of a wider projection's rows, and a call on a stream of its own."""
    rng = np.random.default_rng(11)
    c = cache(rng, [9, 20], [100, 333], 4, 2, 128, 16)
    want, _ = run(w4v_mod, gpu, c)
    wide = torch.full((29, 6, 128), float("nan"), dtype=torch.float16, device=gpu)
    wide[:, 1:5] = to_dev(c["q"], gpu)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w4v_mod.paged_attn(wide[:, 1:5], d["k"], d["v"], d["table"], d["lengths"], d["offsets"])
    s.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_results_at_16_byte_addresses(w4v_mod, gpu, D):
    """out and the workspace at addresses that are multiples of 16 bytes and not of 32."""
    rng = np.random.default_rng([11, D])
    c = cache(rng, [9, 200], [100, 5000], 4, 2, D, 16)
    want, _ = run(w4v_mod, gpu, c)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    size = c["q"].size
    out = torch.zeros(size + 16, dtype=torch.float16, device=gpu)[8:8 + size].view(c["q"].shape)
    nbytes = w4v_mod.paged_attn_workspace_bytes(209, 2, 4, 2, D, d["table"].shape[1] * 16)
    ws = torch.zeros(nbytes + 16, dtype=torch.uint8, device=gpu)[16:]
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    w4v_mod.paged_attn(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"], out=out, ws=ws)
    assert np.array_equal(out.cpu().numpy(), want)


def test_repeatable_and_graph_replay(w4v_mod, gpu):
    """The same bits on every call with one workspace; a captured call follows lengths that change."""
    rng = np.random.default_rng(12)
    c = cache(rng, [16, 16], [3000, 1777], 8, 2, 128, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    w = w4v_mod
    ws = w.workspace(w.paged_attn_workspace_bytes(32, 2, 8, 2, 128, d["table"].shape[1] * 16))
    out = torch.empty_like(d["q"])
    call = lambda: w.paged_attn(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"], out=out, ws=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    first = out.clone()
    for _ in range(3):
        out.fill_(3.0)
        call()
        assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["lengths"].copy_(torch.tensor([1000, 40], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], [1000, 40], c["offsets"], 128 ** -0.5)
    assert np.all(np.abs(got - ref[0]) <= attention_bounds(c, ref)[0])


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (256, 0), (128, 300)])
def test_batch_invariance(w4v_mod, gpu, D, window):
    """Verified positions equal the one-token steps they stand for, bit for bit, alone or in a batch."""
    rng = np.random.default_rng(13)
    T, lens = 16, [2100, 530, 16, 1029]
    c = cache(rng, [T] * 4, lens, 10, 2, D, 16)
    check(w4v_mod, gpu, c, window=window, invariant=True)
    got, lse = run(w4v_mod, gpu, c, window=window, invariant=True)
    for b in range(4):
        for t in (0, 1, 7, T - 1):
            one = dict(c, q=c["q"][b * T + t:b * T + t + 1], table=c["table"][b:b + 1],
                       lengths=np.array([lens[b] - T + t + 1], np.int32), offsets=np.array([0, 1], np.int32))
            o1, l1 = run(w4v_mod, gpu, one, window=window, invariant=True)
            assert np.array_equal(o1[0], got[b * T + t]) and np.array_equal(l1[0], lse[b * T + t])


def test_ids_outside_the_cache_read_as_zeros(w4v_mod, gpu):
    rng = np.random.default_rng(14)
    c = cache(rng, [2], [200], 2, 1, 64, 16)
    bad = dict(c, table=c["table"].copy())
    bad["table"][0, 3], bad["table"][0, 5] = -7, c["k"].shape[0] + 2
    zero = dict(c, k=c["k"].copy(), v=c["v"].copy())
    for i in (3, 5):
        zero["k"][c["table"][0, i]] = 0
        zero["v"][c["table"][0, i]] = 0
    a, _ = run(w4v_mod, gpu, bad)
    b, _ = run(w4v_mod, gpu, zero)
    assert np.array_equal(a, b)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_token_that_is_not_finite_touches_only_rows_that_see_it(w4v_mod, gpu, value, D):
    """A drafted token whose key or value overflowed: earlier positions are as without it, later ones carry it."""
    rng = np.random.default_rng(15)
    c = cache(rng, [8, 3], [140, 60], 4, 2, D, 16)
    clean, _ = run(w4v_mod, gpu, c)
    for name in ("v", "k"):
        bad = dict(c, **{name: c[name].copy()})
        p = 136                                                     # row 4 of the first sequence's eight
        bad[name][c["table"][0, p // 16], 1, p % 16, 3] = value
        got, _ = run(w4v_mod, gpu, bad)
        assert np.array_equal(got[:4], clean[:4]) and np.array_equal(got[8:], clean[8:])
        assert np.array_equal(got[4:8, :2], clean[4:8, :2])         # the other key/value head
        if name == "v":
            assert not np.isfinite(got[4:8, 2:, 3]).any()
            rest = np.arange(D) != 3
            assert np.array_equal(got[4:8, 2:][..., rest], clean[4:8, 2:][..., rest])


@pytest.mark.parametrize("invariant", [True, False])
def test_offsets_that_count_rows_again_and_again(w4v_mod, gpu, invariant):
    """Offsets that go up and down ask for more than the workspace (batch-invariant) or 32 bits of work hold:
    nothing is written, neither results nor past the workspace, the status says so, and the next call is as ever."""
    w, rng = w4v_mod, np.random.default_rng(16)
    n, Hq, Hkv, page, length = (3200, 16, 4, 16, 3200) if invariant else (32768, 128, 1, 256, 1 << 21)
    width = length // page
    i32 = lambda a: to_dev(np.asarray(a, np.int32), gpu)  # noqa: E731
    lengths, offsets = i32([length] * 9), i32([0, n] * 5)
    table = torch.full((9, width), -1, dtype=torch.int32, device=gpu)
    k = torch.zeros((4, Hkv, page, 64), dtype=torch.float16, device=gpu)
    q = torch.zeros((n, Hq, 64), dtype=torch.float16, device=gpu)
    out = torch.full_like(q, 9.0)
    nbytes = w.paged_attn_workspace_bytes(n, 9, Hq, Hkv, 64, length, invariant)
    around = torch.full((nbytes + (1 << 20),), 0x5A, dtype=torch.uint8, device=gpu)
    w.paged_attn(q, k, k, table, lengths, offsets, out=out, ws=around[:nbytes], batch_invariant=invariant)
    assert w.get_status() == w.ERR_SHAPE and w.get_status() == w.OK
    assert torch.all(out == 9.0) and torch.all(around[nbytes:] == 0x5A)
    if invariant:                                      # ascending offsets that need every row tile there is
        c = cache(rng, [1] * 8 + [25], [3190] * 8 + [25], Hq, Hkv, 64, page)
        ws = around[:w.paged_attn_workspace_bytes(33, 9, Hq, Hkv, 64, c["table"].shape[1] * page, True)]
        check(w, gpu, c, invariant=True)
        want, got = run(w, gpu, c, invariant=True), run(w, gpu, c, invariant=True, ws=ws.zero_())
        assert np.array_equal(want[0], got[0])


def same_as_alone(w, gpu, c, rows, window=0, **kw):
    """Rows (sequence, index among its new tokens) of a batch-invariant call, bit for bit as one-token calls."""
    got, lse = run(w, gpu, c, window=window, invariant=True, **kw)
    for b, i in rows:
        t, n = c["offsets"][b] + i, c["offsets"][b + 1] - c["offsets"][b]
        one = dict(c, q=c["q"][t:t + 1], table=c["table"][b:b + 1], offsets=np.array([0, 1], np.int32),
                   lengths=np.array([c["lengths"][b] - n + i + 1], np.int32))
        o1, l1 = run(w, gpu, one, window=window, invariant=True, **kw)
        assert np.array_equal(o1[0], got[t]) and np.array_equal(l1[0], lse[t]), (b, i)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_batch_invariance_where_a_key_tile_ends_inside_a_part(w4v_mod, gpu, D):
    """Rows whose last key tile is not the last one of their part, because later tokens of the block see more:
    which group of warps joins the two groups' sums then differs from the one-token call."""
    rng = np.random.default_rng(17)
    c = cache(rng, [16, 16, 16], [650, 901, 135], 10, 2, D, 16)
    same_as_alone(w4v_mod, gpu, c, [(b, i) for b in range(3) for i in range(16)])
    # Sums of equal size: 128 keys from 512 on, then one that raises the maximum by 6.5 to 7.2 powers of two,
    # so that whether their joining rounds once or twice shows (in a fifth of the sums).
    c = cache(rng, [128], [773], 8, 8, D, 16)
    c["q"][:] = 0
    c["q"][:, :, 0] = 8 * rng.uniform(0.95, 1.05, (128, 8))
    level = np.full(c["table"].shape[1] * 16, -40.0)
    level[512:640], level[517], level[640] = rng.uniform(-2, 0, 128), 0.0, 4.75
    for p in range(-(-773 // 16)):
        c["k"][c["table"][0, p], :, :, 0] = level[16 * p:16 * p + 16]
    same_as_alone(w4v_mod, gpu, c, [(0, i) for i in range(128)], scale=0.125)


@pytest.mark.parametrize("invariant", [False, True])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_value_that_is_not_finite_shows_whatever_its_weight(w4v_mod, gpu, value, D, invariant):
    """An early token's value that overflowed, in a context cut into parts whose weights run over 290 powers of
    two: rows that see the token are not finite there, as where the context is one part."""
    rng = np.random.default_rng(19)
    for length in (300, 5000):
        c = cache(rng, [3], [length], 2, 1, D, 16)
        c["q"][:] = 0
        c["q"][:, :, 0] = 8.0
        ramp = (np.arange(c["table"].shape[1] * 16) / length * 100.0).astype(np.float16)
        for p in range(-(-length // 16)):
            c["k"][c["table"][0, p], 0, :, 0] = ramp[16 * p:16 * p + 16]
        clean, _ = run(w4v_mod, gpu, c, scale=0.25, invariant=invariant)
        bad = dict(c, v=c["v"].copy())
        bad["v"][c["table"][0, 0], 0, 5, 3] = value
        got, lse = run(w4v_mod, gpu, bad, scale=0.25, invariant=invariant)
        rest = np.arange(D) != 3
        assert not np.isfinite(got[..., 3]).any() and np.isfinite(lse).all()
        assert np.array_equal(got[..., rest], clean[..., rest])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [-20.0, -22.5, -30.0, -32.0, -32.875])
def test_small_weights(w4v_mod, gpu, D, power):
    """A weight 2^power of the largest is off by at most 2^-11 of itself or 2^-33 of the largest, and not lost
    above that.  Its value is 2^15 and all others are 0, so the result is that weight.  (The power itself is a
    score in fp32, good to 2^-18; the result is rounded to fp16, of 2^-24 at the least.)"""
    rng = np.random.default_rng(20)
    for first, small in ((0, 77), (77, 0), (3, 200)):              # in one key tile, in either order, and in two
        c = cache(rng, [1], [260], 2, 1, D, 16)
        c["q"][:], c["k"][:], c["v"][:] = 0, 0, 0
        c["q"][:, :, 0] = 1.0
        at = lambda a, j: a[c["table"][0, j // 16], 0, j % 16]  # noqa: E731
        c["k"][:, :, :, 0] = -200.0
        at(c["k"], first)[0], at(c["k"], small)[0], at(c["v"], small)[:] = 0.0, power, 2.0 ** 15
        got, _ = run(w4v_mod, gpu, c, scale=float(np.log(2.0)))
        want = 2.0 ** (power + 15)
        tol = max(2.0 ** -11 * want, 2.0 ** (15 - 33)) + 2.0 ** -17 * want + max(2.0 ** -11 * want, 2.0 ** -25)
        assert np.all(np.abs(got.astype(np.float64) - want) <= tol) and np.all(got > 0)


@pytest.mark.parametrize("invariant", [False, True])
def test_rows_of_no_sequence_are_left_alone(w4v_mod, gpu, invariant):
    """Rows before the first offset and from the last one on (a batch padded to a fixed size)."""
    rng = np.random.default_rng(21)
    c = cache(rng, [3, 0, 16], [500, 40, 2000], 4, 2, 64, 16)
    want, lse = run(w4v_mod, gpu, c, invariant=invariant)
    pad = dict(c, offsets=c["offsets"] + 5, q=np.concatenate([c["q"][:5], c["q"], np.full((9, 4, 64), np.nan, np.float16)]))
    got, l = run(w4v_mod, gpu, pad, invariant=invariant)
    assert np.all(got[:5] == 9) and np.all(got[24:] == 9) and np.all(l[:5] == 7) and np.all(l[24:] == 7)
    assert np.array_equal(l[5:24], lse) and np.array_equal(got[5:24], want)      # the same work, split in the same way


@pytest.mark.parametrize("D", [64, 128, 256])
def test_batch_invariance_over_tables_of_one_class(w4v_mod, gpu, D):
    """A table trimmed to the batch's longest context and one with room for more give the same bits while both
    hold up to 16,384 tokens, or lie between the same powers of two; and so do pages of another size."""
    rng = np.random.default_rng(18)
    c = cache(rng, [4, 1, 7], [2100, 530, 1029], 6, 2, D, 16)

    def at(width):
        wide = np.full((3, width), -1, np.int32)
        wide[:, :132] = c["table"][:, :132]
        return run(w4v_mod, gpu, dict(c, table=wide), invariant=True)
    for widths in ((132, 500, 1024), (1025, 1500, 2048), (40000, 65536)):
        results = [at(width) for width in widths]
        for got in results[1:]:
            assert np.array_equal(got[0], results[0][0]) and np.array_equal(got[1], results[0][1]), widths
    c = cache(rng, [5], [34900], 2, 1, D, 64)
    check(w4v_mod, gpu, c, invariant=True)
    same_as_alone(w4v_mod, gpu, c, [(0, 0), (0, 3)])
    same_as_alone(w4v_mod, gpu, c, [(0, 2)], window=19000)
    got = run(w4v_mod, gpu, c, invariant=True)
    k, v = (x.reshape(x.shape[0], 1, 8, 8, D).swapaxes(1, 2).reshape(-1, 1, 8, D) for x in (c["k"], c["v"]))
    ids = np.where(c["table"][:, :, None] < 0, -1, c["table"][:, :, None] * 8 + np.arange(8, dtype=np.int32))
    eight = run(w4v_mod, gpu, dict(c, k=k, v=v, table=ids.reshape(1, -1)), invariant=True)
    assert np.array_equal(got[0], eight[0]) and np.array_equal(got[1], eight[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_contexts_to_the_weights_rounding(w4v_mod, gpu, D):
    """The bound of attention_bounds charges every key a step of one running sum.  Dealt out over at least 148
    CTAs, 20,011 keys are at most two tiles (256 keys) to a part and 157 parts to join: with these steps instead, what
    is left is little more than the weights' and the result's roundings."""
    rng = np.random.default_rng([22, D])
    c = cache(rng, [2], [20011], 3, 1, D, 16)
    got, _ = run(w4v_mod, gpu, c)
    o, _, mag, absdot = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], D ** -0.5)
    eps = (D + 8) * 2.0 ** -23 * absdot + 2.0 ** -20
    rel = 2.0 ** -11 + 2 * eps + 2 * (256 + 157) * 2.0 ** -23
    assert np.all(np.abs(got - o) <= 2.0 ** -11 * np.abs(o) + rel[..., None] * (1 + 2.0 ** -10) * mag + 2.0 ** -24)
