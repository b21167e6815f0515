"""paged_attn with a window and first tokens that stay visible, against the oracle (double precision).
Bounds: paged_helpers."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import attention_bounds, cache

pytestmark = pytest.mark.gpu


def run(w, gpu, c, window, sinks, invariant=False, scale=None):
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    n, Hq, _ = c["q"].shape
    lse = torch.full((n, Hq), 7.0, dtype=torch.float32, device=gpu)
    out = torch.full(c["q"].shape, 9.0, dtype=torch.float16, device=gpu)
    w.paged_attn(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"], scale=scale, window=window, sinks=sinks,
                 out=out, lse=lse, batch_invariant=invariant)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    return out.cpu().numpy(), lse.cpu().numpy()


def check(w, gpu, c, window, sinks, invariant=False, scale=None):
    s = c["q"].shape[2] ** -0.5 if scale is None else scale
    got, lse = run(w, gpu, c, window, sinks, invariant, scale)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], s, window, sinks)
    (o, l, _, _), (bo, bl) = ref, attention_bounds(c, ref)
    err = np.abs(got.astype(np.float64) - o)
    assert np.all(err <= bo), (float(np.max(err / bo)), np.unravel_index(np.argmax(err / bo), err.shape))
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(lse), ~fin)
    assert np.all(np.abs(lse[fin] - l[fin]) <= bl[fin]), float(np.max(np.abs(lse[fin] - l[fin]) / bl[fin]))


@pytest.mark.parametrize("D,page", [(64, 8), (128, 16), (256, 256)])
@pytest.mark.parametrize("window", [1, 2, 100, 129, 1000])
@pytest.mark.parametrize("sinks", [1, 4, 127, 128, 129, 300])
def test_windows_and_first_tokens(w4v_mod, gpu, D, page, window, sinks):
    """First tokens and windows that end around tiles, overlap, and leave gaps of none to several tiles."""
    rng = np.random.default_rng([D, window, sinks])
    check(w4v_mod, gpu, cache(rng, [1, 30, 150, 3], [700, 290, 420, 129], 4, 2, D, page), window, sinks)


@pytest.mark.parametrize("length", [1, 2, 127, 128, 129, 256, 384, 513, 640, 1000])
def test_lengths(w4v_mod, gpu, length):
    """Sequences shorter than the first tokens, shorter than both, and longer."""
    rng = np.random.default_rng(length)
    for T in (1, min(length, 40)):
        check(w4v_mod, gpu, cache(rng, [T, 0, 1], [length, 9, 60], 6, 3, 64, 16), 100, 130)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (21, 3), (128, 1), (40, 2)])
def test_head_groups(w4v_mod, gpu, Hq, Hkv):
    rng = np.random.default_rng([Hq, Hkv])
    check(w4v_mod, gpu, cache(rng, [3, 0, 40, 1], [900, 50, 1300, 1], Hq, Hkv, 64, 16), 200, 33)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_contexts_and_prompts(w4v_mod, gpu, D):
    rng = np.random.default_rng([D, 1])
    check(w4v_mod, gpu, cache(rng, [16, 1], [20011, 9000], 4, 1, D, 16), 3000, 500)
    check(w4v_mod, gpu, cache(rng, [700, 300], [1500, 1100], 3, 1, D, 32), 256, 64)


def test_many_sequences(w4v_mod, gpu):
    rng = np.random.default_rng(10)
    n = rng.integers(0, 4, 500)
    check(w4v_mod, gpu, cache(rng, n, n + rng.integers(0, 400, 500), 2, 1, 64, 8), 40, 9)


@pytest.mark.parametrize("stale", [np.nan, np.inf, 65504.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_no_row_sees_is_never_used(w4v_mod, gpu, stale, D):
    """Past the sequences, and between the first tokens and the window, inside shared tiles too."""
    rng = np.random.default_rng(5)
    window, sinks = 100, 40
    c = cache(rng, [1, 5, 0, 17, 1], [3, 430, 40, 657, 228], 6, 2, D, 32, stale=stale)
    for b, (n, length) in enumerate(zip(np.diff(c["offsets"]), c["lengths"])):
        for j in range(sinks, max(sinks, length - n - window + 1)):
            i = c["table"][b, j // 32]
            c["k"][i, :, j % 32] = c["v"][i, :, j % 32] = stale
    check(w4v_mod, gpu, c, window, sinks)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("D", [64, 256])
def test_a_value_that_is_not_finite_reaches_those_that_see_it(w4v_mod, gpu, value, D):
    """In the first tokens every row from there on sees it; before the last rows' windows, only the first rows;
    among the new tokens, the rows from it on."""
    rng = np.random.default_rng(6)
    T, length, window, sinks = 40, 500, 64, 20
    for j in (7, 19, 20, 470 - window, 465, 490):
        c = cache(rng, [T], [length], 4, 2, D, 16)
        c["v"][c["table"][0, j // 16], :, j % 16, 3] = value
        got, _ = run(w4v_mod, gpu, c, window, sinks)
        pos = np.arange(length - T, length)
        sees = (j <= pos) & ((j > pos - window) | (j < sinks))
        assert np.array_equal(~np.isfinite(got[:, 0, 3].astype(np.float64)), sees), j
        assert np.all(np.isfinite(np.delete(got, 3, axis=2)))


@pytest.mark.parametrize("T,length,sinks", [(64, 70, 50), (64, 64, 64), (130, 400, 390)])
def test_new_tokens_among_the_first_ones(w4v_mod, gpu, T, length, sinks):
    """Rows that stand before the last first token see those up to themselves; a NaN among them reaches later rows only."""
    rng = np.random.default_rng(7)
    c = cache(rng, [T], [length], 4, 2, 64, 16)
    check(w4v_mod, gpu, c, 5, sinks)
    j = length - T + 20
    c["v"][c["table"][0, j // 16], :, j % 16, 0] = np.nan
    got, _ = run(w4v_mod, gpu, c, 5, sinks)
    pos = np.arange(length - T, length)
    assert np.array_equal(np.isnan(got[:, 0, 0]), (j <= pos) & ((j > pos - 5) | (j < sinks)))


def test_rows_that_see_nothing(w4v_mod, gpu):
    rng = np.random.default_rng(8)
    c = cache(rng, [4, 3, 200], [10, 3, 200], 4, 2, 128, 16)
    c["lengths"] = np.array([2, 0, 130], np.int32)
    got, lse = run(w4v_mod, gpu, c, 16, 8)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], 128 ** -0.5, 16, 8)
    o, l = ref[:2]
    assert np.all(got[~np.isfinite(l)] == 0) and np.array_equal(np.isneginf(lse), ~np.isfinite(l))
    assert np.all(np.abs(got - o) <= attention_bounds(c, ref)[0])


def test_degenerate_windows_are_paged_attn(w4v_mod, gpu):
    """No window: everything is visible; no first tokens: the window alone; more first tokens than there are: all."""
    rng = np.random.default_rng(9)
    c = cache(rng, [16, 3], [700, 90], 4, 2, 128, 16)
    for a, b in (((0, 50), (0, 0)), ((100, 0), (100, 0)), ((1, 5000), (0, 0)), ((1, (1 << 31) - 1), (0, 0))):
        x, y = run(w4v_mod, gpu, c, *a), run(w4v_mod, gpu, c, *b)
        if b == a or a[0] == 0:
            assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])
        else:
            ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], 128 ** -0.5)
            assert np.all(np.abs(x[0] - ref[0]) <= attention_bounds(c, ref)[0])


@pytest.mark.parametrize("D,window,sinks", [(64, 300, 4), (128, 300, 130), (256, 700, 40), (128, 40, 600)])
def test_batch_invariance(w4v_mod, gpu, D, window, sinks):
    """Verified positions equal the one-token steps they stand for, bit for bit, alone or in a batch."""
    rng = np.random.default_rng(13)
    T, lens = 30, [2100, 530, 30, 1029]
    c = cache(rng, [T] * 4, lens, 10, 2, D, 16)
    check(w4v_mod, gpu, c, window, sinks, invariant=True)
    got, lse = run(w4v_mod, gpu, c, window, sinks, invariant=True)
    for b in range(4):
        for t in (0, 1, 7, 13, 22, T - 1):
            one = dict(c, q=c["q"][b * T + t:b * T + t + 1], table=c["table"][b:b + 1],
                       lengths=np.array([lens[b] - T + t + 1], np.int32), offsets=np.array([0, 1], np.int32))
            o1, l1 = run(w4v_mod, gpu, one, window, sinks, invariant=True)
            assert np.array_equal(o1[0], got[b * T + t]) and np.array_equal(l1[0], lse[b * T + t])


def test_rows_of_no_sequence_and_graph_replay(w4v_mod, gpu):
    rng, w = np.random.default_rng(14), w4v_mod
    c = cache(rng, [16, 16], [3000, 1777], 8, 2, 128, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    q = torch.cat([d["q"], d["q"][:5]])                       # a batch padded to a fixed size
    out = torch.full_like(q, 3.0)
    ws = w.workspace(w.paged_attn_workspace_bytes(37, 2, 8, 2, 128, d["table"].shape[1] * 16))
    call = lambda: w.paged_attn(q, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], window=500, sinks=20, out=out, ws=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert torch.all(out[32:] == 3.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["lengths"].copy_(torch.tensor([1000, 40], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], [1000, 40], c["offsets"], 128 ** -0.5, 500, 20)
    assert np.all(np.abs(out[:32].cpu().numpy() - ref[0]) <= attention_bounds(c, ref)[0])
