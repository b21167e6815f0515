"""token_logprobs on the GPU against the oracle (double precision)."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import scores

pytestmark = pytest.mark.gpu


def logits(rng, M, V, half=False, size=2.0):
    x = (rng.standard_normal((M, V)) * size).astype(np.float32)
    x[::2, rng.integers(0, V)] += 9
    return x.astype(np.float16) if half else x


def given(rng, M, V, n):
    t = rng.integers(0, V, (M, n)).astype(np.int32)
    if n > 1:
        t[:, -1] = -1
    if n > 2:
        t[:, 1] = V
    return t


def compare(x, tokens, top, temperature, got):
    lp, h, ids, tops = (t.cpu().numpy() for t in got)
    lp = lp.reshape(len(x), -1)
    for r in range(len(x)):
        want = scores.row(x[r], tokens[r], top, temperature)
        per, eh = scores.bounds(x[r], temperature)
        xr = x[r].astype(np.float64)
        high = np.nanmax(np.where(np.isneginf(xr), np.nan, xr)) if np.isfinite(xr).any() else 0.0

        def near(a, b, logit):
            b, logit = np.asarray(b, np.float64), np.asarray(logit, np.float64)
            fin = np.isfinite(b)
            assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~fin & ~np.isnan(b)], b[~fin & ~np.isnan(b)])
            tol = per + 2.0 ** -21 * np.abs(logit[fin] - high) / temperature
            assert np.all(np.abs(a[fin] - b[fin]) <= tol), (r, float(np.max(np.abs(a[fin] - b[fin]) / tol)))
        near(lp[r], want[0], [xr[t] if 0 <= t < len(xr) else 0.0 for t in tokens[r]])
        assert np.array_equal(ids[r], want[2]), (r, ids[r], want[2])
        near(tops[r], want[3], xr[ids[r]])
        assert (np.isnan(h[r]) and np.isnan(want[1])) or abs(h[r] - want[1]) <= eh, (r, h[r], want[1], eh)


def check(w, gpu, x, tokens, top=5, temperature=1.0, **kw):
    got = w.token_logprobs(to_dev(x, gpu), to_dev(tokens, gpu), top=top, temperature=temperature, **kw)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    compare(x, tokens.reshape(len(x), -1), top, temperature, got)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 7, 8, 9, 31, 100, 127, 128, 129, 511, 1000, 2047, 2048, 2049, 4095, 4096,
                               4097, 8193, 16385, 20479, 20480, 20481])
def test_vocabularies_around_vectors_and_pieces(w4v_mod, gpu, half, V):
    rng = np.random.default_rng([V, half])
    check(w4v_mod, gpu, logits(rng, 3, V, half), given(rng, 3, V, 3), top=min(V, 20))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [40961, 81923, 151936, 163840, 163841, 200003, 400001])
def test_large_vocabularies(w4v_mod, gpu, half, V):
    """Clusters of every size, and pieces that a CTA takes in turn."""
    rng = np.random.default_rng([V, half])
    check(w4v_mod, gpu, logits(rng, 2, V, half), given(rng, 2, V, 4), top=32, temperature=0.7)


@pytest.mark.parametrize("M,V", [(400, 1000), (40, 30011), (20, 50257), (160, 21000)])
def test_many_rows(w4v_mod, gpu, M, V):
    rng = np.random.default_rng([M, V])
    check(w4v_mod, gpu, logits(rng, M, V), given(rng, M, V, 1), top=7)


@pytest.mark.parametrize("half,V,top", [(False, 20011, 32), (True, 20011, 5), (False, 151936, 20), (True, 151936, 32)])
def test_a_long_prompt(w4v_mod, gpu, half, V, top):
    """Enough rows for small CTAs at any vocabulary; rows of every shape among them, and all of a few values."""
    w, M = w4v_mod, 1300
    g = torch.Generator(device=gpu).manual_seed(V)
    x = torch.randn((M, V), generator=g, device=gpu).mul_(2).to(torch.float16 if half else torch.float32)
    shaped = shaped_rows(V, half)
    at = [7 + 90 * i for i in range(len(shaped))]
    x[at] = to_dev(shaped, gpu)
    x[3, V // 2], x[5, ::2], x[1299, :] = float("nan"), -float("inf"), 0.25
    t = torch.randint(0, V, (M, 2), generator=g, device=gpu).int()
    got = w.token_logprobs(x, t, top=top)
    rows = sorted([0, 3, 5, 640, 1299] + at)
    compare(x[rows].cpu().numpy(), t[rows].cpu().numpy(), top, 1.0, [y[rows] for y in got])
    few = w.token_logprobs(x[640:700], t[640:700], top=top)
    assert torch.equal(few[2], got[2][640:700])
    assert torch.allclose(few[0], got[0][640:700], rtol=1e-5, atol=2e-5) and torch.allclose(few[1], got[1][640:700], rtol=1e-5)


@pytest.mark.parametrize("top", [0, 1, 2, 19, 31, 32])
@pytest.mark.parametrize("temperature", [0.05, 0.5, 1.0, 3.0])
def test_alternatives_and_temperatures(w4v_mod, gpu, top, temperature):
    rng = np.random.default_rng(top)
    check(w4v_mod, gpu, logits(rng, 3, 9001), given(rng, 3, 9001, 2), top=top, temperature=temperature)


def shaped_rows(V, half):
    i = np.arange(V, dtype=np.float64)
    few = np.full(V, -np.inf)
    few[[V // 3, V - 1]] = 1.5, 1.5
    rows = [np.zeros(V), i / V * 30, -i / V * 30, np.where(i % 2 == 0, 1.0, 2.0), np.where(i < V - 3, 1.0, 0.5),
            np.full(V, -7.0), np.where(i == V - 1, 3.0, -np.inf), few, np.floor(i / V * 10), np.where(i % 97 == 3, 4.0, -1.0),
            np.where(i % 3 == 0, -0.0, 0.0), np.where(i < 40, 2.0, -np.inf), np.where(i >= V - 40, 2.0, -np.inf),
            np.where(i % 16 < 4, 20.0 + i / V, 0.0)]
    return np.stack(rows).astype(np.float16 if half else np.float32)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [50, 700, 5000, 21000, 170001])
@pytest.mark.parametrize("top", [3, 32])
def test_ties_orders_and_masks(w4v_mod, gpu, half, V, top):
    """Rows of one value, of two, in order up and down, with few tokens above -inf, alternatives in a few threads' hands."""
    x = shaped_rows(V, half)
    check(w4v_mod, gpu, x, given(np.random.default_rng(1), len(x), V, 2), top=top)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("M,V", [(60, 5000), (5, 170001), (1300, 20011)])
@pytest.mark.parametrize("top", [1, 20, 32])
def test_rows_gone_through_again_every_time(w4v_mod, gpu, half, M, V, top):
    """Rows in ascending order, and of values that very many tokens share, many times over: the last batch leaves
    hundreds of candidates, which must not be taken for the list's length behind it."""
    i = torch.arange(V, device=gpu, dtype=torch.float64)
    shapes = [i / V * 30, torch.floor(i / V * 10), torch.where(i % 2 == 0, 1.0, 2.0), (i % 4096) / 200,
              torch.where(i % 16 < 4, 20.0 + i / V, 0.0), i / V * 30 - 60 * (i % 3 == 1)]
    x = torch.stack(shapes).to(torch.float16 if half else torch.float32)
    want = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top].int()
    at = torch.arange(M, device=gpu) % len(x)
    x, want = x[at], want[at]
    for _ in range(100):
        ids, lps = w4v_mod.token_logprobs(x, top=top)[2:]
        assert torch.equal(ids, want)
        assert torch.all(lps[:, 1:] <= lps[:, :-1])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [64, 3001, 25000])
def test_what_is_not_finite(w4v_mod, gpu, half, V):
    rng = np.random.default_rng(2)
    x = logits(rng, 8, V, half)
    x[0] = -np.inf
    x[1, V // 2] = np.nan
    x[2, V - 1] = np.inf
    x[3] = np.nan
    x[4, :V - 2] = -np.inf
    x[5, ::3] = -np.inf
    x[6, 0], x[6, 1] = np.nan, -np.inf
    x[7, 1:] = -np.inf
    check(w4v_mod, gpu, x, given(rng, 8, V, 4), top=32)


@pytest.mark.parametrize("size", [1e-30, 1e4, 3e37])
def test_sizes(w4v_mod, gpu, size):
    """Logits that differ by nothing, by thousands, and by more than fp32 holds."""
    rng = np.random.default_rng(3)
    x = np.clip(rng.standard_normal((4, 6001)) * size, -3e38, 3e38).astype(np.float32)
    check(w4v_mod, gpu, x, given(rng, 4, 6001, 3), top=9)


@pytest.mark.parametrize("V", [500, 6001, 40_000])
@pytest.mark.parametrize("size,temperature", [(1e30, 1e30), (1e37, 1e37), (3e37, 1e38), (1.0, 1e38), (1e-37, 1e-37)])
def test_logits_and_temperatures_of_a_size(w4v_mod, gpu, V, size, temperature):
    """Ordinary ratios of numbers at the ends of fp32: no sum is taken in the logits' own unit."""
    rng = np.random.default_rng([V, 5])
    x = np.clip(rng.standard_normal((3, V)) * size, -1.6e38, 1.6e38).astype(np.float32)
    check(w4v_mod, gpu, x, given(rng, 3, V, 3), top=9, temperature=temperature)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("off,pad", [(0, 1), (1, 0), (2, 3), (3, 2), (5, 7), (7, 8)])
def test_rows_anywhere(w4v_mod, gpu, half, off, pad):
    """Rows that begin on no boundary, of a longer matrix whose other elements are NaN."""
    rng, M, V = np.random.default_rng([off, pad]), 5, 4501
    x, t = logits(rng, M, V, half), given(rng, M, V, 2)
    wide = torch.full((M * (V + pad) + off + 8,), float("nan"), dtype=torch.float16 if half else torch.float32, device=gpu)
    view = wide[off:off + M * (V + pad)].view(M, V + pad)[:, :V]
    view.copy_(to_dev(x, gpu))
    got = w4v_mod.token_logprobs(view, to_dev(t, gpu), top=20)
    compare(x, t, 20, 1.0, got)


@pytest.mark.parametrize("half,M,V,top", [(False, 4, 1 << 22, 0), (False, 4, 1 << 26, 0), (False, 4, 1 << 24, 3),
                                          (True, 4, 1 << 26, 0), (True, 4, 1 << 26, 2), (False, 1300, 400_000, 0),
                                          (True, 1300, 400_000, 0), (False, 1300, 800_000, 5)])
def test_long_sums_of_equal_terms(w4v_mod, gpu, half, M, V, top):
    """One value over and over beside a higher one: the terms are equal and no power of two, so that what the additions
    round off adds up instead of averaging out.  The bound is that of any row (scores.bounds), the expectation a
    period's."""
    d = torch.tensor([-0.3, -1.7, -np.log(3.0), -2.9], device=gpu)
    d = (d.half() if half else d).double()
    low = d.cpu().numpy()[np.arange(M) % 4]
    x = torch.zeros((M, V), device=gpu, dtype=torch.float16 if half else torch.float32)
    for r in range(M):
        x[r].view(-1, 4)[:, 1:] = float(low[r])
    t = torch.tensor([[0, 1]], dtype=torch.int32, device=gpu).expand(M, 2).contiguous()
    lp, h, _, _ = (y.cpu().numpy() for y in w4v_mod.token_logprobs(x, t, top=top))
    for r in range(M):
        period = np.array([0.0, low[r], low[r], low[r]])
        per, eh = scores.bounds(period)
        more = 2.0 ** -22 * np.log(V / 4)                  # the logarithm's own term in both bounds, of the whole row
        lse = np.log(V / 4) + np.log(np.exp(period).sum())
        p = np.exp(period - lse) * (V / 4)
        assert abs(lp[r, 0] + lse) <= per + more
        assert abs(lp[r, 1] - (low[r] - lse)) <= per + more + 2.0 ** -21 * abs(low[r])
        assert abs(h[r] - (lse - (p * period).sum())) <= eh + more, (r, h[r], lse - (p * period).sum(), eh + more)


def test_rows_past_32_bits(w4v_mod, gpu):
    """Rows 2^30 elements apart."""
    rng = np.random.default_rng(4)
    x, t = logits(rng, 3, 2000, True), given(rng, 3, 2000, 1)
    big = torch.empty((2 << 30) + 2000, dtype=torch.float16, device=gpu)
    view = torch.as_strided(big, (3, 2000), (1 << 30, 1))
    view.copy_(to_dev(x, gpu))
    compare(x, t, 4, 1.0, w4v_mod.token_logprobs(view, to_dev(t, gpu), top=4))


def test_forms_of_a_call(w4v_mod, gpu):
    """Tokens as a vector, none at all, results into given tensors, no rows; the same bits every time."""
    rng, w = np.random.default_rng(5), w4v_mod
    x = logits(rng, 6, 30000)
    d, t = to_dev(x, gpu), to_dev(given(rng, 6, 30000, 1), gpu)
    a = w.token_logprobs(d, t[:, 0].contiguous(), top=8)
    assert a[0].shape == (6,) and a[2].shape == (6, 8)
    b = w.token_logprobs(d, t, top=8)
    for _ in range(5):
        out = tuple(torch.full_like(y, 3) for y in b)
        assert w.token_logprobs(d, t, top=8, out=out) is out
        assert all(torch.equal(p, q) for p, q in zip(b, out))
    assert torch.equal(a[0], b[0][:, 0]) and all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))
    none = w.token_logprobs(d)
    assert none[0].shape == (6, 0) and none[2].shape == (6, 0) and torch.equal(none[1], b[1])
    empty = w.token_logprobs(d[:0], t[:0], top=8)
    assert [tuple(y.shape) for y in empty] == [(0, 1), (0,), (0, 8), (0, 8)]


def test_results_that_do_not_fit_are_refused(w4v_mod, gpu):
    w, i = w4v_mod, torch.int32
    x, t = torch.zeros(3, 50, device=gpu), torch.zeros(3, 2, dtype=i, device=gpu)
    out = lambda top: [torch.zeros(3, 2, device=gpu), torch.zeros(3, device=gpu), torch.zeros(3, top, dtype=i, device=gpu),  # noqa: E731
                       torch.zeros(3, top, device=gpu)]
    w.token_logprobs(x, t, top=3, out=out(3))
    for at, bad, code in ((0, torch.zeros(3, 3, device=gpu), "SHAPE"), (1, torch.zeros(2, device=gpu), "SHAPE"),
                          (2, torch.zeros(3, 4, dtype=i, device=gpu), "SHAPE"), (3, torch.zeros(2, 3, device=gpu), "SHAPE"),
                          (0, torch.zeros(3, 2, device=gpu).half(), "ARG"), (1, torch.zeros(6, device=gpu)[::2], "ARG"),
                          (2, torch.zeros(3, 3, device=gpu), "ARG"), (3, torch.zeros(3, 3), "ARG")):
        given_out = out(3)
        given_out[at] = bad
        with pytest.raises(w.W4VError) as e:
            w.token_logprobs(x, t, top=3, out=given_out)
        assert e.value.code == getattr(w, "ERR_" + code)
    with pytest.raises(w.W4VError) as e:
        w.token_logprobs(x, t.cpu(), top=3)
    assert e.value.code == w.ERR_ARG


def test_another_stream_and_graph_replay(w4v_mod, gpu):
    rng, w = np.random.default_rng(6), w4v_mod
    x, t = logits(rng, 4, 12345), given(rng, 4, 12345, 2)
    d, dt = to_dev(x, gpu), to_dev(t, gpu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = w.token_logprobs(d, dt, top=5, stream=s)
    s.synchronize()
    compare(x, t, 5, 1.0, got)
    out = tuple(torch.empty_like(y) for y in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.token_logprobs(d, dt, top=5, out=out)
    x2 = logits(rng, 4, 12345)
    d.copy_(to_dev(x2, gpu))
    g.replay()
    torch.cuda.synchronize()
    compare(x2, t, 5, 1.0, out)


def test_scores_of_the_lm_head(w4v_mod, gpu):
    """The verify step's own logits: the argmax is the first alternative."""
    rng, w = np.random.default_rng(7), w4v_mod
    X = to_dev(rng.standard_normal((16, 256)).astype(np.float16), gpu)
    W8 = to_dev(rng.integers(-127, 128, (4096, 256)).astype(np.int8), gpu)
    s8 = to_dev((rng.random(4096) * 0.002).astype(np.float16), gpu)
    x = torch.empty((16, 4096), dtype=torch.float32, device=gpu)
    best = w.w8_lmhead_argmax(X, W8, s8, logits=x)
    got = w.token_logprobs(x, best, top=3)
    assert torch.equal(got[2][:, 0], best) and torch.equal(got[3][:, 0], got[0])
    compare(x.cpu().numpy(), best.cpu().numpy()[:, None], 3, 1.0, got)
