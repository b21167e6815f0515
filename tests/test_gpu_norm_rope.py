"""norm_rope_append on the GPU against the oracle (double precision)."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import cache

pytestmark = pytest.mark.gpu


def bound(y, normed, mul):
    """One rounding to fp16 (2^-11 of the value, 2^-25 among subnormals), and fp32 along the way: the sum of
    256 squares is within 256 roundings of 2^-24, half of that counts in its root, and the factor's root, the
    weights' sums and products, the angle, cos, sin and the two products add some 2^-20: 2^-16 of a pair's size."""
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -16 * mul * 2 * np.abs(normed).max(-1, keepdims=True) + 2.0 ** -25


def rows(rng, n, Hq, Hkv, D, size=1.0):
    return [np.clip(rng.standard_normal((n, h, D)) * size, -65504, 65504).astype(np.float16) for h in (Hq, Hkv, Hkv)]


def weights(rng, D, centred=False):
    return [(rng.standard_normal(D) * 0.3 + (0.0 if centred else 1.0)).astype(np.float16) for _ in range(2)]


def check(w, gpu, c, rot, inter, q, k, v, wq=None, wk=None, eps=1e-6, centred=False, scaling=None, positions=None,
          fused=False, in_place=False, stream=None):
    D = q.shape[2]
    rope = w.Rope(rot, interleaved=inter, scaling=scaling)
    norm = w.HeadNorm(*(None if x is None else to_dev(x, gpu) for x in (wq, wk)), eps=eps, zero_centred=centred)
    f, mul = paged.frequencies(rot, scaling=scaling)
    d = {x: to_dev(a, gpu) for x, a in c.items() if x != "q"}
    if fused:
        row = torch.cat([to_dev(x, gpu).flatten(1) for x in (q, k, v)], 1)
        dq, dk, dv = (x.unflatten(1, (-1, D)) for x in row.split([x.shape[1] * D for x in (q, k, v)], 1))
    else:
        dq, dk, dv = (to_dev(x, gpu) for x in (q, k, v))
    pos_t = None if positions is None else to_dev(np.asarray(positions, np.int32), gpu)
    torch.cuda.synchronize()
    qo = w.norm_rope_append(dq, dk, dv, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope, norm,
                            q_out=dq if in_place else None, positions=pos_t, stream=stream)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    places = paged.token_places(c["lengths"], c["offsets"])
    pos = np.array([p for _, p in places]) if positions is None else np.asarray(positions)
    nq, nk = (paged.head_norm(x, g, eps, float(centred)) for x, g in ((q, wq), (k, wk)))
    yq, yk = (paged.rotate(x, pos, f, mul, inter) for x in (nq, nk))
    assert np.all(np.abs(qo.cpu().numpy() - yq) <= bound(yq, nq, mul))
    ck, cv, tol = c["k"].astype(np.float64), c["v"].copy(), np.zeros(c["k"].shape)
    page, bk = c["k"].shape[2], bound(yk, nk, mul)
    for t, (b, p) in enumerate(places):
        if p >= 0:
            i = c["table"][b, p // page]
            ck[i, :, p % page], tol[i, :, p % page], cv[i, :, p % page] = yk[t], bk[t], v[t]
    assert np.all(np.abs(d["k"].cpu().numpy() - ck) <= tol)          # every other slot untouched
    assert np.array_equal(d["v"].cpu().numpy(), cv)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 50), (128, 128), (128, 32), (128, 96), (128, 2), (128, 0),
                                   (256, 64), (256, 242), (256, 256), (128, 8), (128, 24), (64, 16)])
def test_parts_of_the_head(w4v_mod, gpu, inter, D, rot):
    rng = np.random.default_rng([D, rot])
    c = cache(rng, [1, 0, 7, 20], [1, 9, 40, 300], 1, 2, D, 16)
    check(w4v_mod, gpu, c, rot, inter, *rows(rng, 28, 5, 2, D), *weights(rng, D))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (21, 3), (40, 8), (66, 1), (20, 20)])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 64, True), (256, 50, False)])
def test_head_counts(w4v_mod, gpu, Hq, Hkv, D, rot, inter):
    rng = np.random.default_rng([Hq, Hkv, D])
    c = cache(rng, [3, 1], [50, 17], 1, Hkv, D, 8)
    check(w4v_mod, gpu, c, rot, inter, *rows(rng, 4, Hq, Hkv, D), *weights(rng, D))


@pytest.mark.parametrize("which", ["none", "q", "k", "both"])
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("rot", [128, 50])
def test_weights(w4v_mod, gpu, which, centred, rot):
    rng = np.random.default_rng(3)
    c = cache(rng, [5], [40], 1, 2, 128, 16)
    wq, wk = weights(rng, 128, centred)
    check(w4v_mod, gpu, c, rot, False, *rows(rng, 5, 6, 2, 128), wq if which in ("q", "both") else None,
          wk if which in ("k", "both") else None, centred=centred and which == "both")


@pytest.mark.parametrize("size,eps", [(1.0, 1e-6), (6e-4, 1e-6), (2e4, 1e-5), (1.0, 0.0), (1.0, 0.5)])
def test_sizes_and_eps(w4v_mod, gpu, size, eps):
    """Heads from where eps decides to where fp16 ends."""
    rng = np.random.default_rng(4)
    c = cache(rng, [9], [33], 1, 2, 128, 16)
    check(w4v_mod, gpu, c, 128, False, *rows(rng, 9, 4, 2, 128, size), *weights(rng, 128), eps=eps)


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (50, False)])
def test_zeros_and_what_is_not_finite_stay_in_their_head(w4v_mod, gpu, rot, inter):
    """A head of zeros gives zeros, an infinity or a NaN spoils its own head and no other."""
    rng = np.random.default_rng(5)
    c = cache(rng, [3], [30], 1, 2, 128, 16)
    q, k, v = rows(rng, 3, 4, 2, 128)
    clean = [x.copy() for x in (q, k, v)]
    q[0, 1], q[1, 2, 5], k[2, 0, 127] = 0, np.inf, np.nan
    w, d = w4v_mod, {x: to_dev(a, gpu) for x, a in c.items()}
    call = lambda a: w.norm_rope_append(*(to_dev(x, gpu) for x in a), d["k"], d["v"], d["table"], d["lengths"],  # noqa: E731
                                        d["offsets"], w.Rope(rot, interleaved=inter), w.HeadNorm())
    want = call(clean).clone()
    kept = d["k"].clone()
    got = call((q, k, v))
    assert torch.all(got[0, 1] == 0) and torch.isnan(got[1, 2, 5])
    same = torch.ones_like(got, dtype=torch.bool)
    same[0, 1], same[1, 2] = False, False
    assert torch.equal(got[same], want[same])
    at = d["table"][0, 29 // 16].long()
    assert torch.all(torch.isnan(d["k"][at, 0, 29 % 16]))
    kept[at, 0, 29 % 16] = d["k"][at, 0, 29 % 16]
    assert torch.equal(d["k"].nan_to_num(7.0), kept.nan_to_num(7.0))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [64, 50, 0])
@pytest.mark.parametrize("n", [3, 4000])
def test_an_infinity_divides_the_rest_of_its_head(w4v_mod, gpu, n, rot, inter):
    """x / sqrt(inf) is 0 for what is finite; the infinity itself, and what it is rotated with, becomes NaN."""
    rng, w = np.random.default_rng([n, rot, inter]), w4v_mod
    c = cache(rng, [n], [n + 3], 1, 2, 128, 64)
    q, k, v = rows(rng, n, 3, 2, 128)
    bad = {0: (100,), 1: (101,), 2: (66, 127)} if rot else {0: (0,), 1: (1,), 2: (66, 127)}
    for h, at in bad.items():
        for i in at:
            q[:, h, i] = np.inf if i % 2 else -np.inf
    k[:, 1, 111] = np.inf
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    wq, wk = weights(rng, 128)
    got = w.norm_rope_append(*(to_dev(x, gpu) for x in (q, k, v)), d["k"], d["v"], d["table"], d["lengths"], d["offsets"],
                             w.Rope(rot, interleaved=inter), w.HeadNorm(to_dev(wq, gpu), to_dev(wk, gpu)))
    for h, at in bad.items():
        nan = torch.zeros(128, dtype=torch.bool, device=gpu)
        nan[list(at)] = True
        assert torch.equal(torch.isnan(got[:, h]), nan.expand(n, 128))
        assert torch.all(got[:, h][:, ~nan] == 0)
    page = d["k"][d["table"][0, 0].long(), 1, 3:10]               # the first new tokens' second key head
    nan = torch.arange(128, device=gpu) == 111
    for row in page[:min(n, 7)]:
        assert torch.equal(torch.isnan(row), nan) and torch.all(row[~nan] == 0)


def test_positions_and_scalings(w4v_mod, gpu):
    rng = np.random.default_rng(6)
    c = cache(rng, [6], [100], 1, 2, 128, 8)
    for scaling in (("linear", 4.0), ("ntk", 4.0), ("yarn", 8.0, 16384.0), ("banded", 8.0, 1.0, 4.0, 8192.0)):
        check(w4v_mod, gpu, c, 128, False, *rows(rng, 6, 4, 2, 128), *weights(rng, 128), scaling=scaling,
              positions=[0, 1, 100_003, 1 << 20, (1 << 31) - 1, 131_071])


def test_fused_rows_in_place_and_another_stream(w4v_mod, gpu):
    rng = np.random.default_rng(7)
    c = cache(rng, [16, 33], [1000, 33], 1, 4, 128, 64)
    x = rows(rng, 49, 20, 4, 128) + weights(rng, 128)
    check(w4v_mod, gpu, c, 128, False, *x, fused=True)
    check(w4v_mod, gpu, c, 64, False, *x, in_place=True)
    check(w4v_mod, gpu, c, 50, True, *x, in_place=True)
    check(w4v_mod, gpu, c, 128, True, *x, stream=torch.cuda.Stream())


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 32, False), (256, 64, True), (64, 22, False), (256, 256, False)])
def test_many_rows(w4v_mod, gpu, D, rot, inter):
    """Enough rows for the kernel that takes a long prompt, more heads than its threads load at once, in place too."""
    rng = np.random.default_rng([D, rot, 9])
    c = cache(rng, [2500, 0, 100], [2600, 5, 100], 1, 3, D, 64)
    x = rows(rng, 2600, 21, 3, D) + weights(rng, D)
    check(w4v_mod, gpu, c, rot, inter, *x)
    check(w4v_mod, gpu, c, rot, inter, *x, in_place=True)


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (64, 32, True), (128, 128, False), (256, 64, False), (256, 256, True)])
@pytest.mark.parametrize("Hq,Hkv", [(5, 3), (8, 2)])
def test_a_long_prompt(w4v_mod, gpu, D, rot, inter, Hq, Hkv):
    """Enough rows for a warp each; passes that hold query and key heads, and rows without a place or a sequence."""
    rng, w = np.random.default_rng([D, rot, Hq]), w4v_mod
    n = 4100
    c = cache(rng, [3000, 0, n - 3000], [3100, 5, n - 3000], 1, Hkv, D, 64)
    x = rows(rng, n, Hq, Hkv, D) + weights(rng, D, True)
    check(w, gpu, c, rot, inter, *x, centred=True)
    check(w, gpu, c, rot, inter, *x[:3], in_place=True)
    c["lengths"][0] = 2990                                # its first ten rows sit before position 0
    c["table"][2, 3] = -1
    d = {a: to_dev(b, gpu) for a, b in c.items()}
    q, k, v = (to_dev(torch.cat([torch.from_numpy(b), torch.from_numpy(b[:7])]).numpy(), gpu) for b in x[:3])
    out = torch.full_like(q, 5.0)
    w.norm_rope_append(q, k, v, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], w.Rope(rot, interleaved=inter),
                       w.HeadNorm(), q_out=out)
    torch.cuda.synchronize()
    assert torch.all(out[n:] == 5.0) and not torch.any(torch.all((out[:n] == 5.0).flatten(1), 1))
    want = c["v"].copy()
    for t in range(n):
        b, p = (0, t - 10) if t < 3000 else (2, t - 3000)
        if p >= 0 and c["table"][b, p // 64] >= 0:
            want[c["table"][b, p // 64], :, p % 64] = x[2][t]
    assert np.array_equal(d["v"].cpu().numpy(), want)


def test_rows_without_a_place(w4v_mod, gpu):
    """Rows before position 0 and pages that are not there are not written; rows of no sequence are left alone."""
    rng = np.random.default_rng(8)
    w = w4v_mod
    for rot in (64, 50):
        c = cache(rng, [4, 2], [40, 20], 1, 2, 64, 16)
        q, k, v = (to_dev(x, gpu) for x in rows(rng, 9, 2, 2, 64))
        c["lengths"] = np.array([2, 20], np.int32)
        c["table"][1, 1] = -1
        d = {x: to_dev(a, gpu) for x, a in c.items()}
        out = torch.full_like(q, 5.0)
        w.norm_rope_append(q, k, v, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], w.Rope(rot), w.HeadNorm(),
                           q_out=out)
        torch.cuda.synchronize()
        want = c["v"].copy()
        for t, p in ((2, 0), (3, 1)):
            want[c["table"][0, 0], :, p] = v[t].cpu().numpy()
        assert np.array_equal(d["v"].cpu().numpy(), want)
        changed = (d["k"].cpu().numpy() != c["k"]).any(axis=(1, 3))
        assert changed.sum() == 2 and changed[c["table"][0, 0], :2].all()
        assert torch.all(out[6:] == 5.0) and not torch.any(torch.all((out[:6] == 5.0).flatten(1), 1))


def test_graph_replay_follows_what_changes(w4v_mod, gpu):
    rng, w = np.random.default_rng(9), w4v_mod
    c = cache(rng, [3], [40], 1, 2, 128, 16)
    q, k, v = rows(rng, 3, 4, 2, 128)
    wq, wk = weights(rng, 128)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    dev = [to_dev(x, gpu) for x in (q, k, v)]
    rope, norm, out = w.Rope(128), w.HeadNorm(to_dev(wq, gpu), to_dev(wk, gpu)), torch.empty_like(dev[0])
    call = lambda: w.norm_rope_append(*dev, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope, norm, q_out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["lengths"].fill_(20)
    norm.q_weight.fill_(0.5)
    g.replay()
    torch.cuda.synchronize()
    f, mul = paged.frequencies(128)
    nq = paged.head_norm(q, np.full(128, 0.5))
    y = paged.rotate(nq, [17, 18, 19], f, mul, False)
    assert np.all(np.abs(out.cpu().numpy() - y) <= bound(y, nq, mul))


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 96, True), (256, 64, False), (128, 50, False), (64, 22, True)])
def test_rows_do_not_depend_on_the_others(w4v_mod, gpu, D, rot, inter):
    """The same bits in a long prompt, in a chunk of it and alone: verified positions equal the steps they stand for."""
    rng, w = np.random.default_rng([D, 11]), w4v_mod
    c = cache(rng, [4000], [4096], 1, 2, D, 64)
    q, k, v = (to_dev(x, gpu) for x in rows(rng, 4000, 6, 2, D))
    norm = w.HeadNorm(*(to_dev(x, gpu) for x in weights(rng, D)))
    d, rope = {x: to_dev(a, gpu) for x, a in c.items()}, w.Rope(rot, interleaved=inter)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    whole = w.norm_rope_append(q, k, v, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope, norm)
    kept = d["k"].clone()
    for a, b in ((0, 2500), (17, 18), (1000, 1016), (3999, 4000)):
        got = w.norm_rope_append(q[a:b], k[a:b], v[a:b], d["k"], d["v"], d["table"], i32(96 + b), i32(0, b - a), rope, norm)
        assert torch.equal(got, whole[a:b]) and torch.equal(d["k"], kept)


@pytest.mark.parametrize("D,rot,inter", [(128, 32, False), (64, 16, False), (256, 64, True), (64, 8, True), (128, 50, False),
                                         (64, 22, True), (128, 0, False)])
def test_zeros_keep_their_signs_in_every_call(w4v_mod, gpu, D, rot, inter):
    """Bit for bit means zeros too: negative ones among the inputs, past the rotated part and in it."""
    rng, w = np.random.default_rng([D, rot, 12]), w4v_mod
    c = cache(rng, [4000], [4096], 1, 2, D, 64)
    x = [np.where(rng.random(a.shape) < 0.3, np.float16(-0.0), np.where(rng.random(a.shape) < 0.2, np.float16(0.0), a))
         for a in rows(rng, 4000, 6, 2, D)]
    q, k, v = (to_dev(a, gpu) for a in x)
    norm = w.HeadNorm(*(to_dev(g * np.where(rng.random(D) < 0.5, 1, -1).astype(np.float16), gpu) for g in weights(rng, D)))
    d, rope = {a: to_dev(b, gpu) for a, b in c.items()}, w.Rope(rot, interleaved=inter)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=gpu)  # noqa: E731
    bits = lambda a: a.view(torch.int16)  # noqa: E731
    whole = w.norm_rope_append(q, k, v, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope, norm)
    kept = d["k"].clone()
    for a, b in ((0, 2500), (17, 18), (1000, 1016), (3999, 4000)):
        got = w.norm_rope_append(q[a:b], k[a:b], v[a:b], d["k"], d["v"], d["table"], i32(96 + b), i32(0, b - a), rope, norm)
        assert torch.equal(bits(got), bits(whole[a:b])) and torch.equal(bits(d["k"]), bits(kept))


def test_agrees_with_the_separate_steps(w4v_mod, gpu):
    """rope_append of heads normed beforehand: one more rounding to fp16, of the normed head."""
    rng, w = np.random.default_rng(10), w4v_mod
    c = cache(rng, [12], [90], 1, 2, 256, 16)
    q, k, v = (to_dev(x, gpu) for x in rows(rng, 12, 6, 2, 256))
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    cache_args = [d[x] for x in ("k", "v", "table", "lengths", "offsets")]
    rope = w.Rope(64)
    got = w.norm_rope_append(q, k, v, *cache_args, rope, w.HeadNorm())
    unit = [(x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()) for x in (q, k)]
    two = w.rope_append(unit[0].half(), unit[1].half(), v, *cache_args, rope)
    # both are within a rounding of the rotated heads, and the second had its input rounded before (2^-11 of a pair's size)
    size = unit[0].abs().amax(-1, keepdim=True)
    assert torch.all((got.double() - two.double()).abs() <= 2.0 ** -10 * (got.double().abs() + size))
