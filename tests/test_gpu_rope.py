"""rope_append on the GPU against the oracle (double precision)."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import cache

pytestmark = pytest.mark.gpu


def bound(y, x, mul):
    """One rounding to fp16 (2^-11), and fp32 along the way: the angle's fraction of a turn, cos, sin,
    the factor and the two products are each within a few 2^-24 of the pair's size (2^-20 in all)."""
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -20 * mul * np.abs(x.astype(np.float64)).max() * 2 + 2.0 ** -25


def rows(rng, n, Hq, Hkv, D):
    return [rng.standard_normal((n, h, D)).astype(np.float16) for h in (Hq, Hkv, Hkv)]


def check(w, gpu, c, rot, inter, scaling, q, k, v, positions=None, fused=False, in_place=False):
    D = q.shape[2]
    rope = w.Rope(rot, interleaved=inter, scaling=scaling)
    f, mul = paged.frequencies(rot, scaling=scaling)
    d = {x: to_dev(a, gpu) for x, a in c.items() if x != "q"}
    if fused:
        row = torch.cat([to_dev(x, gpu).flatten(1) for x in (q, k, v)], 1)
        heads = [x.shape[1] * D for x in (q, k, v)]
        dq, dk, dv = (x.unflatten(1, (-1, D)) for x in row.split(heads, 1))
    else:
        dq, dk, dv = (to_dev(x, gpu) for x in (q, k, v))
    pos_t = None if positions is None else to_dev(np.asarray(positions, np.int32), gpu)
    qo = w.rope_append(dq, dk, dv, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], rope, positions=pos_t,
                       q_out=dq if in_place else None)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    places = paged.token_places(c["lengths"], c["offsets"])
    at = np.array([p for _, p in places])
    pos = at if positions is None else np.asarray(positions)
    wq, wk = (paged.rotate(x, pos, f, mul, inter) for x in (q, k))
    assert np.all(np.abs(qo.cpu().numpy() - wq) <= bound(wq, q, mul))
    ck, cv = c["k"].astype(np.float64), c["v"].copy()
    tol = np.zeros_like(ck)
    page = c["k"].shape[2]
    bk = bound(wk, k, mul)
    for t, (b, p) in enumerate(places):
        if p >= 0:
            i = c["table"][b, p // page]
            ck[i, :, p % page], tol[i, :, p % page], cv[i, :, p % page] = wk[t], bk[t], v[t]
    assert np.all(np.abs(d["k"].cpu().numpy() - ck) <= tol)          # every other slot untouched
    assert np.array_equal(d["v"].cpu().numpy(), cv)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 50), (128, 128), (128, 32), (128, 96), (128, 2), (128, 0),
                                   (256, 64), (256, 242), (256, 256), (128, 8), (128, 24)])
def test_parts_of_the_head(w4v_mod, gpu, inter, D, rot):
    rng = np.random.default_rng([D, rot])
    c = cache(rng, [1, 0, 7, 20], [1, 9, 40, 300], 1, 2, D, 16)
    check(w4v_mod, gpu, c, rot, inter, None, *rows(rng, 28, 5, 2, D))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", [("linear", 4.0), ("ntk", 4.0), ("yarn", 8.0, 16384.0),
                                     ("banded", 8.0, 1.0, 4.0, 8192.0)])
def test_scalings_far_out(w4v_mod, gpu, inter, scaling):
    """Positions up to 2^31 - 1, given apart from the cache's own (there the oracle's angle itself
    is off by up to 2^-53 of it, 3e-7 radians, inside the bound)."""
    rng = np.random.default_rng(3)
    c = cache(rng, [6], [100], 1, 2, 128, 8)
    check(w4v_mod, gpu, c, 128, inter, scaling, *rows(rng, 6, 4, 2, 128),
          positions=[0, 1, 100_003, 1 << 20, (1 << 31) - 1, 131_071])


def test_fused_rows_and_in_place(w4v_mod, gpu):
    rng = np.random.default_rng(4)
    c = cache(rng, [16, 33], [1000, 33], 1, 4, 128, 64)
    x = rows(rng, 49, 20, 4, 128)
    check(w4v_mod, gpu, c, 128, False, None, *x, fused=True)
    check(w4v_mod, gpu, c, 64, False, None, *x, in_place=True)
    check(w4v_mod, gpu, c, 50, True, None, *x, in_place=True)


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 32, False), (256, 64, True), (64, 22, False), (256, 256, False)])
def test_many_rows(w4v_mod, gpu, D, rot, inter):
    """Enough rows for the kernel that takes a long prompt, more heads than its threads load at once, in place too."""
    rng = np.random.default_rng([D, rot, 9])
    c = cache(rng, [2500, 0, 100], [2600, 5, 100], 1, 3, D, 64)
    x = rows(rng, 2600, 21, 3, D)
    check(w4v_mod, gpu, c, rot, inter, None, *x)
    check(w4v_mod, gpu, c, rot, inter, None, *x, in_place=True)


def test_rows_without_a_place(w4v_mod, gpu):
    """Rows before position 0 and pages that are not there are not written; rows of no sequence are left alone."""
    rng = np.random.default_rng(5)
    c = cache(rng, [4, 2], [40, 20], 1, 2, 64, 16)
    q, k, v = (to_dev(x, gpu) for x in rows(rng, 9, 2, 2, 64))
    c["lengths"] = np.array([2, 20], np.int32)
    c["table"][1, 1] = -1
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    out = torch.full_like(q, 5.0)
    w4v_mod.rope_append(q, k, v, d["k"], d["v"], d["table"], d["lengths"], d["offsets"], w4v_mod.Rope(64), q_out=out)
    torch.cuda.synchronize()
    want = c["v"].copy()
    for t, p in ((2, 0), (3, 1)):
        want[c["table"][0, 0], :, p] = v[t].cpu().numpy()
    assert np.array_equal(d["v"].cpu().numpy(), want)
    assert torch.all(out[6:] == 5.0) and not torch.any(torch.all((out[:6] == 5.0).flatten(1), 1))
