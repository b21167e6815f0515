"""Pins of the paged cache's oracle by cases small enough to work by hand, and
the host side of the rotary phases against it (no GPU)."""
import math

import numpy as np
import pytest

from oracle import paged


def test_attention_by_hand():
    """Two cached tokens with scores 0 and ln 3: weights 1/4 and 3/4 for the second row, 1 for the first."""
    k = np.zeros((1, 1, 8, 64))
    v = np.zeros((1, 1, 8, 64))
    k[0, 0, 1, 0] = math.log(3.0)
    v[0, 0, 0, 5], v[0, 0, 1, 5], v[0, 0, 1, 6] = 4.0, 8.0, -4.0
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 1.0
    o, lse, mag, absdot = paged.attention(q, k, v, np.zeros((1, 1), int), [2], [0, 2], 1.0)
    assert np.allclose(o[0, 0, 5], 4.0) and np.allclose(o[1, 0, 5:7], [7.0, -3.0])
    assert np.allclose(mag[1, 0, 5:7], [7.0, 3.0]) and np.allclose(lse[:, 0], [0.0, math.log(4.0)])
    assert np.allclose(absdot[:, 0], [0.0, math.log(3.0)])
    o, lse, _, _ = paged.attention(q, k, v, np.zeros((1, 1), int), [2], [0, 2], 1.0, window=1)
    assert np.allclose(o[1, 0, 5:7], [8.0, -4.0]) and np.allclose(lse[1, 0], math.log(3.0))
    o, lse, _, _ = paged.attention(q, k, v, np.zeros((1, 1), int), [1], [0, 2], 1.0)      # row 0 sits before the cache
    assert np.all(o[0] == 0) and lse[0, 0] == -np.inf and np.allclose(o[1, 0, 5], 4.0)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_hand(inter):
    """A quarter turn takes (1, 0) to (0, 1); elements past the pairs stay."""
    x = np.zeros((1, 1, 8))
    x[0, 0, 0], x[0, 0, 7] = 1.0, 3.0
    y = paged.rotate(x, [1], [math.pi / 2, 0.0], 1.0, inter)
    assert np.allclose(y[0, 0], [0, 1, 0, 0, 0, 0, 0, 3] if inter else [0, 0, 1, 0, 0, 0, 0, 3])


def test_scalings_by_hand():
    f, m = paged.frequencies(4, 100.0)
    assert np.allclose(f, [1.0, 0.1]) and m == 1.0
    assert np.allclose(paged.frequencies(4, 100.0, ("linear", 2.0))[0], [0.5, 0.05])
    assert np.allclose(paged.frequencies(4, 100.0, ("ntk", 3.0))[0], [1.0, 900.0 ** -0.5])
    f, m = paged.frequencies(64, 10000.0, ("yarn", 8.0, 4096.0))
    g, _ = paged.frequencies(64, 10000.0)
    assert np.allclose(f[0], g[0]) and np.allclose(f[-1], g[-1] / 8) and np.isclose(m, 0.1 * math.log(8) + 1)
    f, _ = paged.frequencies(64, 10000.0, ("banded", 8.0, 1.0, 4.0, 8192.0))
    assert np.allclose(f[0], g[0]) and np.allclose(f[-1], g[-1] / 8)


@pytest.mark.parametrize("rot", [2, 6, 64, 114, 128, 256])
@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("ntk", 4.0), ("yarn", 8.0, 16384.0),
                                     ("yarn", 2.5, 100.0, 16.0, 2.0), ("banded", 8.0, 1.0, 4.0, 8192.0)])
def test_phases_against_the_oracle(w4v_mod, rot, scaling):
    """A phase is a truncated 2^-64 of a turn, from doubles that both sides round a few times each."""
    if rot == 2 and scaling and scaling[0] == "ntk":
        with pytest.raises(w4v_mod.W4VError) as e:
            w4v_mod.Rope(rot, scaling=scaling, device="cpu")
        assert e.value.code == w4v_mod.ERR_SHAPE
        return
    rope = w4v_mod.Rope(rot, scaling=scaling, device="cpu")
    f, mul = paged.frequencies(rot, scaling=scaling)
    turns = rope.phases.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs(turns * 2 * math.pi - f) <= 64 * 2.0 ** -53 * f + 2.0 ** -60)
    assert abs(rope.mul - mul) <= 2.0 ** -23 * mul


def test_pool_by_hand():
    """Page 4, six pages: extend, roll back, share, copy on write, compact."""
    p = paged.Pool(np.arange(6.0).reshape(1, 6, 1), np.zeros(6, int), np.full((3, 4), -1), np.zeros(3, int), 4)
    assert p.extend([5, 3, 0]) == 0                                  # pages 0, 1 | 2
    assert p.table[0].tolist() == [0, 1, -1, -1] and p.table[1].tolist() == [2, -1, -1, -1]
    assert p.fork([0], [2]) == 0                                     # page 0 shared, page 1 copied to 3
    assert p.table[2].tolist() == [0, 3, -1, -1] and p.refs.tolist() == [2, 1, 1, 1, 0, 0]
    assert p.pool[0, :, 0].tolist() == [0, 1, 2, 1, 4, 5]
    p.truncate([2, 0, 9])                                            # seq 0 now ends inside the shared page
    assert p.refs.tolist() == [2, 0, 0, 1, 0, 0] and p.lengths.tolist() == [2, 0, 5]
    assert p.extend([17, 0, 5]) == -1 and p.extend([3, 17, 0]) == -1
    assert p.extend([3, 16, 5]) == 1 and p.refs.tolist() == [2, 0, 0, 1, 0, 0]     # five pages wanted, four free
    assert p.extend([3, 0, 5]) == 0                                  # copy on write: page 0 -> 1
    assert p.table[0].tolist() == [1, -1, -1, -1] and p.refs.tolist() == [1, 1, 0, 1, 0, 0]
    assert p.pool[0, 1, 0] == 0
    p.compact()                                                      # three live: page 3 -> 2
    assert p.table[2].tolist() == [0, 2, -1, -1] and p.refs.tolist() == [1, 1, 1, 0, 0, 0] and p.pool[0, 2, 0] == 1
    assert p.fork([0, 0], [1, 1]) == -1 and p.fork([0], [2]) == -1 and p.fork([0], [3]) == -1


def test_head_norm_by_hand():
    """3 and 4 of a head of four: mean square 25 / 4; weights and what is added to them multiply; zeros stay."""
    x = np.zeros((1, 2, 4), np.float16)
    x[0, 0, :2] = 3, 4
    assert np.allclose(paged.head_norm(x, eps=0.0 + 1e-300)[0, 0], [1.2, 1.6, 0, 0])
    assert np.allclose(paged.head_norm(x, [1, 0.5, 1, 1], 1e-300, 1.0)[0, 0], [2.4, 2.4, 0, 0])
    assert np.allclose(paged.head_norm(x, None, 6.25 * 3)[0, 0], [0.6, 0.8, 0, 0]) and not paged.head_norm(x)[0, 1].any()


def test_first_tokens_by_hand():
    """Five tokens, a window of one, two first ones: the last row averages tokens 0, 1 and 4, the second 0 and 1, once."""
    q = np.zeros((5, 1, 64), np.float16)
    k = np.zeros((1, 1, 8, 64), np.float16)
    v = np.zeros((1, 1, 8, 64), np.float16)
    v[0, 0, :5, 0] = 1, 2, 4, 8, 16
    o, lse, _, _ = paged.attention(q, k, v, np.array([[0]]), [5], [0, 5], 1.0, window=1, sinks=2)
    assert np.allclose(o[:, 0, 0], [1, 1.5, 7 / 3, 11 / 3, 19 / 3]) and np.allclose(np.exp(lse[:, 0]), [1, 2, 3, 3, 3])
