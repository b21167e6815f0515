"""Pins of the log probabilities' oracle by rows small enough to work by hand (no GPU)."""
import math

import numpy as np

from oracle import scores


def test_by_hand():
    """Probabilities 1/4, 1/2, 1/4: entropy 3/2 ln 2; at half the temperature 1/6, 2/3, 1/6."""
    x = [0.0, math.log(2.0), 0.0]
    lp, h, ids, tops = scores.row(x, [1, 0, -1, 3], 3)
    assert np.allclose(lp[:2], [math.log(0.5), math.log(0.25)]) and lp[2:] == [-math.inf] * 2
    assert math.isclose(h, 1.5 * math.log(2)) and ids == [1, 0, 2] and np.allclose(tops, np.log([0.5, 0.25, 0.25]))
    assert np.allclose(scores.row(x, [0, 1, 2], 0, 0.5)[0], np.log([1 / 6, 2 / 3, 1 / 6]))


def test_what_is_not_finite():
    lp, h, ids, tops = scores.row([-np.inf, 2.0, -np.inf], [0, 1], 3)
    assert lp == [-np.inf, 0.0] and h == 0.0 and ids == [1, 0, 2] and tops == [0.0, -np.inf, -np.inf]
    assert scores.row([-np.inf] * 2, [0, 5], 2) == ([-np.inf] * 2, 0.0, [0, 1], [-np.inf] * 2)
    lp, h, ids, tops = scores.row([1.0, np.nan, 3.0, -np.inf], [2, -1], 4)
    assert np.isnan(lp[0]) and lp[1] == -np.inf and np.isnan(h) and ids == [2, 0, 1, 3] and np.isnan(tops).all()
    lp, _, ids, _ = scores.row([1.0, np.inf], [0], 2)
    assert np.isnan(lp[0]) and ids == [1, 0]
    assert scores.order([-0.0, 0.0, np.nan]) == [0, 1, 2]
