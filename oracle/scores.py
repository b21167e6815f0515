"""Oracle of the log probabilities: one row after the other in double precision.
Test infrastructure (see the package docstring); shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np


def order(x):
    """Tokens of a row from the largest logit down, the lower one first among equals; NaN counts as -inf."""
    y = [-math.inf if math.isnan(v) else float(v) for v in x]
    return sorted(range(len(y)), key=lambda i: (-y[i], i))


def row(x, tokens, top, temperature=1.0):
    """(logprobs of tokens, entropy, top ids, top logprobs) of one row of logits."""
    x = np.asarray(x, np.float64)
    ids = order(x)[:top]
    if np.isnan(x).any() or np.isposinf(x).any():
        lp = np.full(len(x), np.nan)
        return [lp[t] if 0 <= t < len(x) else -np.inf for t in tokens], np.nan, ids, [np.nan] * len(ids)
    m = x.max()
    if np.isneginf(m):
        return [-np.inf] * len(tokens), 0.0, ids, [-np.inf] * len(ids)
    lp = (x - m) / temperature
    lp = lp - math.log(np.exp(lp).sum())
    p, live = np.exp(lp), lp > -np.inf
    entropy = -float((p[live] * lp[live]).sum())
    return [lp[t] if 0 <= t < len(x) else -np.inf for t in tokens], entropy, ids, [lp[i] for i in ids]


def bounds(x, temperature=1.0):
    """Forward error of a row's (log probability per unit of 1 + |z - z_max|, entropy) in fp32: a power is off by 2^-22
    and 2^-22 of its exponent, a sum by 64 roundings in a chain, 2^-18, whatever the row's length (longer sums
    are made of such pieces, added up with what the additions round off), the logarithm by 2^-22 of itself."""
    x = np.asarray(x, np.float64)
    live = x[np.isfinite(x)]
    if not len(live) or np.isnan(x).any() or np.isposinf(x).any():
        return 0.0, 0.0
    z = (live - live.max()) / temperature
    p = np.exp(z)
    s = p.sum()
    p /= s
    first, second = float((p * -z).sum()), float((p * z * z).sum())
    log = 2.0 ** -17 + 2.0 ** -21 * first + 2.0 ** -22 * abs(math.log(s))
    return log, log + 2.0 ** -17 * first + 2.0 ** -21 * (first + second)
