"""Inputs and error bounds of the paged cache's GPU tests."""
import numpy as np


def cache(rng, n_new, lengths, Hq, Hkv, D, page, spare=3, extra_width=2, stale=None):
    """A cache for the given new tokens and lengths, its pages without order, and the rows that go
    with it.  What no token of a sequence occupies holds `stale` (None: numbers as everywhere)."""
    lengths, n_new = np.asarray(lengths, np.int64), np.asarray(n_new, np.int64)
    need = -(-lengths // page)
    n_pages = int(need.sum()) + spare
    ids = rng.permutation(n_pages)
    table = np.full((len(lengths), int(need.max(initial=0)) + extra_width), -1, np.int32)
    k, v = (rng.standard_normal((n_pages, Hkv, page, D)).astype(np.float16) for _ in range(2))
    used = np.zeros((n_pages, page), bool)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        for i in range(c):
            used[ids[at + i], :min(page, lengths[b] - i * page)] = True
        at += c
    if stale is not None:
        mask = np.broadcast_to(~used[:, None, :, None], k.shape)
        k[mask], v[mask] = stale, stale
    n = int(n_new.sum())
    return dict(q=(rng.standard_normal((n, Hq, D)) * 1.5).astype(np.float16), k=k, v=v, table=table,
                lengths=lengths.astype(np.int32), offsets=np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32))


def attention_bounds(c, ref):
    """Forward error of every row against the oracle's (out, lse, mag, absdot): the weights are
    rounded to fp16 (2^-11), the result once more; scores are fp32 sums of D exact products, each
    step off by at most 2^-23 of the absolute sum (a factor of two over rounding to nearest, for an
    accumulator that truncates), and so are the sums over the keys; exp2 and the score's scaling
    add a few units of the score (2^-20 in all for scores below 2^6).  Returns (bound of out,
    bound of lse)."""
    o, lse, mag, absdot = ref
    eps = (c["q"].shape[2] + 8) * 2.0 ** -23 * absdot + 2.0 ** -20
    keys = c["table"].shape[1] * c["k"].shape[2] + 64
    rel = 2.0 ** -11 + 2 * eps + 2 * keys * 2.0 ** -23
    fin = np.isfinite(lse)
    lb = np.where(fin, eps + keys * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(fin, lse, 0)), 0)
    return 2.0 ** -11 * np.abs(o) + rel[..., None] * (1 + 2.0 ** -10) * mag + 2.0 ** -24, lb
