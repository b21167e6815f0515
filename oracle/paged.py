"""Oracle of the paged key/value cache: rotary positions, attention of new
tokens over the pages, and the page bookkeeping, one element after the other
in double precision or in Python integers.  Test infrastructure (see the
package docstring); shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot: int, base: float = 10000.0, scaling=None):
    """(angle per position of each pair, factor of cos and sin) for the scalings of rope_phases."""
    kind = scaling[0] if scaling else "none"
    if kind == "ntk":
        base = base * scaling[1] ** (rot / (rot - 2))
    out, mul = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if kind == "linear":
            f /= scaling[1]
        elif kind == "yarn":
            factor, context = scaling[1], scaling[2]
            fast, slow = (list(scaling[3:]) + [32.0, 1.0][len(scaling) - 3:])
            edge = [rot * math.log(context / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (fast, slow)]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            share = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = share * f / factor + (1 - share) * f
            mul = 0.1 * math.log(factor) + 1
        elif kind == "banded":
            factor, low, high, context = scaling[1:]
            keep = min(max((context * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = (1 - keep) * f / factor + keep * f
        out.append(f)
    return np.array(out), mul


def rotate(x, positions, freqs, mul, interleaved):
    """x [n][heads][D] with its first 2 len(freqs) elements turned by the rows' positions."""
    y = x.astype(np.float64).copy()
    half = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(positions, np.float64) * f
        c, s = mul * np.cos(ang)[:, None], mul * np.sin(ang)[:, None]
        xa, xb = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        y[:, :, a], y[:, :, b] = xa * c - xb * s, xb * c + xa * s
    return y


def head_norm(x, weight=None, eps=1e-6, centre=0.0):
    """Every head of x [n][heads][D] over its root mean square, times weight + centre (weight None: as it is)."""
    y = x.astype(np.float64)
    for t in range(y.shape[0]):
        for h in range(y.shape[1]):
            y[t, h] /= math.sqrt(float(np.dot(y[t, h], y[t, h])) / y.shape[2] + eps)
    return y if weight is None else y * (np.asarray(weight, np.float64) + centre)


def token_places(lengths, offsets):
    """(sequence, position) of every new row, (-1, 0) for one that no sequence covers."""
    places = [(-1, 0)] * int(max(offsets))
    for b in range(len(lengths)):
        for t in range(offsets[b], offsets[b + 1]):
            places[t] = (b, int(lengths[b]) - int(offsets[b + 1]) + t)
    return places


def attention(q, k_cache, v_cache, table, lengths, offsets, scale, window=0, sinks=0):
    """(out, lse, mag, absdot) of every new row in double; what error bounds go by: mag is
    sum_j p_j |v_j|, absdot the largest scale sum_d |q_d k_jd| of a row's keys.  With a window the
    `sinks` first keys are visible too.  A row without a visible key, or of no sequence (which
    paged_attn leaves alone): zeros and -inf."""
    n, Hq, D = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, absdot = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for t, (b, pos) in enumerate(token_places(lengths, offsets)):
        lo = max(0, pos - window + 1) if window else 0
        if b < 0 or pos < lo or pos < 0:
            continue
        js = np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, pos + 1)])
        ids = table[b][js // page]
        K = k_cache[ids, :, js % page].astype(np.float64)        # [keys][Hkv][D]
        V = v_cache[ids, :, js % page].astype(np.float64)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            x = K[:, kh] @ q[t, h].astype(np.float64) * scale
            top = x.max()
            absdot[t, h] = (np.abs(K[:, kh]) @ np.abs(q[t, h].astype(np.float64))).max() * scale
            p = np.exp(x - top)
            out[t, h] = p @ V[:, kh] / p.sum()
            mag[t, h] = p @ np.abs(V[:, kh]) / p.sum()
            lse[t, h] = top + math.log(p.sum())
    return out, lse, mag, absdot


class Pool:
    """Pages, references and tables in Python; contents as one array [planes][n_pages][...]."""

    def __init__(self, pool, refs, table, lengths, page):
        self.pool, self.refs, self.table, self.lengths = (np.array(a).copy() for a in (pool, refs, table, lengths))
        self.page = page

    def count(self, tokens):
        return -(-int(tokens) // self.page)

    def free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def copy(self, src, dst):
        self.pool[:, dst] = self.pool[:, src]

    def extend(self, want):
        if any(int(w) > self.table.shape[1] * self.page for w, n in zip(want, self.lengths) if w > n):
            return -1
        refs, moves, need = self.refs.copy(), [], 0
        for s, w in enumerate(want):
            n = int(self.lengths[s])
            if w <= n:
                continue
            need += self.count(w) - self.count(n)
            if n % self.page and refs[self.table[s, n // self.page]] > 1:
                refs[self.table[s, n // self.page]] -= 1
                moves.append(s)
                need += 1
        free = self.free()
        if need > len(free):
            return need - len(free)
        self.refs = refs
        for s, w in enumerate(want):
            n = int(self.lengths[s])
            if w <= n:
                continue
            if s in moves:
                new = free.pop(0)
                self.copy(self.table[s, n // self.page], new)
                self.table[s, n // self.page], self.refs[new] = new, 1
            for i in range(self.count(n), self.count(w)):
                self.table[s, i] = free.pop(0)
                self.refs[self.table[s, i]] = 1
            self.lengths[s] = w
        return 0

    def truncate(self, want):
        for s, w in enumerate(want):
            w = max(int(w), 0)
            if w >= self.lengths[s]:
                continue
            for i in range(self.count(w), self.count(self.lengths[s])):
                self.refs[self.table[s, i]] -= 1
                self.table[s, i] = -1
            self.lengths[s] = w

    def fork(self, parents, children):
        S = len(self.lengths)
        if any(not 0 <= x < S for x in [*parents, *children]) or len(set(children)) < len(children) or \
                set(parents) & set(children) or any(self.lengths[c] for c in children):
            return -1
        free = self.free()
        need = sum(1 for a in parents if self.lengths[a] % self.page)
        if need > len(free):
            return need - len(free)
        for a, c in zip(parents, children):
            n = int(self.lengths[a])
            self.table[c] = -1
            for i in range(n // self.page):
                self.table[c, i] = self.table[a, i]
                self.refs[self.table[a, i]] += 1
            if n % self.page:
                new = free.pop(0)
                self.copy(self.table[a, n // self.page], new)
                self.table[c, n // self.page], self.refs[new] = new, 1
            self.lengths[c] = n
        return 0

    def compact(self):
        live = [i for i, r in enumerate(self.refs) if r > 0]
        holes = [i for i in self.free() if i < len(live)]
        to = dict(zip([i for i in live if i >= len(live)], holes))
        for a, z in to.items():
            self.copy(a, z)
            self.refs[z], self.refs[a] = self.refs[a], 0
        for s in range(len(self.lengths)):
            for i in range(self.count(self.lengths[s])):
                self.table[s, i] = to.get(int(self.table[s, i]), self.table[s, i])
