"""paged_attn_shared on the GPU against the oracle (double precision), which attends every sequence over its
own pages.  Bounds: paged_helpers (joining the two results adds two weights of 2^-22 and a rounding of 2^-24
each, inside the bound's 2^-20)."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged
from paged_helpers import attention_bounds, cache

pytestmark = pytest.mark.gpu


def forked(rng, groups, prefix, n_new, tails, Hq, Hkv, D, page, poison=None, **kw):
    """A cache whose groups share their prefixes' whole pages; what is left of a prefix in a page of its own
    is copied.  poison: what the pages hold that are no longer in use, or None."""
    n_new = np.asarray(n_new)
    lead = np.repeat([g[0] for g in groups], [len(g) for g in groups])
    P = np.repeat(prefix, [len(g) for g in groups])
    lengths = np.asarray(tails) + n_new
    lengths[:len(P)] += P
    c = cache(rng, n_new, lengths, Hq, Hkv, D, page, **kw)
    for b, (a, p) in enumerate(zip(lead, P)):
        if a == b:
            continue
        whole = p // page
        old = c["table"][b, :whole].copy()
        c["table"][b, :whole] = c["table"][a, :whole]
        if poison is not None:
            c["k"][old] = c["v"][old] = poison
        if p % page:
            for x in ("k", "v"):
                c[x][c["table"][b, whole], :, :p % page] = c[x][c["table"][a, whole], :, :p % page]
    c["groups"] = np.array([g[0] for g in groups] + [groups[-1][-1] + 1], np.int32) if groups else np.zeros(1, np.int32)
    c["prefix"] = np.asarray(prefix, np.int32)
    return c


def run(w, gpu, c, scale=None, lse=True):
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    n, Hq, _ = c["q"].shape
    L = torch.full((n, Hq), 7.0, dtype=torch.float32, device=gpu) if lse else None
    out = torch.full(c["q"].shape, 9.0, dtype=torch.float16, device=gpu)
    w.paged_attn_shared(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["offsets"], d["groups"], d["prefix"],
                        scale=scale, out=out, lse=L)
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    return out.cpu().numpy(), L.cpu().numpy() if lse else None


def check(w, gpu, c, scale=None, table=None):
    s = c["q"].shape[2] ** -0.5 if scale is None else scale
    got, lse = run(w, gpu, c, scale)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"] if table is None else table, c["lengths"], c["offsets"], s)
    (o, l, _, _), (bo, bl) = ref, attention_bounds(c, ref)
    err = np.abs(got.astype(np.float64) - o)
    assert np.all(err <= bo), (float(np.max(err / bo)), np.unravel_index(np.argmax(err / bo), err.shape))
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(lse), ~fin)
    assert np.all(np.abs(lse[fin] - l[fin]) <= bl[fin]), float(np.max(np.abs(lse[fin] - l[fin]) / bl[fin]))


@pytest.mark.parametrize("D,page", [(64, 8), (128, 16), (128, 128), (256, 256), (64, 64)])
@pytest.mark.parametrize("prefix", [1, 7, 16, 127, 128, 129, 300, 513])
def test_prefixes_around_tiles_and_pages(w4v_mod, gpu, D, page, prefix):
    rng = np.random.default_rng([D, page, prefix])
    check(w4v_mod, gpu, forked(rng, [range(5)], [prefix], [1, 3, 0, 16, 2], [0, 10, 5, 200, 127], 4, 2, D, page))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (21, 3), (128, 1), (40, 2)])
def test_head_groups(w4v_mod, gpu, Hq, Hkv):
    rng = np.random.default_rng([Hq, Hkv])
    check(w4v_mod, gpu, forked(rng, [range(3), range(3, 7)], [200, 77], [2, 1, 0, 5, 1, 1, 30], [0, 30, 4, 5, 0, 260, 9],
                               Hq, Hkv, 64, 16))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefixes_and_many_continuations(w4v_mod, gpu, D):
    rng = np.random.default_rng(D)
    check(w4v_mod, gpu, forked(rng, [range(40)], [5003], [1] * 40, rng.integers(0, 300, 40), 4, 1, D, 16))
    check(w4v_mod, gpu, forked(rng, [range(2), range(2, 12)], [3000, 1500], [16] * 12, rng.integers(0, 200, 12), 6, 2, D, 64))


def test_many_groups(w4v_mod, gpu):
    """More groups and sequences than a warp has lanes, some without new tokens, sequences before and behind all groups."""
    rng = np.random.default_rng(3)
    sizes = rng.integers(1, 9, 90)
    edges = np.concatenate([[0], np.cumsum(sizes)])
    B = int(edges[-1]) + 6
    groups = [range(a, b) for a, b in zip(edges[:-1], edges[1:])]
    c = forked(rng, groups, rng.integers(1, 200, 90), rng.integers(0, 4, B), rng.integers(0, 40, B), 2, 1, 64, 8)
    check(w4v_mod, gpu, c)
    c["groups"], c["prefix"] = c["groups"][5:], c["prefix"][5:]          # the first five groups' sequences share nothing now
    check(w4v_mod, gpu, c)


@pytest.mark.parametrize("D,C", [(64, 400), (128, 900)])
def test_more_sequences_than_shared_memory_lists(w4v_mod, gpu, D, C):
    rng = np.random.default_rng(C)
    groups = [range(C // 2), range(C // 2, C)] + [range(b, b + 1) for b in range(C, C + C // 2)]
    B = C + C // 2
    c = forked(rng, groups, [130, 60] + [9] * (C // 2), rng.integers(0, 2, B), rng.integers(0, 30, B), 2, 1, D, 16)
    check(w4v_mod, gpu, c)


def test_long_runs_of_sequences_without_new_tokens(w4v_mod, gpu):
    """Requests that wait: a range's next sequence with something to do is more than a warp's lanes away."""
    rng = np.random.default_rng(13)
    n = np.zeros(300, np.int64)
    n[[0, 70, 71, 190, 299]] = 3, 1, 40, 2, 5
    c = forked(rng, [range(150), range(150, 300)], [300, 40], n, np.where(n > 0, 200, rng.integers(0, 20, 300)), 4, 1, 64, 16)
    check(w4v_mod, gpu, c)
    n[[0, 70, 71, 190]] = 0
    check(w4v_mod, gpu, forked(rng, [range(150), range(150, 300)], [30, 40], n, rng.integers(0, 9, 300), 4, 2, 128, 16))


def test_large_prefixes_side_by_side(w4v_mod, gpu):
    """Prefixes beyond what L2 keeps, with two row tiles each: their ranges are aligned.  What the pages hold repeats,
    so that a short oracle stands for the long prefix: m copies of every key add ln m to the log-sum-exp and change
    no average (the lse's bound takes the longer sums)."""
    rng = np.random.default_rng(14)
    m, page, D, Hkv = 513, 64, 256, 2
    c = forked(rng, [range(34), range(34, 68)], [page, page], [1] * 68, [0] * 68, 8, Hkv, D, page)
    wide = np.full((68, m + 2), -1, np.int32)
    wide[:, :m] = c["table"][:, :1]
    wide[:, m] = c["table"][:, 1]
    long = dict(c, table=wide, lengths=np.full(68, m * page + 1, np.int32), prefix=np.full(2, m * page, np.int32))
    assert 2 * m * page * Hkv * D * 4 > 64 << 20
    got, lse = run(w4v_mod, gpu, long)
    # the new token's own weight is 1 / m of what the short sequence gives it
    s = D ** -0.5
    for t in range(0, 68, 5):
        K = np.concatenate([c["k"][c["table"][t, 0]], c["k"][c["table"][t, 1]][:, :1]], 1).astype(np.float64)      # [Hkv][page + 1][D]
        Vv = np.concatenate([c["v"][c["table"][t, 0]], c["v"][c["table"][t, 1]][:, :1]], 1).astype(np.float64)
        for h in range(8):
            x = K[h // 4] @ c["q"][t, h].astype(np.float64) * s
            p = np.exp(x - x.max())
            p[:page] *= m
            o, want = p @ Vv[h // 4] / p.sum(), x.max() + np.log(p.sum())
            mag = p @ np.abs(Vv[h // 4]) / p.sum()
            absdot = (np.abs(K[h // 4]) @ np.abs(c["q"][t, h].astype(np.float64))).max() * s
            eps = (D + 8) * 2.0 ** -23 * absdot + 2.0 ** -20            # as attention_bounds, over the long table
            keys = wide.shape[1] * page + 64
            rel = 2.0 ** -11 + 2 * eps + 2 * keys * 2.0 ** -23
            assert np.all(np.abs(got[t, h] - o) <= 2.0 ** -11 * np.abs(o) + rel * (1 + 2.0 ** -10) * mag + 2.0 ** -24)
            assert abs(lse[t, h] - want) <= eps + keys * 2.0 ** -23 + 2.0 ** -22 * abs(want)


def test_a_prompt_chunk_behind_a_shared_prefix(w4v_mod, gpu):
    """Row tiles of many tokens, over the group's sequences and their own."""
    rng = np.random.default_rng(4)
    check(w4v_mod, gpu, forked(rng, [range(3)], [700], [300, 0, 150], [0, 10, 33], 4, 2, 128, 32))


def test_only_the_first_sequences_pages_hold_the_prefix(w4v_mod, gpu):
    """The other members' tables need no pages for it; what lies in the page that a prefix ends in is never used."""
    rng = np.random.default_rng(5)
    for prefix in (160, 170):
        c = forked(rng, [range(4)], [prefix], [1, 4, 16, 2], [0, 60, 5, 300], 4, 2, 128, 16, poison=np.nan)
        table = c["table"].copy()
        c["table"][1:, :prefix // 16] = -1
        for b in (1, 2, 3):
            if prefix % 16:                                # (their own copy of the prefix's end, as no one reads it)
                for x in ("k", "v"):
                    c[x][c["table"][b, prefix // 16], :, :prefix % 16] = np.nan
        ref = dict(c, k=c["k"].copy(), v=c["v"].copy())
        for b in (1, 2, 3):
            for x in ("k", "v"):
                ref[x][table[b, prefix // 16], :, :prefix % 16] = c[x][table[0, prefix // 16], :, :prefix % 16]
        got, lse = run(w4v_mod, gpu, c)
        want = paged.attention(c["q"], ref["k"], ref["v"], table, c["lengths"], c["offsets"], 128 ** -0.5)
        bo, bl = attention_bounds(c, want)
        assert np.all(np.abs(got - want[0]) <= bo) and np.all(np.abs(lse - want[1]) <= bl)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_lies_past_a_sequence_or_a_prefix_is_never_used(w4v_mod, gpu, D):
    rng = np.random.default_rng(6)
    check(w4v_mod, gpu, forked(rng, [range(4)], [203], [1, 5, 0, 17], [3, 130, 40, 0], 6, 2, D, 32, poison=np.nan, stale=np.nan))


@pytest.mark.parametrize("where", ["prefix", "own"])
def test_a_value_that_is_not_finite_reaches_those_that_see_it(w4v_mod, gpu, where):
    rng = np.random.default_rng(7)
    c = forked(rng, [range(3)], [150], [4, 4, 4], [10, 20, 30], 4, 2, 64, 16)
    j = 149 if where == "prefix" else 150 + 20 + 2          # of the second sequence: its third new token
    for b in range(3) if where == "prefix" else (1,):
        c["v"][c["table"][b, j // 16], :, j % 16, 3] = np.inf
    got, _ = run(w4v_mod, gpu, c)
    bad = ~np.isfinite(got[:, 0, 3].astype(np.float64))
    assert np.array_equal(bad, np.full(12, True) if where == "prefix" else np.isin(np.arange(12), [6, 7]))
    assert np.all(np.isfinite(np.delete(got, 3, axis=2)))


def test_sequences_that_cannot_share(w4v_mod, gpu):
    """A member with fewer tokens than the prefix before its new ones, a group whose first sequence is shorter, prefixes
    of 0 and below, no groups: their rows attend over their own pages."""
    rng = np.random.default_rng(8)
    c = forked(rng, [range(3), range(3, 5)], [100, 40], [2, 30, 5, 1, 1], [0, 0, 9, 4, 6], 4, 2, 64, 16)
    for prefix in ([120, 47], [100, 0], [-5, 40], [100, 1 << 30], [0, 0]):
        check(w4v_mod, gpu, dict(c, prefix=np.array(prefix, np.int32)))
    for lengths in ([102, 120, 114, 45, 47], [102, 130, 104, 41, 40], [99, 130, 114, 39, 47], [101, 129, 104, 45, 30]):
        check(w4v_mod, gpu, dict(c, lengths=np.array(lengths, np.int32)))
    check(w4v_mod, gpu, dict(c, groups=np.zeros(1, np.int32), prefix=np.zeros(0, np.int32)))
    for groups in ([0, 0, 5], [0, 3, 3], [3, 3, 3], [1, 3, 5], [5, 5, 5], [-4, 3, 90]):
        ok = dict(c, groups=np.array(groups, np.int32))
        ok["prefix"] = np.array([40, 40] if groups in ([0, 0, 5],) else [100, 40], np.int32)
        if groups == [0, 0, 5]:
            ok["prefix"][1] = 0                            # (all five have nothing in common)
        check(w4v_mod, gpu, ok)
    for groups in ([5, 0, 3], [3, 0, 5], [4, 2, 0]):       # decreasing: whoever is found to share has the prefix in common
        check(w4v_mod, gpu, dict(c, groups=np.array(groups, np.int32), prefix=np.array([0, 0], np.int32)))


def test_lengths_at_the_edge(w4v_mod, gpu):
    """Members of length 0 and with more new tokens than cached ones."""
    rng = np.random.default_rng(9)
    c = forked(rng, [range(4)], [50], [1, 6, 4, 1], [0, 0, 0, 3], 4, 2, 128, 16)
    c["lengths"] = np.array([51, 3, 0, 54], np.int32)
    got, lse = run(w4v_mod, gpu, c)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], 128 ** -0.5)
    o, l = ref[:2]
    assert np.all(got[~np.isfinite(l)] == 0) and np.array_equal(np.isneginf(lse), ~np.isfinite(l))
    assert np.all(np.abs(got - o) <= attention_bounds(c, ref)[0])


def test_rows_of_no_sequence_one_workspace_and_graph_replay(w4v_mod, gpu):
    """The same bits on every call; a captured call follows lengths, groups and prefixes that change; calls of other
    sizes may use the workspace in between; rows behind the last sequence stay as they are."""
    rng, w = np.random.default_rng(10), w4v_mod
    c = forked(rng, [range(4)], [500], [4] * 4, [100, 0, 30, 7], 8, 2, 128, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    q = torch.cat([d["q"], d["q"][:5]])
    ws = w.workspace(w.paged_attn_shared_workspace_bytes(21, 4, 1, 8, 2, 128))
    out, lse = torch.full_like(q, 3.0), torch.full((21, 8), 3.0, device=gpu)
    args = [d[x] for x in ("k", "v", "table", "lengths", "offsets", "groups", "prefix")]
    call = lambda: w.paged_attn_shared(q, *args, out=out, lse=lse, ws=ws)  # noqa: E731
    call()
    first = out.clone()
    small = w.paged_attn_shared(d["q"][:1], *args[:4], torch.tensor([0, 1, 1, 1, 1], dtype=torch.int32, device=gpu), *args[5:], ws=ws)
    for _ in range(3):
        out.fill_(3.0)
        call()
        assert torch.equal(out, first)
    assert torch.all(out[16:] == 3.0) and torch.all(lse[16:] == 3.0) and small.shape == (1, 8, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    lengths = [450, 504, 300, 511]
    d["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))
    d["groups"].copy_(torch.tensor([1, 3], dtype=torch.int32))
    d["prefix"].fill_(290)
    g.replay()
    torch.cuda.synchronize()
    assert w.get_status() == w.OK
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], lengths, c["offsets"], 128 ** -0.5)
    assert np.all(np.abs(out[:16].cpu().numpy() - ref[0]) <= attention_bounds(c, ref)[0])


def test_strided_rows_and_another_stream(w4v_mod, gpu):
    rng, w = np.random.default_rng(11), w4v_mod
    c = forked(rng, [range(3)], [220], [9, 20, 1], [3, 40, 0], 4, 2, 128, 16)
    want, _ = run(w, gpu, c, lse=False)
    wide = torch.full((30, 6, 128), float("nan"), dtype=torch.float16, device=gpu)
    wide[:, 1:5] = to_dev(c["q"], gpu)
    args = [to_dev(c[x], gpu) for x in ("k", "v", "table", "lengths", "offsets", "groups", "prefix")]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = w.paged_attn_shared(wide[:, 1:5], *args, stream=s)
    s.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)


def test_offsets_that_name_rows_again_and_again(w4v_mod, gpu):
    """More work than is counted in 32 bits: nothing is written, and the status says so."""
    w, rng = w4v_mod, np.random.default_rng(12)
    n, Hq, page, length = 32768, 128, 256, 1 << 21           # five times 32,768 row tiles of over 16,000 key tiles
    i32 = lambda x: to_dev(np.asarray(x, np.int32), gpu)  # noqa: E731
    table = torch.full((9, length // page), -1, dtype=torch.int32, device=gpu)
    k = torch.zeros((4, 1, page, 64), dtype=torch.float16, device=gpu)
    q = torch.zeros((n, Hq, 64), dtype=torch.float16, device=gpu)
    out = torch.full_like(q, 5.0)
    ws = w.workspace(w.paged_attn_shared_workspace_bytes(n, 9, 1, Hq, 1, 64))
    w.paged_attn_shared(q, k, k, table, i32([length] * 9), i32([0, n] * 5), i32([0, 9]), i32([0]), out=out, ws=ws)
    assert w.get_status() == w.ERR_SHAPE and w.get_status() == w.OK
    assert torch.all(out == 5.0)
    c = forked(rng, [range(2)], [40], [3, 1], [2, 5], 4, 2, 64, 16)
    d = {x: to_dev(a, gpu) for x, a in c.items()}
    got = w.paged_attn_shared(*(d[x] for x in ("q", "k", "v", "table", "lengths", "offsets", "groups", "prefix")), ws=ws)
    ref = paged.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["offsets"], 0.125)
    assert np.all(np.abs(got.cpu().numpy() - ref[0]) <= attention_bounds(c, ref)[0])
