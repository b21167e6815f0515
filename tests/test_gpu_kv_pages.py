"""kv_extend, kv_truncate, kv_fork, kv_compact and kv_copy on the GPU against
the oracle, value for value (page ids, counts and copied contents are exact)."""
import numpy as np
import pytest
import torch

from helpers import to_dev
from oracle import paged

pytestmark = pytest.mark.gpu


class Both:
    """One cache on the GPU and in the oracle; every step runs on both and compares all of it."""

    def __init__(self, w, gpu, n_pages, S, width, page, planes=3, seed=0, tail=(2, 8)):
        r = np.random.default_rng(seed)
        pool = r.standard_normal((planes, n_pages, tail[0], page, tail[1])).astype(np.float16)
        self.w, self.page = w, page
        self.o = paged.Pool(pool, np.zeros(n_pages, np.int32), np.full((S, width), -1, np.int32),
                            np.zeros(S, np.int32), page)
        self.pool, self.refs, self.table, self.lengths = (to_dev(a, gpu) for a in
                                                          (pool, self.o.refs, self.o.table, self.o.lengths))
        self.ws = w.workspace(w.kv_workspace_bytes(n_pages, S))
        self.dev = lambda a: to_dev(np.asarray(a, np.int32), gpu)

    def same(self, short=None, want=0):
        torch.cuda.synchronize()
        if short is not None:
            assert int(short.cpu()[0]) == want
        for a, b in ((self.refs, self.o.refs), (self.table, self.o.table), (self.lengths, self.o.lengths),
                     (self.pool, self.o.pool)):
            assert np.array_equal(a.cpu().numpy(), b)
        assert self.w.get_status() == self.w.OK

    def state(self):
        return self.pool, self.refs, self.table, self.lengths

    def extend(self, want):
        self.same(self.w.kv_extend(*self.state(), self.dev(want), ws=self.ws), self.o.extend(want))

    def truncate(self, want):
        self.w.kv_truncate(self.refs, self.table, self.lengths, self.dev(want), self.page)
        self.o.truncate(want)
        self.same()

    def fork(self, parents, children):
        short = self.w.kv_fork(*self.state(), self.dev(parents), self.dev(children), ws=self.ws)
        self.same(short, self.o.fork(list(parents), list(children)))

    def compact(self):
        self.w.kv_compact(*self.state(), ws=self.ws)
        self.o.compact()
        self.same()


@pytest.mark.parametrize("page,n_pages,S", [(8, 60, 5), (16, 5000, 40), (64, 33, 3), (256, 12, 2)])
def test_random_histories(w4v_mod, gpu, page, n_pages, S):
    """Long random runs of all calls, shortages and sharing among them."""
    r = np.random.default_rng([page, S])
    b = Both(w4v_mod, gpu, n_pages, S, max(4, 3 * n_pages // S), page, seed=page)
    top = min(b.o.table.shape[1], 2 * n_pages // S + 1) * page
    for _ in range(40):
        kind = r.integers(0, 5)
        if kind <= 1:
            b.extend(np.where(r.random(S) < 0.5, r.integers(0, top + 1, S), b.o.lengths + r.integers(0, 22, S)))
        elif kind == 2:
            b.truncate(b.o.lengths - np.where(r.random(S) < 0.4, r.integers(0, top, S), r.integers(-2, 5, S)))
        elif kind == 3:
            free = [s for s in range(S) if b.o.lengths[s] == 0]
            used = [s for s in range(S) if b.o.lengths[s] > 0]
            if free and used:
                b.fork(r.choice(used, len(free)), free)
        else:
            b.compact()


def test_shared_last_pages_are_copied_before_they_grow(w4v_mod, gpu):
    """Four holders of one page that a rollback left partly filled: all but the last take a copy."""
    b = Both(w4v_mod, gpu, 40, 5, 6, 16)
    b.extend([32, 0, 0, 0, 7])
    b.fork([0, 0, 0], [1, 2, 3])
    b.truncate([20, 20, 20, 20, 7])
    b.extend([21, 20, 40, 21, 7])                      # sequence 1 stays: three holders grow, all take copies
    b.extend([21, 21, 40, 21, 8])                      # now it is alone
    b.truncate([0] * 5)
    assert not b.o.refs.any()


def test_shortages_change_nothing(w4v_mod, gpu):
    b = Both(w4v_mod, gpu, 8, 4, 20, 8)
    b.extend([30, 17, 0, 0])                           # 4 + 3 pages
    b.extend([40, 25, 0, 0])                           # two wanted, one free
    b.fork([0, 1], [2, 3])                             # two partial pages, one free
    b.extend([30, 17, 161, 0])                         # longer than a table row
    b.fork([0], [1])
    b.fork([0, 0], [2, 2])
    b.fork([0, 2], [2, 3])                             # a child as parent
    b.fork([0, 9], [2, 3])
    b.fork([0, 1], [2, -1])
    b.fork([], [])
    b.fork([1], [2])
    # a shared partial page, and no page left for its copy
    b.truncate([30, 8 + 3, 8 + 3, 0])
    b.extend([30, 17, 11, 0])
    b.truncate([30, 17, 11, -4])


def test_enough_pages_for_several_rounds_of_the_scan(w4v_mod, gpu):
    b = Both(w4v_mod, gpu, 20000, 1500, 40, 8, planes=1, tail=(1, 8))
    r = np.random.default_rng(1)
    b.extend(r.integers(0, 90, 1500))
    b.truncate(np.where(r.random(1500) < 0.5, 0, b.o.lengths))
    b.compact()
    b.extend(b.o.lengths + 16)
    b.extend(np.full(1500, 310))                       # 58500 pages wanted


def test_compaction_into_other_arrays(w4v_mod, gpu):
    """With arrays of its own for the results the old tables stay, and what they point at."""
    b = Both(w4v_mod, gpu, 100, 6, 12, 16)
    b.extend([100, 50, 170, 3, 0, 60])
    b.truncate([0, 50, 170, 0, 0, 60])
    before = [x.clone() for x in b.state()]
    held = before[1] > 0
    refs, table = torch.full_like(b.refs, 77), torch.full_like(b.table, 77)
    b.w.kv_compact(*b.state(), refs_out=refs, table_out=table, ws=b.ws)
    b.o.compact()
    torch.cuda.synchronize()
    assert torch.equal(b.refs, before[1]) and torch.equal(b.table, before[2])
    assert np.array_equal(refs.cpu().numpy(), b.o.refs) and np.array_equal(table.cpu().numpy(), b.o.table)
    assert np.array_equal(b.pool.cpu().numpy(), b.o.pool)
    assert torch.equal(b.pool[:, held], before[0][:, held])


@pytest.mark.parametrize("tail,page", [((1, 8), 8), ((4, 128), 16), ((3, 64), 256), ((5, 72), 8)])
def test_copies(w4v_mod, gpu, tail, page):
    """Page sizes below, at and above the copy's own pieces; pairs with ids outside the pool are skipped."""
    b = Both(w4v_mod, gpu, 30, 1, 4, page, planes=5, tail=tail)
    src, dst = [3, 29, -1, 4, 30, 7], [0, 1, 2, -3, 5, 28]
    w4v_mod.kv_copy(b.pool, b.dev(src), b.dev(dst))
    for a, z in ((3, 0), (29, 1), (7, 28)):
        b.o.copy(a, z)
    b.same()
    w4v_mod.kv_copy(b.pool, b.dev([]), b.dev([]))
    b.same()


def test_no_pool(w4v_mod, gpu):
    """kv_truncate takes no pool; a big cache's offsets pass 32 bits (2.5 GB of one plane's pages)."""
    n = 80000
    pool = torch.zeros((1, n, 1, 128, 128), dtype=torch.float16, device=gpu)
    pool[0, n - 1], pool[0, 7] = 2.0, 3.0
    w4v_mod.kv_copy(pool, torch.tensor([n - 1, 7], dtype=torch.int32, device=gpu),
                    torch.tensor([0, n - 2], dtype=torch.int32, device=gpu))
    assert torch.all(pool[0, 0] == 2.0) and torch.all(pool[0, n - 2] == 3.0) and not torch.any(pool[0, 1:7])


@pytest.mark.parametrize("fill", [0, 0x45])
def test_one_workspace_for_caches_of_different_sizes(w4v_mod, gpu, fill):
    """Two pools of other sizes, and calls on the first sequences of a batch alone, through one workspace
    that nothing clears: what a call leaves in it never looks like a mark to the next."""
    r = np.random.default_rng(20)
    a = Both(w4v_mod, gpu, 100, 64, 6, 16)
    b = Both(w4v_mod, gpu, 20, 4, 6, 16)
    c = Both(w4v_mod, gpu, 100, 32, 6, 16)
    ws = torch.full((w4v_mod.kv_workspace_bytes(100, 64),), fill, dtype=torch.uint8, device=gpu)
    for x in (a, b, c):
        x.ws = ws
    for _ in range(3):
        a.extend(r.integers(1, 24, 64))                # base holds page ranks where c has its marks
        c.extend([16 * 5, 16 + 7, *[0] * 30])
        c.fork([0, 1], [5, 31])
        a.compact()                                    # list holds page ids where b has its marks
        b.extend([20, 33, 0, 0])
        b.fork([0, 1], [2, 3])
        a.extend(np.where(r.random(64) < 0.5, 30, 0))
        b.truncate([10, 20, 10, 20])                   # last pages shared, partly filled
        b.extend([10, 25, 12, 20])                     # only two of the holders grow
        c.truncate([0, 16 + 3, *[0] * 3, 16 * 5 - 9, *[0] * 25, 16 + 3])
        a.fork([], [])
        c.extend([3, 16 + 3, *[0] * 3, 16 * 5, *[0] * 25, 16 + 7])
        for x in (a, b, c):
            x.truncate([0] * len(x.o.lengths))
            assert not x.o.refs.any()
