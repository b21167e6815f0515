"""What the paged cache's entry points refuse, before anything is launched (no
GPU: every call here with fake pointers fails validation or is a no-op), and
the binding's own checks of tensors."""
import ctypes

import pytest
import torch

FAKE = 0x10000
BIG = 1 << 40


def _kv(w, **kw):
    d = dict(k=FAKE, v=FAKE, table=FAKE, lengths=FAKE, offsets=FAKE, B=2, table_width=10, n_pages=40, kv_heads=4,
             page=16, head_dim=128)
    d.update(kw)
    return w._KV.pack(*(x or 0 for x in d.values()))


def _pages(w, **kw):
    d = dict(pool=FAKE, refs=FAKE, table=FAKE, lengths=FAKE, page_bytes=4096, planes=2, n_pages=40, S=3,
             table_width=10, page=16)
    d.update(kw)
    return w._PAGES.pack(*(x or 0 for x in d.values()))


KV_FAULTS = [(dict(page=12), "SHAPE"), (dict(page=4), "SHAPE"), (dict(page=512), "SHAPE"),
             (dict(head_dim=96), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(table_width=0), "SHAPE"),
             (dict(n_pages=0), "SHAPE"), (dict(kv_heads=0), "SHAPE"), (dict(table_width=1 << 27), "SHAPE"),
             (dict(n_pages=1 << 30), "SHAPE"), (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(table=None), "ARG"),
             (dict(lengths=None), "ARG"), (dict(offsets=None), "ARG"), (dict(k=FAKE + 8), "ALIGN"),
             (dict(v=FAKE + 2), "ALIGN"), (dict(table=FAKE + 2), "ALIGN"), (dict(offsets=FAKE + 1), "ALIGN")]


@pytest.mark.parametrize("kw,code", KV_FAULTS)
def test_cache_refusals(w4v_mod, kw, code):
    lib, want = w4v_mod.load(), getattr(w4v_mod, "ERR_" + code)
    kv = _kv(w4v_mod, **kw)
    assert lib.paged_attn(kv, FAKE, 2560, 8, 20, 0.1, 0, FAKE, None, FAKE, BIG, 0, None) == want
    assert lib.rope_append(kv, FAKE, FAKE, FAKE, 2560, 512, 512, 8, 20, None, FAKE, 128, 1.0, 0, FAKE, None) == want


def test_attention_refusals(w4v_mod):
    lib, w = w4v_mod.load(), w4v_mod

    def call(kv=None, q=FAKE, stride=2560, n=8, heads=20, scale=0.1, window=0, out=FAKE, lse=None, ws=FAKE, nb=BIG,
             flags=0):
        return lib.paged_attn(_kv(w) if kv is None else kv, q, stride, n, heads, scale, window, out, lse, ws, nb,
                              flags, None)
    assert lib.paged_attn(None, FAKE, 2560, 8, 20, 0.1, 0, FAKE, None, FAKE, BIG, 0, None) == w.ERR_ARG
    assert call(n=-1) == call(heads=0) == call(heads=18) == call(window=-1) == w.ERR_SHAPE
    assert call(stride=2552) == call(stride=2564) == w.ERR_SHAPE
    assert call(kv=_kv(w, kv_heads=1), heads=129, stride=129 * 128) == w.ERR_SHAPE
    assert call(scale=0.0) == call(scale=-1.0) == call(scale=float("inf")) == call(scale=float("nan")) == w.ERR_ARG
    assert call(flags=1) == call(flags=4) == call(q=None) == call(out=None) == w.ERR_ARG
    assert call(q=FAKE + 8) == call(out=FAKE + 2) == call(lse=FAKE + 2) == call(ws=FAKE + 4) == w.ERR_ALIGN
    assert call(ws=None) == call(nb=16) == call(nb=16, flags=2) == w.ERR_WORKSPACE
    assert call(n=0, q=None, out=None, ws=None) == call(kv=_kv(w, B=0), q=None, ws=None) == w.OK


@pytest.mark.parametrize("row_tiles,code", [((1 << 31) // (133 * 64), "SHAPE"), ((1 << 31) // (133 * 64) - 1, "WORKSPACE")])
def test_attention_work_fits_32_bits(w4v_mod, row_tiles, code):
    # row tiles of 128 tokens, 64 heads, 128 key tiles and 5 units more a row tile: from 2^31 units on refused
    w = w4v_mod
    kv = _kv(w, B=1, table_width=128, page=128, kv_heads=64)
    n = 128 * row_tiles + (0 if code == "SHAPE" else -128)
    assert ((n // 128 + 1) * 64 * 133 >= 1 << 31) == (code == "SHAPE")
    assert w.load().paged_attn(kv, FAKE, 64 * 128, n, 64, 0.1, 0, FAKE, None, FAKE, 16, 0, None) == getattr(w, "ERR_" + code)


def test_attention_workspace_sizes(w4v_mod):
    size = w4v_mod.paged_attn_workspace_bytes
    assert size(16, 1, 20, 4, 128, 4096) > 0 and size(16, 1, 20, 4, 128, 4096, True) > 0
    assert size(8192, 1, 20, 4, 128, 8192) >= size(16, 1, 20, 4, 128, 8192)
    assert size(-1, 1, 20, 4, 128, 64) == size(1, -1, 20, 4, 128, 64) == size(1, 1, 18, 4, 128, 64) == 0
    assert size(1, 1, 20, 4, 100, 64) == size(1, 1, 129, 1, 64, 64) == size(1, 1, 20, 4, 128, -1) == 0


def test_rope_refusals(w4v_mod):
    lib, w = w4v_mod.load(), w4v_mod

    def call(q=FAKE, k=FAKE, v=FAKE, qs=2560, ks=512, vs=512, n=8, heads=20, pos=None, ph=FAKE, rot=128, flags=0,
             out=FAKE + 4096):
        return lib.rope_append(_kv(w), q, k, v, qs, ks, vs, n, heads, pos, ph, rot, 1.0, flags, out, None)
    assert lib.rope_append(None, FAKE, FAKE, FAKE, 2560, 512, 512, 8, 20, None, FAKE, 128, 1.0, 0, FAKE,
                           None) == w.ERR_ARG
    assert call(rot=129) == call(rot=130) == call(rot=-2) == call(n=-1) == call(heads=0) == w.ERR_SHAPE
    assert call(qs=2558) == call(ks=504) == call(vs=516) == w.ERR_SHAPE
    assert call(flags=2) == call(q=None) == call(k=None) == call(v=None) == call(out=None) == call(ph=None) == w.ERR_ARG
    assert call(qs=5120, out=FAKE) == w.ERR_ARG                       # in place needs dense rows
    assert call(q=FAKE + 2) == call(v=FAKE + 8) == call(ph=FAKE + 4) == call(pos=FAKE + 2) == w.ERR_ALIGN
    assert call(n=0, q=None, out=None) == w.OK


def test_phase_refusals(w4v_mod):
    lib, w = w4v_mod.load(), w4v_mod
    out, mul = (ctypes.c_uint64 * 128)(), ctypes.c_float()

    def call(rot=64, base=1e4, kind=0, params=(2.0, 0, 0, 0), o=out, m=mul):
        p = None if params is None else (ctypes.c_double * 4)(*params)
        return lib.rope_phases(rot, base, kind, p, o, ctypes.byref(m) if m is not None else None)
    assert call() == call(params=None) == w.OK
    assert call(rot=0) == call(rot=3) == call(rot=258) == call(base=1.0) == call(base=float("nan")) == w.ERR_SHAPE
    assert call(kind=1, params=(0.5, 0, 0, 0)) == call(kind=2, rot=2) == w.ERR_SHAPE
    assert call(kind=3, params=(2, 0, 32, 1)) == call(kind=3, params=(2, 100, 1, 32)) == w.ERR_SHAPE
    assert call(kind=4, params=(2, 4, 1, 100)) == call(kind=4, params=(2, 1, 4, 0)) == w.ERR_SHAPE
    assert call(kind=5) == call(kind=-1) == call(kind=1, params=None) == call(o=None) == call(m=None) == w.ERR_ARG


@pytest.mark.parametrize("kw,code", [(dict(n_pages=0), "SHAPE"), (dict(n_pages=1 << 25), "SHAPE"), (dict(S=-1), "SHAPE"),
                                     (dict(S=65536), "SHAPE"), (dict(page=24), "SHAPE"), (dict(table_width=0), "SHAPE"),
                                     (dict(table_width=1 << 28), "SHAPE"), (dict(refs=None), "ARG"),
                                     (dict(table=None), "ARG"), (dict(lengths=None), "ARG"),
                                     (dict(refs=FAKE + 2), "ALIGN"), (dict(lengths=FAKE + 1), "ALIGN")])
def test_page_refusals(w4v_mod, kw, code):
    lib, want, g = w4v_mod.load(), getattr(w4v_mod, "ERR_" + code), _pages(w4v_mod, **kw)
    assert lib.kv_extend(g, FAKE, FAKE, FAKE, BIG, None) == want
    assert lib.kv_truncate(g, FAKE, None) == want
    assert lib.kv_fork(g, FAKE, FAKE, 1, FAKE, FAKE, BIG, None) == want
    assert lib.kv_compact(g, FAKE, FAKE, FAKE, BIG, None) == want


def test_page_call_refusals(w4v_mod):
    lib, w = w4v_mod.load(), w4v_mod
    g = _pages(w)
    for bad, code in ((_pages(w, page_bytes=24), w.ERR_SHAPE), (_pages(w, planes=-1), w.ERR_SHAPE),
                      (_pages(w, pool=None), w.ERR_ARG), (_pages(w, pool=FAKE + 8), w.ERR_ALIGN), (None, w.ERR_ARG)):
        assert lib.kv_extend(bad, FAKE, FAKE, FAKE, BIG, None) == code
        assert lib.kv_fork(bad, FAKE, FAKE, 1, FAKE, FAKE, BIG, None) == code
        assert lib.kv_compact(bad, FAKE, FAKE, FAKE, BIG, None) == code
    assert lib.kv_truncate(None, FAKE, None) == w.ERR_ARG
    assert lib.kv_extend(g, None, FAKE, FAKE, BIG, None) == lib.kv_extend(g, FAKE, None, FAKE, BIG, None) == w.ERR_ARG
    assert lib.kv_extend(g, FAKE + 2, FAKE, FAKE, BIG, None) == lib.kv_extend(g, FAKE, FAKE, FAKE + 8, BIG,
                                                                              None) == w.ERR_ALIGN
    assert lib.kv_extend(g, FAKE, FAKE, None, BIG, None) == lib.kv_extend(g, FAKE, FAKE, FAKE, 64,
                                                                          None) == w.ERR_WORKSPACE
    assert lib.kv_truncate(g, None, None) == w.ERR_ARG and lib.kv_truncate(g, FAKE + 1, None) == w.ERR_ALIGN
    assert lib.kv_fork(g, FAKE, FAKE, 4, FAKE, FAKE, BIG, None) == lib.kv_fork(g, FAKE, FAKE, -1, FAKE, FAKE, BIG,
                                                                              None) == w.ERR_SHAPE
    assert lib.kv_fork(g, None, FAKE, 1, FAKE, FAKE, BIG, None) == lib.kv_fork(g, FAKE, FAKE, 1, None, FAKE, BIG,
                                                                              None) == w.ERR_ARG
    assert lib.kv_fork(g, FAKE, FAKE, 1, FAKE, FAKE, 64, None) == w.ERR_WORKSPACE
    assert lib.kv_compact(g, None, FAKE, FAKE, BIG, None) == lib.kv_compact(g, FAKE, None, FAKE, BIG, None) == w.ERR_ARG
    assert lib.kv_compact(g, FAKE, FAKE, None, BIG, None) == w.ERR_WORKSPACE
    empty = _pages(w, S=0, refs=None, table=None, lengths=None, pool=None)
    assert lib.kv_extend(empty, None, None, None, 0, None) == lib.kv_truncate(empty, None, None) == w.OK
    assert lib.kv_copy(FAKE, 2, 40, 4096, FAKE, FAKE, -1, None) == lib.kv_copy(FAKE, 0, 40, 4096, FAKE, FAKE, 1,
                                                                             None) == w.ERR_SHAPE
    assert lib.kv_copy(FAKE, 2, 40, 4090, FAKE, FAKE, 1, None) == lib.kv_copy(FAKE, 2, 40, 0, FAKE, FAKE, 1,
                                                                            None) == w.ERR_SHAPE
    assert lib.kv_copy(None, 2, 40, 4096, FAKE, FAKE, 1, None) == lib.kv_copy(FAKE, 2, 40, 4096, None, FAKE, 1,
                                                                            None) == w.ERR_ARG
    assert lib.kv_copy(FAKE + 8, 2, 40, 4096, FAKE, FAKE, 1, None) == w.ERR_ALIGN
    assert lib.kv_copy(None, 2, 40, 4096, None, None, 0, None) == w.OK
    assert w.kv_workspace_bytes(40, 3) >= 4 * 3 * 43 and w.kv_workspace_bytes(0, 3) == w.kv_workspace_bytes(4, -1) == 0


def test_binding_refuses_wrong_tensors(w4v_mod):
    """Types, shapes and strides that the C entries cannot see."""
    w = w4v_mod
    h, i = torch.float16, torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=h)
    table, lens, offs = torch.zeros(2, 3, dtype=i), torch.zeros(2, dtype=i), torch.zeros(3, dtype=i)
    q, kn = torch.zeros(5, 4, 64, dtype=h), torch.zeros(5, 2, 64, dtype=h)
    rope = w.Rope(64, device="cpu")

    def code(f, *a, **kw):
        with pytest.raises(w.W4VError) as e:
            f(*a, **kw)
        return e.value.code
    at = w.paged_attn
    assert code(at, q.float(), k, k, table, lens, offs) == w.ERR_ARG
    assert code(at, q, k, k.float(), table, lens, offs) == w.ERR_ARG
    assert code(at, q, k, k, table.long(), lens, offs) == w.ERR_ARG
    assert code(at, q, k, k[:2], table, lens, offs) == w.ERR_SHAPE
    assert code(at, q, k, k, table, lens, offs[:2]) == w.ERR_SHAPE
    assert code(at, q[:, :, :32], k, k, table, lens, offs) == w.ERR_SHAPE
    assert code(at, q.transpose(0, 1).contiguous().transpose(0, 1), k, k, table, lens, offs) == w.ERR_ARG
    assert code(at, q, k.transpose(0, 1).contiguous().transpose(0, 1), k, table, lens, offs) == w.ERR_ARG
    assert code(at, q, k, k, table, lens, offs, out=q[:3]) == w.ERR_SHAPE
    assert code(at, q, k, k, table, lens, offs, lse=torch.zeros(5, 4, dtype=h)) == w.ERR_ARG
    ra = w.rope_append
    assert code(ra, q, kn, kn[:4], k, k, table, lens, offs, rope) == w.ERR_SHAPE
    assert code(ra, q, kn.float(), kn, k, k, table, lens, offs, rope) == w.ERR_ARG
    assert code(ra, q, kn, kn, k, k, table, lens, offs, rope, positions=torch.zeros(5)) == w.ERR_ARG
    assert code(w.Rope, 64, scaling=("unknown", 2.0), device="cpu") == w.ERR_ARG
    assert code(w.Rope, 64, scaling=("yarn", 2.0), device="cpu") == w.ERR_ARG
    assert code(w.Rope, 63, device="cpu") == w.ERR_SHAPE
    pool, refs = torch.zeros(2, 4, 2, 16, 64, dtype=h), torch.zeros(4, dtype=i)
    assert code(w.kv_extend, pool, refs[:3], table, lens, lens) == w.ERR_SHAPE
    assert code(w.kv_extend, pool, refs, table, lens, lens.long()) == w.ERR_ARG
    assert code(w.kv_truncate, refs, table, lens, lens[:1], 16) == w.ERR_SHAPE
    assert code(w.kv_fork, pool, refs, table, lens, lens, lens[:1]) == w.ERR_SHAPE
    assert code(w.kv_compact, pool, refs, table, lens, refs_out=refs[:2]) == w.ERR_SHAPE
    assert code(w.kv_copy, pool[0], refs, refs) == w.ERR_SHAPE


@pytest.mark.parametrize("group", [1, 3, 5, 128])
def test_invariant_workspace_holds_every_part(w4v_mod, group):
    """One slot per row tile and 512 keys of its context (tables up to 16,384 tokens): enough for all ascending
    offsets, the fullest ones (a sequence for every row, full contexts) included."""
    import random
    rng = random.Random(group)
    tok = 128 // group
    for _ in range(300):
        B, Hkv, width = rng.randint(1, 40), rng.randint(1, 5), rng.randint(1, 16384)
        news = [rng.choice([0, 1, tok, tok + 1, rng.randint(0, 4 * tok)]) for _ in range(B)]
        n = sum(news) + rng.choice([0, 0, 3])
        slot = min(tok, max(n, 1)) * group * (64 * 4 + 8) + 16
        slots = (w4v_mod.paged_attn_workspace_bytes(n, B, Hkv * group, Hkv, 64, width, True) - 256) // slot
        assert Hkv * sum(-(-m // tok) for m in news) * -(-width // 512) <= slots
