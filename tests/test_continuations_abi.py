"""What the entry points for continuations of one prompt refuse, before anything is launched (no GPU: every
call here with fake pointers fails validation or is a no-op), and the binding's own checks of tensors."""
import pytest
import torch

FAKE = 0x10000
BIG = 1 << 40


def _kv(w, **kw):
    d = dict(k=FAKE, v=FAKE, table=FAKE, lengths=FAKE, offsets=FAKE, B=2, table_width=10, n_pages=40, kv_heads=4,
             page=16, head_dim=128)
    d.update(kw)
    return w._KV.pack(*(x or 0 for x in d.values()))


KV_FAULTS = [(dict(page=12), "SHAPE"), (dict(head_dim=96), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(table_width=0), "SHAPE"),
             (dict(n_pages=0), "SHAPE"), (dict(kv_heads=0), "SHAPE"), (dict(table_width=1 << 27), "SHAPE"),
             (dict(n_pages=1 << 30), "SHAPE"), (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(table=None), "ARG"),
             (dict(lengths=None), "ARG"), (dict(offsets=None), "ARG"), (dict(k=FAKE + 8), "ALIGN"),
             (dict(v=FAKE + 2), "ALIGN"), (dict(table=FAKE + 2), "ALIGN"), (dict(offsets=FAKE + 1), "ALIGN")]


def norm_rope(w, kv=None, q=FAKE, k=FAKE, v=FAKE, qs=2560, ks=512, vs=512, n=8, heads=20, wq=FAKE, wk=None, eps=1e-6,
              pos=None, ph=FAKE, rot=128, flags=0, out=FAKE + 4096):
    return w.load().norm_rope_append(_kv(w) if kv is None else kv, q, k, v, qs, ks, vs, n, heads, wq, wk, eps, pos, ph,
                                     rot, 1.0, flags, out, None)


@pytest.mark.parametrize("kw,code", KV_FAULTS)
def test_cache_refusals(w4v_mod, kw, code):
    assert norm_rope(w4v_mod, kv=_kv(w4v_mod, **kw)) == getattr(w4v_mod, "ERR_" + code)


def test_norm_rope_refusals(w4v_mod):
    w = w4v_mod
    call = lambda **kw: norm_rope(w, **kw)  # noqa: E731
    assert w.load().norm_rope_append(None, FAKE, FAKE, FAKE, 2560, 512, 512, 8, 20, FAKE, FAKE, 1e-6, None, FAKE, 128,
                                     1.0, 0, FAKE, None) == w.ERR_ARG
    assert call(rot=129) == call(rot=130) == call(rot=-2) == call(n=-1) == call(heads=0) == w.ERR_SHAPE
    assert call(qs=2558) == call(ks=504) == call(vs=516) == w.ERR_SHAPE
    assert call(flags=2) == call(flags=1) == call(flags=16) == w.ERR_ARG
    assert call(q=None) == call(k=None) == call(v=None) == call(out=None) == call(ph=None) == w.ERR_ARG
    assert call(eps=-1e-6) == call(eps=float("nan")) == call(eps=float("inf")) == w.ERR_ARG
    assert call(qs=5120, out=FAKE) == w.ERR_ARG                       # in place needs dense rows
    assert call(q=FAKE + 2) == call(v=FAKE + 8) == call(ph=FAKE + 4) == call(pos=FAKE + 2) == w.ERR_ALIGN
    assert call(wq=FAKE + 2) == call(wk=FAKE + 8) == w.ERR_ALIGN
    assert call(n=0, q=None, out=None) == call(kv=_kv(w, B=0), q=None) == w.OK


def _tensors():
    h, i = torch.float16, torch.int32
    return dict(k=torch.zeros(4, 2, 16, 64, dtype=h), table=torch.zeros(2, 3, dtype=i), lens=torch.zeros(2, dtype=i),
                offs=torch.zeros(3, dtype=i), q=torch.zeros(5, 4, 64, dtype=h), kn=torch.zeros(5, 2, 64, dtype=h))


def _code(w, f, *a, **kw):
    with pytest.raises(w.W4VError) as e:
        f(*a, **kw)
    return e.value.code


def test_binding_refuses_norm_tensors(w4v_mod):
    w, t = w4v_mod, _tensors()
    rope, norm, cache = w.Rope(64, device="cpu"), w.HeadNorm(), (t["k"], t["k"], t["table"], t["lens"], t["offs"])
    code = lambda *a, **kw: _code(w, w.norm_rope_append, *a, **kw)  # noqa: E731
    q, kn = t["q"], t["kn"]
    assert code(q, kn, kn[:4], *cache, rope, norm) == code(q[0], kn, kn, *cache, rope, norm) == w.ERR_SHAPE
    assert code(q, kn.float(), kn, *cache, rope, norm) == w.ERR_ARG
    assert code(q, kn, kn, *cache, rope, norm, positions=torch.zeros(5)) == w.ERR_ARG
    assert code(q, kn, kn, *cache, rope, w.HeadNorm(torch.zeros(32, dtype=torch.float16))) == w.ERR_SHAPE
    assert code(q, kn, kn, *cache, rope, w.HeadNorm(None, torch.zeros(128, dtype=torch.float16))) == w.ERR_SHAPE
    assert code(q, kn, kn, *cache, rope, norm) == w.ERR_ARG            # tensors of the host
    assert _code(w, w.HeadNorm, torch.zeros(64)) == _code(w, w.HeadNorm, eps=-1.0) == w.ERR_ARG
    assert _code(w, w.HeadNorm, eps=float("nan")) == w.ERR_ARG
    assert _code(w, w.HeadNorm, torch.zeros(1, 64, dtype=torch.float16)) == w.ERR_SHAPE
    assert _code(w, w.HeadNorm, None, torch.zeros(128, dtype=torch.float16)[::2]) == w.ERR_ARG


def test_logprob_refusals(w4v_mod):
    w = w4v_mod

    def call(x=FAKE, stride=1000, M=2, V=1000, t=FAKE, n=1, heat=1.0, lp=FAKE, h=None, top=3, ids=FAKE, tops=FAKE, flags=0):
        return w.load().token_logprobs(x, stride, M, V, t, n, heat, lp, h, top, ids, tops, flags, None)
    assert call(M=-1) == call(M=(1 << 24) + 1) == call(V=0) == call(V=(1 << 28) + 1, stride=1 << 30) == w.ERR_SHAPE
    assert call(n=-1) == call(n=(1 << 20) + 1) == call(top=-1) == call(top=33) == call(top=3, V=2) == w.ERR_SHAPE
    assert call(stride=999) == call(stride=0) == call(stride=1 << 38) == w.ERR_SHAPE
    for heat in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert call(heat=heat) == w.ERR_ARG
    assert call(flags=1) == call(flags=8) == call(flags=32) == w.ERR_ARG
    assert call(x=None) == call(t=None) == call(lp=None) == call(ids=None) == call(tops=None) == w.ERR_ARG
    assert call(x=FAKE + 2) == call(x=FAKE + 1, flags=16) == call(t=FAKE + 2) == call(lp=FAKE + 1) == w.ERR_ALIGN
    assert call(h=FAKE + 2) == call(ids=FAKE + 2) == call(tops=FAKE + 3) == w.ERR_ALIGN
    assert call(M=0, x=None, t=None, lp=None, ids=None, tops=None) == w.OK


def test_binding_refuses_logprob_tensors(w4v_mod):
    w, i = w4v_mod, torch.int32
    x, t = torch.zeros(3, 50), torch.zeros(3, 2, dtype=i)
    code = lambda *a, **kw: _code(w, w.token_logprobs, *a, **kw)  # noqa: E731
    out = lambda top: (torch.zeros(3, 2), torch.zeros(3), torch.zeros(3, top, dtype=i), torch.zeros(3, top))  # noqa: E731
    assert code(x[0], t) == code(x, t[:2]) == code(x, t[None]) == code(x, t, top=33) == code(x, t, top=-1) == w.ERR_SHAPE
    assert code(x.double(), t) == code(x.t().contiguous().t(), t) == code(x, t.long()) == code(x, t.t().contiguous().t()) == w.ERR_ARG
    assert code(x, t) == code(x, t, top=3, out=out(3)) == w.ERR_ARG      # tensors of the host


def test_sinks_refusals(w4v_mod):
    w = w4v_mod

    def call(kv=None, q=FAKE, stride=2560, n=8, heads=20, scale=0.1, window=9, sinks=4, out=FAKE, lse=None, ws=FAKE,
             nb=BIG, flags=0):
        return w.load().paged_attn_sinks(_kv(w) if kv is None else kv, q, stride, n, heads, scale, window, sinks, out, lse,
                                         ws, nb, flags, None)
    for kw, code in KV_FAULTS:
        assert call(kv=_kv(w, **kw)) == getattr(w, "ERR_" + code)
    assert w.load().paged_attn_sinks(None, FAKE, 2560, 8, 20, 0.1, 9, 4, FAKE, None, FAKE, BIG, 0, None) == w.ERR_ARG
    assert call(sinks=-1) == call(window=-1) == call(n=-1) == call(heads=18) == call(stride=2552) == w.ERR_SHAPE
    assert call(flags=4) == call(scale=0.0) == call(q=None) == call(out=None) == w.ERR_ARG
    assert call(q=FAKE + 8) == call(out=FAKE + 2) == call(lse=FAKE + 2) == call(ws=FAKE + 4) == w.ERR_ALIGN
    assert call(ws=None) == call(nb=16) == call(nb=16, flags=2) == w.ERR_WORKSPACE
    assert call(n=0, q=None, out=None, ws=None) == call(kv=_kv(w, B=0), q=None, ws=None) == w.OK
    t = _tensors()
    with pytest.raises(w.W4VError) as e:
        w.paged_attn(t["q"], t["k"], t["k"], t["table"], t["lens"], t["offs"], window=4, sinks=-1,
                     out=torch.zeros_like(t["q"]), ws=torch.zeros(1 << 24, dtype=torch.uint8), stream=0)
    assert e.value.code == w.ERR_SHAPE


def test_shared_refusals(w4v_mod):
    w = w4v_mod

    def call(kv=None, q=FAKE, stride=2560, n=8, heads=20, scale=0.1, g=FAKE, p=FAKE, G=2, out=FAKE, lse=None, ws=FAKE, nb=BIG,
             flags=0):
        return w.load().paged_attn_shared(_kv(w) if kv is None else kv, q, stride, n, heads, scale, g, p, G, out, lse, ws, nb,
                                          flags, None)
    for kw, code in KV_FAULTS:
        assert call(kv=_kv(w, **kw)) == getattr(w, "ERR_" + code)
    assert w.load().paged_attn_shared(None, FAKE, 2560, 8, 20, 0.1, FAKE, FAKE, 1, FAKE, None, FAKE, BIG, 0, None) == w.ERR_ARG
    assert call(G=-1) == call(G=3) == call(n=-1) == call(heads=18) == call(stride=2552) == w.ERR_SHAPE
    assert call(flags=2) == call(flags=1) == call(scale=0.0) == call(scale=float("nan")) == w.ERR_ARG
    assert call(q=None) == call(out=None) == call(g=None) == call(p=None) == w.ERR_ARG
    assert call(q=FAKE + 8) == call(out=FAKE + 2) == call(lse=FAKE + 2) == call(ws=FAKE + 4) == w.ERR_ALIGN
    assert call(g=FAKE + 2) == call(p=FAKE + 1) == w.ERR_ALIGN
    size = w.paged_attn_shared_workspace_bytes
    assert call(ws=None) == call(nb=size(8, 2, 2, 20, 4, 128) - 1) == w.ERR_WORKSPACE
    assert call(n=0, q=None, out=None, ws=None) == call(kv=_kv(w, B=0), q=None, ws=None) == w.OK
    assert size(8, 2, 2, 20, 4, 128) >= 2 * 8 * 20 * (128 * 4 + 8) and size(9, 2, 2, 20, 4, 128) > size(8, 2, 2, 20, 4, 128)
    assert size(-1, 2, 2, 20, 4, 128) == size(8, 2, -1, 20, 4, 128) == size(8, 2, 2, 18, 4, 128) == size(8, 2, 2, 20, 4, 96) == 0


@pytest.mark.parametrize("row_tiles,code", [((1 << 31) // (133 * 64), "SHAPE"), ((1 << 31) // (133 * 64) - 2, "WORKSPACE")])
def test_shared_work_fits_32_bits(w4v_mod, row_tiles, code):
    # both passes' row tiles of 128 tokens (and one more each for the sequence and the group), 64 heads, 133 units a row tile
    w, half = w4v_mod, row_tiles // 2
    kv = _kv(w, B=1, table_width=128, page=128, kv_heads=64)
    n = 128 * half - (128 if code == "WORKSPACE" else 0)
    assert (2 * (n // 128 + 1) * 64 * 133 >= 1 << 31) == (code == "SHAPE")
    assert w.load().paged_attn_shared(kv, FAKE, 64 * 128, n, 64, 0.1, FAKE, FAKE, 1, FAKE, None, FAKE, 16, 0,
                                      None) == getattr(w, "ERR_" + code)


def test_binding_refuses_shared_tensors(w4v_mod):
    w, t, i = w4v_mod, _tensors(), torch.int32
    cache = (t["k"], t["k"], t["table"], t["lens"], t["offs"])
    code = lambda *a, **kw: _code(w, w.paged_attn_shared, *a, **kw)  # noqa: E731
    g, p = torch.zeros(2, dtype=i), torch.zeros(1, dtype=i)
    assert code(t["q"], *cache, g[:1], p) == code(t["q"], *cache, g, p[None]) == code(t["q"][0], *cache, g, p) == w.ERR_SHAPE
    assert code(t["q"], *cache, g.long(), p) == code(t["q"], *cache, g, p.float()) == code(t["q"].float(), *cache, g, p) == w.ERR_ARG
    assert code(t["q"], *cache, g, p, lse=torch.zeros(5, 3)) == w.ERR_SHAPE
    assert code(t["q"], *cache, g, p) == w.ERR_ARG                       # tensors of the host
