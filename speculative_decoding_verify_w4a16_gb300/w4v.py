"""Thin ctypes binding of libw4v (include/w4v.h): argument marshalling only.

Every step of the verify path runs in the library's CUDA kernels; this
module passes device pointers from torch tensors, the current stream, and
turns status codes into exceptions.  There is no fallback: if the library is
missing or the GPU is not sm_103, calls raise.

`stream=` takes a torch stream or a raw handle (default: the current stream).
Results and workspaces that the caller does not pass are then that stream's;
ordering the call after its inputs, and what reads its results after it, is
the caller's part.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct
import threading
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libw4v.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "w4v.h")

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_ARCH, ERR_CUDA, ERR_TIMEOUT = range(8)
GROUP = 128

_lock = threading.Lock()
_lib = None


class Problem(ctypes.Structure):
    """w4a16_problem (include/w4v.h)."""
    _fields_ = [("A", ctypes.c_void_p), ("Bq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("C", ctypes.c_void_p), ("N", ctypes.c_int), ("K", ctypes.c_int)]


class GroupedHandle(ctypes.Structure):
    """w4a16_grouped_t (include/w4v.h): filled by w4a16_grouped_plan."""
    _fields_ = [("plan", ctypes.c_void_p), ("units", ctypes.c_longlong), ("n_problems", ctypes.c_int),
                ("M", ctypes.c_int), ("group", ctypes.c_int), ("has_zeros", ctypes.c_int), ("tiles", ctypes.c_int),
                ("check", ctypes.c_uint)]


# w4v_kv_t and w4v_pages_t (include/w4v.h), packed per call: a ctypes structure
# takes several times as long to fill, next to kernels of a few microseconds.
_KV = struct.Struct("PPPPP6i")       # k, v, table, lengths, offsets, B, table_width, n_pages, kv_heads, page, head_dim
_PAGES = struct.Struct("PPPPN5i4x")  # pool, refs, table, lengths, page_bytes, planes, n_pages, S, table_width, page


class W4VError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (w4v status %d)" % (where, status_string(code), code))


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libw4v.so (built by ``_build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError("libw4v.so not built: run speculative_decoding_verify_w4a16_gb300._build.build()")
            lib = ctypes.CDLL(path)
            P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.w4v_status_string.argtypes = [I]
            lib.w4v_status_string.restype = ctypes.c_char_p
            lib.w4v_init.restype = I
            lib.w4v_get_status.argtypes = [P]
            lib.w4v_get_status.restype = I
            lib.w4v_packed_bytes.argtypes = [I, I]
            lib.w4v_packed_bytes.restype = S
            lib.w4v_pack_int4.argtypes = [P, I, I, P]
            lib.w4v_pack_int4.restype = I
            lib.w4v_unpack_int4.argtypes = [P, I, I, P]
            lib.w4v_unpack_int4.restype = I
            lib.w4a16_workspace_bytes.argtypes = [I, I, I]
            lib.w4a16_workspace_bytes.restype = S
            lib.w4a16_gemm.argtypes = [P, P, P, P, I, P, I, I, I, P, S, P]
            lib.w4a16_gemm.restype = I
            lib.w4a16_gemm_ex.argtypes = [P, P, P, P, I, P, I, I, I, P, S, ctypes.c_uint, P]
            lib.w4a16_gemm_ex.restype = I
            lib.w4a16_grouped_plan_bytes.argtypes = [I]
            lib.w4a16_grouped_plan_bytes.restype = S
            lib.w4a16_grouped_plan.argtypes = [P, I, I, I, P, S, P, P]
            lib.w4a16_grouped_plan.restype = I
            lib.w4a16_grouped_workspace_bytes.argtypes = [P]
            lib.w4a16_grouped_workspace_bytes.restype = S
            lib.w4a16_gemm_grouped.argtypes = [P, P, S, ctypes.c_uint, P]
            lib.w4a16_gemm_grouped.restype = I
            lib.w8_lmhead_argmax_workspace_bytes.argtypes = [I, I]
            lib.w8_lmhead_argmax_workspace_bytes.restype = S
            lib.w8_lmhead_argmax.argtypes = [P, P, P, I, I, I, P, P, P, P, S, P]
            lib.w8_lmhead_argmax.restype = I
            lib.w8_lmhead_argmax_ex.argtypes = [P, P, P, I, I, I, P, P, P, P, S, ctypes.c_uint, P]
            lib.w8_lmhead_argmax_ex.restype = I
            lib.w8_lmhead_argmax_accept_ex.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, S, ctypes.c_uint, P]
            lib.w8_lmhead_argmax_accept_ex.restype = I
            lib.spec_accept.argtypes = [P, P, I, I, P, P, P]
            lib.spec_accept.restype = I
            lib.w8_lmhead_argmax_accept.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, S, P]
            lib.w8_lmhead_argmax_accept.restype = I
            lib.ngram_draft_workspace_bytes.argtypes = [I]
            lib.ngram_draft_workspace_bytes.restype = S
            lib.ngram_draft.argtypes = [P, P, I, I, I, I, I, P, P, P, S, P]
            lib.ngram_draft.restype = I
            lib.gdn_verify.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P]
            lib.gdn_verify.restype = I
            lib.gdn_commit.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
            lib.gdn_commit.restype = I
            lib.gdn_step.argtypes = [P, P, P, P, P, P, I, P, P, P, P, P, I, I, I, I, I, P, P]
            lib.gdn_step.restype = I
            L, F, U = ctypes.c_longlong, ctypes.c_float, ctypes.c_uint
            lib.token_logprobs.argtypes = [P, L, I, I, P, I, F, P, P, I, P, P, U, P]
            lib.token_logprobs.restype = I
            lib.rope_append.argtypes = [P, P, P, P, L, L, L, I, I, P, P, I, F, U, P, P]
            lib.rope_append.restype = I
            lib.norm_rope_append.argtypes = [P, P, P, P, L, L, L, I, I, P, P, F, P, P, I, F, U, P, P]
            lib.norm_rope_append.restype = I
            lib.rope_phases.argtypes = [I, ctypes.c_double, I, P, P, P]
            lib.rope_phases.restype = I
            lib.paged_attn_workspace_bytes.argtypes = [I, I, I, I, I, I, U]
            lib.paged_attn_workspace_bytes.restype = S
            lib.paged_attn.argtypes = [P, P, L, I, I, F, I, P, P, P, S, U, P]
            lib.paged_attn.restype = I
            lib.paged_attn_sinks.argtypes = [P, P, L, I, I, F, I, I, P, P, P, S, U, P]
            lib.paged_attn_sinks.restype = I
            lib.paged_attn_shared_workspace_bytes.argtypes = [I, I, I, I, I, I]
            lib.paged_attn_shared_workspace_bytes.restype = S
            lib.paged_attn_shared.argtypes = [P, P, L, I, I, F, P, P, I, P, P, P, S, U, P]
            lib.paged_attn_shared.restype = I
            lib.kv_workspace_bytes.argtypes = [I, I]
            lib.kv_workspace_bytes.restype = S
            lib.kv_extend.argtypes = [P, P, P, P, S, P]
            lib.kv_extend.restype = I
            lib.kv_truncate.argtypes = [P, P, P]
            lib.kv_truncate.restype = I
            lib.kv_fork.argtypes = [P, P, P, I, P, P, S, P]
            lib.kv_fork.restype = I
            lib.kv_compact.argtypes = [P, P, P, P, S, P]
            lib.kv_compact.restype = I
            lib.kv_copy.argtypes = [P, I, I, S, P, P, I, P]
            lib.kv_copy.restype = I
            _lib = lib
    return _lib


def header_functions(path: str = HEADER):
    """Names of the functions declared in include/w4v.h."""
    with open(path) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b([A-Za-z_][A-Za-z0-9_]*)\s*\(", text)) -
                  {"if", "defined", "sizeof"})


def status_string(code: int) -> str:
    try:
        return load().w4v_status_string(int(code)).decode()
    except Exception:
        return "status %d" % code


def _check(code: int, where: str) -> None:
    if code != OK:
        raise W4VError(code, where)


_torch = None


def _stream(stream=None) -> Optional[int]:
    if stream is None:
        global _torch
        if _torch is None:
            import torch
            _torch = torch
        torch = _torch
        if torch.cuda.is_initialized():          # the raw handle: a Stream object costs more than a small call's checks
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _torch_stream(stream=None):
    """The torch stream of a call's `stream`: a torch stream, a raw handle, or None (the current one)."""
    import torch
    if stream is None:
        return torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        return stream
    handle = (stream.value if isinstance(stream, ctypes.c_void_p) else int(stream)) or 0
    # 0 and 1 (cudaStreamLegacy) both name the default stream
    return torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()


def _new(shape, dtype, device, stream=None, zero=False):
    """A result tensor of a call on `stream`.  Where one is given the tensor is that stream's own, so
    that its memory is not still in use by another stream's earlier work (and cleared in order); the
    current stream, where the caller is likely to read it, counts as a user too."""
    import torch
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream)):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def init() -> None:
    _check(load().w4v_init(), "w4v_init")


def get_status(stream=None) -> int:
    return load().w4v_get_status(_stream(stream))


# ------------------------------------------------------------------ packing --
def packed_bytes(N: int, K: int) -> int:
    return load().w4v_packed_bytes(N, K)


def pack_int4(q: np.ndarray) -> np.ndarray:
    """Logical codes uint8 [N][K] (0..15) -> the library's packed tile layout (host)."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    nbytes = packed_bytes(N, K)
    if nbytes == 0:
        raise W4VError(ERR_SHAPE, "w4v_pack_int4")
    out = np.empty(nbytes, np.uint8)
    _check(load().w4v_pack_int4(q.ctypes.data, N, K, out.ctypes.data), "w4v_pack_int4")
    return out


def unpack_int4(packed: np.ndarray, N: int, K: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    q = np.empty((N, K), np.uint8)
    _check(load().w4v_unpack_int4(packed.ctypes.data, N, K, q.ctypes.data), "w4v_unpack_int4")
    return q


# --------------------------------------------------------------- workspaces --
def w4a16_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().w4a16_workspace_bytes(M, N, K)


def w8_lmhead_argmax_workspace_bytes(M: int, V: int) -> int:
    return load().w8_lmhead_argmax_workspace_bytes(M, V)


def workspace(nbytes: int, device="cuda", stream=None):
    """A zero-filled device workspace (the library leaves it zeroed after each call), allocated and
    cleared on `stream` (default: the current one), in whose order it may be used and given up."""
    import torch
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return workspace(nbytes, device)
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ compute --
STATIC_WEIGHTS = 1
BATCH_INVARIANT = 2


def w4a16_gemm(A, Bq, scales, N: int, zeros=None, out=None, ws=None, stream=None, static_weights=False,
               group: int = GROUP, batch_invariant=False):
    """C = A @ deq(Bq, scales, zeros)^T on the GPU.  A fp16 [M][K] cuda, Bq packed uint8 cuda,
    scales fp16 [K/group][N] (group 128 or 32).
    static_weights: the caller promises no GPU work still in flight writes Bq, scales or zeros
    (w4a16_gemm_ex with W4V_STATIC_WEIGHTS).
    batch_invariant: for M > 32, 32-row blocks through the verify-sized kernel
    (W4V_BATCH_INVARIANT): each row equals the row computed alone."""
    import torch
    M, K = A.shape
    if out is None:
        out = _new((M, N), torch.float16, A.device, stream)
    if ws is None:
        ws = workspace(w4a16_workspace_bytes(M, N, K), A.device, stream)
    flags = (STATIC_WEIGHTS if static_weights else 0) | (BATCH_INVARIANT if batch_invariant else 0)
    code = load().w4a16_gemm_ex(_ptr(A), _ptr(Bq), _ptr(scales), _ptr(zeros), int(group), _ptr(out), M, N, K,
                                _ptr(ws), ws.numel(), flags, _stream(stream))
    _check(code, "w4a16_gemm")
    return out


class GroupedGemm:
    """Several independent W4A16 products in one launch (w4a16_grouped_plan +
    w4a16_gemm_grouped).  `problems` is a list of (A, Bq, scales, zeros, C)
    device tensors (zeros None or a uint8 table for every problem), all with
    the same number of rows M; the plan keeps them alive and refers to their
    addresses, so call it again with the same tensors (refill them in place)."""

    def __init__(self, problems, group: int = GROUP, stream=None):
        import torch
        lib = load()
        self.problems = list(problems)
        n = len(self.problems)
        M = self.problems[0][0].shape[0]
        dev = self.problems[0][0].device
        arr = (Problem * n)()
        for i, (A, Bq, sc, z, C) in enumerate(self.problems):
            arr[i] = Problem(_ptr(A), _ptr(Bq), _ptr(sc), _ptr(z), _ptr(C), int(C.shape[1]), int(A.shape[1]))
        nbytes = lib.w4a16_grouped_plan_bytes(n)
        # torch's allocations start on 512-byte boundaries (the plan needs 64)
        self.plan = _new(max(int(nbytes), 64), torch.uint8, dev, stream)
        self.handle = GroupedHandle()
        code = lib.w4a16_grouped_plan(arr, n, int(M), int(group), _ptr(self.plan), self.plan.numel(),
                                      ctypes.byref(self.handle), _stream(stream))
        _check(code, "w4a16_grouped_plan")
        self.ws = workspace(lib.w4a16_grouped_workspace_bytes(ctypes.byref(self.handle)), dev, stream)
        _torch_stream(stream).synchronize()                    # cleared: calls may run on any stream

    def __call__(self, stream=None, static_weights: bool = False, ws=None):
        ws = self.ws if ws is None else ws
        code = load().w4a16_gemm_grouped(ctypes.byref(self.handle), _ptr(ws), ws.numel(),
                                         STATIC_WEIGHTS if static_weights else 0, _stream(stream))
        _check(code, "w4a16_gemm_grouped")
        return [p[4] for p in self.problems]


def w8_lmhead_argmax(X, W, scale, out=None, maxlogit=None, logits=None, ws=None, stream=None,
                     batch_invariant=False):
    """Greedy token per row of X through the int8 lm_head; returns the int32 [M] token tensor.
    batch_invariant: for M > 32, blocks of 32 rows (W4V_BATCH_INVARIANT): each row's
    logits and token equal those of the row computed alone."""
    import torch
    M, K = X.shape
    V = W.shape[0]
    if out is None:
        out = _new(M, torch.int32, X.device, stream)
    if ws is None:
        ws = workspace(w8_lmhead_argmax_workspace_bytes(M, V), X.device, stream)
    code = load().w8_lmhead_argmax_ex(_ptr(X), _ptr(W), _ptr(scale), M, K, V, _ptr(out), _ptr(maxlogit),
                                      _ptr(logits), _ptr(ws), ws.numel(), BATCH_INVARIANT if batch_invariant else 0,
                                      _stream(stream))
    _check(code, "w8_lmhead_argmax")
    return out


def spec_accept(target, draft, n_out=None, tok_out=None, stream=None):
    """(n [B], tokens [B][K+1]) for int32 target [B][K+1] and drafts [B][K] on the GPU."""
    import torch
    B, K1 = target.shape
    K = K1 - 1
    if n_out is None:
        n_out = _new(B, torch.int32, target.device, stream)
    if tok_out is None:
        tok_out = _new((B, K1), torch.int32, target.device, stream)
    code = load().spec_accept(_ptr(target), _ptr(draft) if K > 0 else None, B, K, _ptr(n_out),
                              _ptr(tok_out), _stream(stream))
    _check(code, "spec_accept")
    return n_out, tok_out


def w8_lmhead_argmax_accept(X, W, scale, draft, out=None, n_out=None, tok_out=None, maxlogit=None, ws=None,
                            stream=None, batch_invariant=False):
    """lm_head argmax of the B*(n+1) rows of X and greedy acceptance of drafts [B][n] in one launch.
    Returns (tokens [B*(n+1)], n_accepted [B], emitted tokens [B][n+1])."""
    import torch
    M, K = X.shape
    V = W.shape[0]
    B, nd = draft.shape
    if out is None:
        out = _new(M, torch.int32, X.device, stream)
    if n_out is None:
        n_out = _new(B, torch.int32, X.device, stream)
    if tok_out is None:
        tok_out = _new((B, nd + 1), torch.int32, X.device, stream)
    if M != B * (nd + 1):
        raise W4VError(ERR_SHAPE, "w8_lmhead_argmax_accept")
    if ws is None:
        ws = workspace(w8_lmhead_argmax_workspace_bytes(M, V), X.device, stream)
    code = load().w8_lmhead_argmax_accept_ex(_ptr(X), _ptr(W), _ptr(scale), B, nd, K, V,
                                             _ptr(draft) if nd > 0 else None, _ptr(out), _ptr(n_out),
                                             _ptr(tok_out), _ptr(maxlogit), _ptr(ws), ws.numel(),
                                             BATCH_INVARIANT if batch_invariant else 0, _stream(stream))
    _check(code, "w8_lmhead_argmax_accept")
    return out, n_out, tok_out


def ngram_draft(context, lengths, n_min: int, n_max: int, K: int, out=None, match=None, ws=None, stream=None):
    """Prompt-lookup drafts on the GPU: context int32 [B][ld], lengths int32 [B] (cuda).
    Returns (drafts int32 [B][K], match length int32 [B])."""
    import torch
    B, ld = context.shape
    if out is None:
        out = _new((B, K), torch.int32, context.device, stream)
    if match is None:
        match = _new(B, torch.int32, context.device, stream)
    if ws is None:
        ws = workspace(load().ngram_draft_workspace_bytes(B), context.device, stream)
    code = load().ngram_draft(_ptr(context), _ptr(lengths), B, ld, int(n_min), int(n_max), int(K),
                              _ptr(out) if K > 0 else None, _ptr(match), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "ngram_draft")
    return out, match


def gdn_verify(state, q, k, v, alpha, beta, out=None, stream=None):
    """Outputs o [B][T][H][dv] (fp16) of the gated delta recurrence over a verify block,
    from the committed fp32 state [B][H][dv][dk]; the state is not written."""
    import torch
    B, H, dv, dk = state.shape
    T = q.shape[1]
    if out is None:
        out = _new((B, T, H, dv), torch.float16, state.device, stream)
    code = load().gdn_verify(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), B, T, H, dk, dv,
                             _ptr(out), _stream(stream))
    _check(code, "gdn_verify")
    return out


def gdn_step(state, prev, q, k, v, alpha, beta, out=None, stream=None):
    """Commit the previous block into the fp32 state (prev = (k, v, alpha, beta,
    n_accepted) of that block, or None) and return the outputs o [B][T][H][dv]
    of the current block from the state just committed; one launch."""
    import torch
    B, H, dv, dk = state.shape
    T = q.shape[1]
    if out is None:
        out = _new((B, T, H, dv), torch.float16, state.device, stream)
    if prev is None:
        kp = vp = ap = bp = n = None
        T_prev = 0
    else:
        kp, vp, ap, bp, n = prev
        T_prev = kp.shape[1]
    code = load().gdn_step(_ptr(state), _ptr(kp), _ptr(vp), _ptr(ap), _ptr(bp), _ptr(n), T_prev, _ptr(q), _ptr(k),
                           _ptr(v), _ptr(alpha), _ptr(beta), B, T, H, dk, dv, _ptr(out), _stream(stream))
    _check(code, "gdn_step")
    return out


def gdn_commit(state, k, v, alpha, beta, n_accepted, stream=None):
    """Advance the committed state in place by positions 0..n_accepted[b] of the block."""
    B, H, dv, dk = state.shape
    T = k.shape[1]
    code = load().gdn_commit(_ptr(state), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(n_accepted), B, T, H,
                             dk, dv, _stream(stream))
    _check(code, "gdn_commit")
    return state


# ---------------------------------------------------------------- paged cache --
ROPE_INTERLEAVED = 4
NORM_ZERO_CENTRED = 8
ROPE_SCALINGS = {"linear": (1, 1), "ntk": (2, 1), "yarn": (3, 4), "banded": (4, 4)}


class Rope:
    """Rotary positions of `rot` elements a head (rope_phases): the phase table on
    the device and the factor of cos and sin.  scaling: None, ("linear", factor),
    ("ntk", factor), ("yarn", factor, context[, fast = 32, slow = 1]) or
    ("banded", factor, low, high, context)."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False, scaling=None, device="cuda"):
        import torch
        self.rot, self.interleaved = int(rot), bool(interleaved)
        phases, mul = np.zeros(max(self.rot // 2, 1), np.uint64), ctypes.c_float(1.0)
        if self.rot:
            kind, params = 0, None
            if scaling is not None:
                if scaling[0] not in ROPE_SCALINGS:
                    raise W4VError(ERR_ARG, "rope_phases")
                kind, count = ROPE_SCALINGS[scaling[0]]
                values = [float(x) for x in scaling[1:]]
                if scaling[0] == "yarn":
                    values += [32.0, 1.0][len(values) - 2:] if len(values) >= 2 else []
                if len(values) != count:
                    raise W4VError(ERR_ARG, "rope_phases")
                params = (ctypes.c_double * 4)(*values)
            _check(load().rope_phases(self.rot, float(base), kind, params, phases.ctypes.data, ctypes.byref(mul)),
                   "rope_phases")
        self.mul = mul.value
        self.phases = torch.from_numpy(phases.view(np.int64)).to(device)


class HeadNorm:
    """Norms of every query and key head (norm_rope_append): fp16 [head_dim] weights on the device (None: no
    weights), eps, and whether 1 is to be added to the weights."""

    def __init__(self, q_weight=None, k_weight=None, eps: float = 1e-6, zero_centred: bool = False):
        import torch
        if not (eps >= 0 and math.isfinite(eps)):
            raise W4VError(ERR_ARG, "HeadNorm")
        for w in (q_weight, k_weight):
            if w is None:
                continue
            if w.dim() != 1:
                raise W4VError(ERR_SHAPE, "HeadNorm")
            if w.dtype is not torch.float16 or not w.is_contiguous():
                raise W4VError(ERR_ARG, "HeadNorm")
        self.q_weight, self.k_weight, self.eps, self.zero_centred = q_weight, k_weight, float(eps), bool(zero_centred)


# What these calls check of their tensors costs as much as their smallest
# kernels run, so the types are looked up once and nothing is imported per call.
_HALF = _INT32 = _FLOAT = None


def _types():
    import torch
    global _HALF, _INT32, _FLOAT, _torch
    _torch = torch
    _HALF, _INT32, _FLOAT = torch.float16, torch.int32, torch.float32


def _i32(t, where, shape):
    """A dense int32 tensor of that shape: its address (0 for None)."""
    if t is None:
        return 0
    if t.shape != shape:
        raise W4VError(ERR_SHAPE, where)
    if t.dtype is not _INT32 or not t.is_contiguous():
        raise W4VError(ERR_ARG, where)
    return t.data_ptr()


def _here(at):
    """Whether device `at` is the GPU that is current (the library launches there)."""
    return at >= 0 and at == _torch._C._cuda_getDevice()


def _raw_stream(at):
    """The current stream of the current device `at`, where a tensor lies."""
    return _torch._C._cuda_getCurrentRawStream(at)


def _other(at, *tensors):
    """Whether one of the tensors (None: not given) lies elsewhere than on device `at`."""
    for t in tensors:
        if t is not None and t.get_device() != at:
            return True
    return False


def _rows(t, where, n, heads, head_dim):
    """Rows of dense heads: the row stride of a fp16 [n][heads][head_dim] tensor."""
    if t.shape != (n, heads, head_dim):
        raise W4VError(ERR_SHAPE, where)
    if t.dtype is not _HALF:
        raise W4VError(ERR_ARG, where)
    rows, head, step = t.stride()
    if n and (step != 1 or (heads > 1 and head != head_dim)):
        raise W4VError(ERR_ARG, where)
    return rows if n > 1 else heads * head_dim


def _dense_out(t, where, like, shape, stream):
    """The fp16 result tensor: t, or a new one of that shape."""
    if t is None:
        return _new(shape, _HALF, like.device, stream)
    if t.shape != shape:
        raise W4VError(ERR_SHAPE, where)
    if t.dtype is not _HALF or not t.is_contiguous():
        raise W4VError(ERR_ARG, where)
    return t


def _kv(where, k_cache, v_cache, table, lengths, offsets):
    """(packed w4v_kv_t, sequences, table width, kv heads, page, head_dim)."""
    if _HALF is None:
        _types()
    shape, seqs = k_cache.shape, table.shape
    if len(shape) != 4 or v_cache.shape != shape or len(seqs) != 2:
        raise W4VError(ERR_SHAPE, where)
    n_pages, heads, page, D = shape
    B, width = seqs
    if not (k_cache.dtype is v_cache.dtype is _HALF and k_cache.is_contiguous() and v_cache.is_contiguous() and
            table.dtype is _INT32 and table.is_contiguous()):
        raise W4VError(ERR_ARG, where)
    if lengths.shape != (B,) or offsets.shape != (B + 1,):
        raise W4VError(ERR_SHAPE, where)
    if not (lengths.dtype is offsets.dtype is _INT32 and lengths.is_contiguous() and offsets.is_contiguous()):
        raise W4VError(ERR_ARG, where)
    return (_KV.pack(k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), offsets.data_ptr(),
                     B, width, n_pages, heads, page, D), B, width, heads, page, D)


def rope_append(q, k, v, k_cache, v_cache, table, lengths, offsets, rope: Rope, q_out=None, positions=None,
                stream=None):
    """Rotate the new tokens' q [n][Hq][D] and k [n][Hkv][D] by their positions, write k and v [n][Hkv][D]
    into their pages of k_cache, v_cache [n_pages][Hkv][page][D] and return the rotated q.  q, k, v may
    be slices of one projection's rows; lengths count the new tokens.  positions: int32 [n], where the
    rotation's position is not the cache position.  Rows that no sequence's offsets cover are left alone:
    in a new q_out they hold anything."""
    where = "rope_append"
    kv, _, _, heads, _, D = _kv(where, k_cache, v_cache, table, lengths, offsets)
    shape = q.shape
    if len(shape) != 3:
        raise W4VError(ERR_SHAPE, where)
    n, Hq, _ = shape
    q_out = _dense_out(q_out, where, q, shape, stream)
    code = load().rope_append(kv, q.data_ptr(), k.data_ptr(), v.data_ptr(), _rows(q, where, n, Hq, D),
                              _rows(k, where, n, heads, D), _rows(v, where, n, heads, D), n, Hq,
                              _i32(positions, where, (n,)), rope.phases.data_ptr(), rope.rot, rope.mul,
                              ROPE_INTERLEAVED if rope.interleaved else 0, q_out.data_ptr(), _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return q_out


def norm_rope_append(q, k, v, k_cache, v_cache, table, lengths, offsets, rope: Rope, norm: HeadNorm, q_out=None,
                     positions=None, stream=None):
    """rope_append with every query and key head normed first (root mean square, weights of `norm`), in the
    same pass: nothing is rounded between the norm and the rotation."""
    where = "norm_rope_append"
    kv, _, _, heads, _, D = _kv(where, k_cache, v_cache, table, lengths, offsets)
    shape = q.shape
    if len(shape) != 3:
        raise W4VError(ERR_SHAPE, where)
    n, Hq, _ = shape
    wq, wk = norm.q_weight, norm.k_weight
    if (wq is not None and wq.shape[0] != D) or (wk is not None and wk.shape[0] != D):
        raise W4VError(ERR_SHAPE, where)
    strides = _rows(q, where, n, Hq, D), _rows(k, where, n, heads, D), _rows(v, where, n, heads, D)
    pos = _i32(positions, where, (n,))
    at = q.get_device()
    if not (at == k.get_device() == v.get_device() == k_cache.get_device() == v_cache.get_device() == table.get_device() ==
            lengths.get_device() == offsets.get_device() == rope.phases.get_device()) or not _here(at) or \
            _other(at, wq, wk, q_out, positions):
        raise W4VError(ERR_ARG, where)
    q_out = _dense_out(q_out, where, q, shape, stream)
    code = load().norm_rope_append(kv, q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, n, Hq,
                                   None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(),
                                   norm.eps, pos, rope.phases.data_ptr(), rope.rot, rope.mul,
                                   (ROPE_INTERLEAVED if rope.interleaved else 0) |
                                   (NORM_ZERO_CENTRED if norm.zero_centred else 0), q_out.data_ptr(),
                                   _raw_stream(at) if stream is None else _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return q_out


def paged_attn_workspace_bytes(n_tokens: int, B: int, q_heads: int, kv_heads: int, head_dim: int, max_context: int,
                               batch_invariant: bool = False) -> int:
    return load().paged_attn_workspace_bytes(n_tokens, B, q_heads, kv_heads, head_dim, max_context,
                                             BATCH_INVARIANT if batch_invariant else 0)


def paged_attn(q, k_cache, v_cache, table, lengths, offsets, scale=None, window: int = 0, out=None, lse=None, ws=None,
               stream=None, batch_invariant=False, sinks: int = 0):
    """Causal attention of the new tokens' q [n][Hq][D] over the paged cache that holds them (scale
    1/sqrt(D) unless given; window > 0: the last `window` tokens only, and with `sinks` the sequence's first
    ones).  Returns out [n][Hq][D].
    lse: float [n][Hq] to fill with the rows' log-sum-exp.
    Rows that no sequence's offsets cover are not written: in a new `out` they hold anything.
    batch_invariant: each row's result does not depend on what shares the call (W4V_BATCH_INVARIANT), as
    long as the table's size width * page stays up to 16,384, or between the same two powers of two."""
    where = "paged_attn"
    kv, B, width, heads, page, D = _kv(where, k_cache, v_cache, table, lengths, offsets)
    shape = q.shape
    if len(shape) != 3:
        raise W4VError(ERR_SHAPE, where)
    n, Hq, _ = shape
    stride = _rows(q, where, n, Hq, D)
    out = _dense_out(out, where, q, shape, stream)
    if lse is not None and (lse.shape != (n, Hq) or lse.dtype is not _FLOAT or not lse.is_contiguous()):
        raise W4VError(ERR_SHAPE if lse.shape != (n, Hq) else ERR_ARG, where)
    if ws is None:
        ws = workspace(paged_attn_workspace_bytes(n, B, Hq, heads, D, width * page, batch_invariant), q.device, stream)
    code = load().paged_attn_sinks(kv, q.data_ptr(), stride, n, Hq, D ** -0.5 if scale is None else scale, int(window),
                                   int(sinks), out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(),
                                   ws.numel(), BATCH_INVARIANT if batch_invariant else 0, _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return out


def paged_attn_shared_workspace_bytes(n_tokens: int, B: int, n_groups: int, q_heads: int, kv_heads: int,
                                      head_dim: int) -> int:
    return load().paged_attn_shared_workspace_bytes(n_tokens, B, n_groups, q_heads, kv_heads, head_dim)


def paged_attn_shared(q, k_cache, v_cache, table, lengths, offsets, groups, prefix, scale=None, out=None, lse=None,
                      ws=None, stream=None):
    """paged_attn for sequences that share a prefix, read once for all of them: sequences groups[g] ..
    groups[g + 1] - 1 (int32 [G + 1]) have their first prefix[g] tokens (int32 [G]) in common, as after
    kv_fork.  Returns out [n][Hq][D]; lse and rows of no sequence as in paged_attn."""
    where = "paged_attn_shared"
    kv, B, width, heads, page, D = _kv(where, k_cache, v_cache, table, lengths, offsets)
    shape = q.shape
    if len(shape) != 3 or prefix.dim() != 1:
        raise W4VError(ERR_SHAPE, where)
    n, Hq, _ = shape
    G = prefix.shape[0]
    stride = _rows(q, where, n, Hq, D)
    g, p = _i32(groups, where, (G + 1,)), _i32(prefix, where, (G,))
    if lse is not None and (lse.shape != (n, Hq) or lse.dtype is not _FLOAT or not lse.is_contiguous()):
        raise W4VError(ERR_SHAPE if lse.shape != (n, Hq) else ERR_ARG, where)
    at = q.get_device()
    if not (at == k_cache.get_device() == v_cache.get_device() == table.get_device() == lengths.get_device() ==
            offsets.get_device() == groups.get_device() == prefix.get_device()) or not _here(at) or \
            _other(at, out, lse, ws):
        raise W4VError(ERR_ARG, where)
    out = _dense_out(out, where, q, shape, stream)
    if ws is None:
        ws = workspace(paged_attn_shared_workspace_bytes(n, B, G, Hq, heads, D), q.device, stream)
    code = load().paged_attn_shared(kv, q.data_ptr(), stride, n, Hq, D ** -0.5 if scale is None else scale, g, p, G,
                                    out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), 0,
                                    _raw_stream(at) if stream is None else _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return out


LOGITS_FP16 = 16


def token_logprobs(logits, tokens=None, top: int = 0, temperature: float = 1.0, out=None, stream=None):
    """Log probabilities of `tokens` (int32 [M] or [M][n]; -1: none) under softmax(logits / temperature), logits
    float or fp16 [M][V] (rows may be part of longer ones).  Returns (logprobs as `tokens`, entropy [M],
    top_ids [M][top], top_logprobs [M][top]), the last two the `top` <= 32 most likely tokens in order.
    out: the four tensors to fill."""
    where = "token_logprobs"
    if _HALF is None:
        _types()
    if logits.dim() != 2 or not 0 <= top <= 32:
        raise W4VError(ERR_SHAPE, where)
    M, V = logits.shape
    half = logits.dtype is _HALF
    if not (half or logits.dtype is _FLOAT) or (M and V > 1 and logits.stride(1) != 1):
        raise W4VError(ERR_ARG, where)
    shape = (M, 0) if tokens is None else tokens.shape
    if len(shape) not in (1, 2) or shape[0] != M:
        raise W4VError(ERR_SHAPE, where)
    at, n = _i32(tokens, where, shape), shape[1] if len(shape) == 2 else 1
    dev = logits.get_device()
    if not _here(dev) or _other(dev, tokens):
        raise W4VError(ERR_ARG, where)
    if out is None:
        new = lambda shape, dtype: _new(shape, dtype, logits.device, stream)  # noqa: E731
        lp, entropy, ids, tops = out = new(shape, _FLOAT), new(M, _FLOAT), new((M, top), _INT32), new((M, top), _FLOAT)
    else:
        lp, entropy, ids, tops = out
        if lp.shape != shape or entropy.shape != (M,) or ids.shape != (M, top) or tops.shape != (M, top):
            raise W4VError(ERR_SHAPE, where)
        if not (lp.dtype is entropy.dtype is tops.dtype is _FLOAT and ids.dtype is _INT32 and lp.is_contiguous() and
                entropy.is_contiguous() and ids.is_contiguous() and tops.is_contiguous()) or _other(dev, *out):
            raise W4VError(ERR_ARG, where)
    code = load().token_logprobs(logits.data_ptr(), logits.stride(0) if M > 1 else V, M, V, at, n, temperature,
                                 lp.data_ptr(), entropy.data_ptr(), top, ids.data_ptr(), tops.data_ptr(),
                                 LOGITS_FP16 if half else 0, _raw_stream(dev) if stream is None else _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return out


def kv_workspace_bytes(n_pages: int, S: int) -> int:
    return load().kv_workspace_bytes(n_pages, S)


def _plane(pool):
    """(planes, n_pages, page, bytes of one page in one plane) of [..., n_pages][heads][page][head_dim]."""
    shape = pool.shape
    if len(shape) < 5:
        raise W4VError(ERR_SHAPE, "pool")
    nbytes = shape[-3] * shape[-2] * shape[-1] * pool.element_size()
    return shape[0] if len(shape) == 5 else math.prod(shape[:-4]), shape[-4], shape[-2], nbytes


def _pages(where, pool, refs, table, lengths, page=None):
    """(packed w4v_pages_t, n_pages, S, table width)."""
    if _HALF is None:
        _types()
    seqs = table.shape
    if refs.dim() != 1 or len(seqs) != 2:
        raise W4VError(ERR_SHAPE, where)
    n_pages, (S, width) = refs.shape[0], seqs
    planes, nbytes, at = 0, 0, 0
    if pool is not None:
        planes, pool_pages, page, nbytes = _plane(pool)
        if pool_pages != n_pages:
            raise W4VError(ERR_SHAPE, where)
        if not pool.is_contiguous():
            raise W4VError(ERR_ARG, where)
        at = pool.data_ptr()
    return (_PAGES.pack(at, _i32(refs, where, (n_pages,)), _i32(table, where, (S, width)), _i32(lengths, where, (S,)),
                        nbytes, planes, n_pages, S, width, page), n_pages, S, width)


def _short(short, where, device, stream):
    if short is None:
        short = _new(1, _INT32, device, stream, zero=True)
    return short, _i32(short, where, (1,))


def kv_extend(pool, refs, table, lengths, new_lengths, short=None, ws=None, stream=None):
    """Pages for new_lengths [S] tokens a sequence (pool [..., n_pages][Hkv][page][D], the planes in front;
    refs int32 [n_pages], table int32 [S][width], lengths int32 [S], all changed in place).  Returns the
    int32 [1] tensor `short`: 0, or what keeps the call from changing anything (see include/w4v.h)."""
    where = "kv_extend"
    pages, n_pages, S, _ = _pages(where, pool, refs, table, lengths)
    want = _i32(new_lengths, where, (S,))
    short, at = _short(short, where, refs.device, stream)
    if ws is None:
        ws = workspace(kv_workspace_bytes(n_pages, S), refs.device, stream)
    code = load().kv_extend(pages, want, at, ws.data_ptr(), ws.numel(), _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return short


def kv_truncate(refs, table, lengths, new_lengths, page: int, stream=None):
    """Lengths down to new_lengths [S], in place; pages that nothing holds any more become free."""
    where = "kv_truncate"
    pages, _, S, _ = _pages(where, None, refs, table, lengths, int(page))
    code = load().kv_truncate(pages, _i32(new_lengths, where, (S,)), _stream(stream))
    if code != OK:
        raise W4VError(code, where)


def kv_fork(pool, refs, table, lengths, parents, children, short=None, ws=None, stream=None):
    """Sequences children[i] become copies of parents[i] (int32 [n]): full pages shared, a partly
    filled last one copied.  Returns `short` as kv_extend does."""
    where = "kv_fork"
    pages, n_pages, S, _ = _pages(where, pool, refs, table, lengths)
    n = parents.numel()
    a, c = _i32(parents, where, (n,)), _i32(children, where, (n,))
    short, at = _short(short, where, refs.device, stream)
    if ws is None:
        ws = workspace(kv_workspace_bytes(n_pages, S), refs.device, stream)
    code = load().kv_fork(pages, a, c, n, at, ws.data_ptr(), ws.numel(), _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return short


def kv_compact(pool, refs, table, lengths, refs_out=None, table_out=None, ws=None, stream=None):
    """All live pages to the lowest ids; returns (refs_out, table_out), the old arrays unless given."""
    where = "kv_compact"
    pages, n_pages, S, width = _pages(where, pool, refs, table, lengths)
    refs_out, table_out = refs if refs_out is None else refs_out, table if table_out is None else table_out
    r, t = _i32(refs_out, where, (n_pages,)), _i32(table_out, where, (S, width))
    if ws is None:
        ws = workspace(kv_workspace_bytes(n_pages, S), refs.device, stream)
    code = load().kv_compact(pages, r, t, ws.data_ptr(), ws.numel(), _stream(stream))
    if code != OK:
        raise W4VError(code, where)
    return refs_out, table_out


def kv_copy(pool, src, dst, stream=None):
    """Contents of pages src[i] to pages dst[i] (int32 [n]) in every plane of pool [..., n_pages][Hkv][page][D]."""
    where = "kv_copy"
    if _HALF is None:
        _types()
    planes, n_pages, _, nbytes = _plane(pool)
    if not pool.is_contiguous():
        raise W4VError(ERR_ARG, where)
    n = src.numel()
    code = load().kv_copy(pool.data_ptr(), planes, n_pages, nbytes, _i32(src, where, (n,)), _i32(dst, where, (n,)), n,
                          _stream(stream))
    if code != OK:
        raise W4VError(code, where)
