"""Binding of the packed-document calls of ``include/wan.h``: rotary positions with the
q/k norm, the gated residual with the norms around it, and attention inside documents,
each with its gradient.

A packed tensor holds documents of different lengths one after another along its rows;
``cu`` is an int32 device tensor of ``n_docs + 1`` row offsets. Every call checks types,
shapes and devices before it reaches the library, and runs on the device of its tensors
(on that device's current stream unless ``stream`` is given); nothing is allocated.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import Config, WAN_BF16, _check, _lib

__all__ = [
    "RopeSpec", "ResidualNormSpec", "Documents", "rope", "residual_norm", "documents", "qk_norm_rope_fwd",
    "qk_norm_rope_bwd", "qk_norm_rope_workspace_bytes", "gated_residual_norm_fwd", "gated_residual_norm_bwd",
    "gated_residual_norm_workspace_bytes", "attention_packed_fwd", "attention_packed_bwd",
    "attention_packed_workspace_bytes",
]

_vp, _i, _i64, _sz, _f, _d = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float,
                              ctypes.c_double)

LAYOUTS = {"interleaved": 0, "half": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
QK_NORMS = {"none": 0, "head": 1, "width": 2}
NORMS = {"none": 0, "layer": 1, "rms": 2}


class Rows(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("row_stride", _i64)]


class RopeSpec(ctypes.Structure):
    """``wan_rope``; made by :func:`rope`."""
    _fields_ = [("layout", _i), ("scaling", _i), ("n_axes", _i), ("axis_dim", _i * 3), ("orig_len", _i * 3),
                ("theta", _d), ("factor", _d * 3), ("fast", _d), ("slow", _d), ("amplitude", _d)]


class ResidualNormSpec(ctypes.Structure):
    """``wan_residual_norm``; made by :func:`residual_norm`, keeps its weight tensors."""
    _fields_ = [("pre", _i), ("post", _i), ("gate", _i), ("chunk", _i), ("residual_scale", _f), ("w_pre", _vp),
                ("b_pre", _vp), ("w_post", _vp)]


class ResidualNormGrads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("de", "dmod_bias", "dw_pre", "db_pre", "dw_post")]


class Documents(ctypes.Structure):
    """``wan_documents``; made by :func:`documents`, keeps its tensors."""
    _fields_ = [("n_docs", _i), ("cu_q", _vp), ("cu_k", _vp), ("prefix", _vp), ("causal_block", _i), ("scale", _f),
                ("cap", _f), ("slopes", _vp)]


def signatures():
    P = ctypes.POINTER
    c, r = P(Config), P(Rows)
    return {
        "wan_qk_norm_rope_fwd": (_i, [c, P(RopeSpec), _vp, _i, _i, _i, r, r, _vp, _vp, r, r, _vp]),
        "wan_qk_norm_rope_bwd": (_i, [c, P(RopeSpec), _vp, _i, _i, _i, r, r, r, r, _vp, _vp, r, r, _vp, _vp, _vp, _sz,
                                      _vp]),
        "wan_qk_norm_rope_workspace_bytes": (_sz, [c, _i, _i, _i]),
        "wan_gated_residual_norm_fwd": (_i, [c, P(ResidualNormSpec), _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp]),
        "wan_gated_residual_norm_bwd": (_i, [c, P(ResidualNormSpec), _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp,
                                             _vp, P(ResidualNormGrads), _vp, _sz, _vp]),
        "wan_gated_residual_norm_workspace_bytes": (_sz, [c, _i, _i]),
        "wan_attention_packed_fwd": (_i, [c, P(Documents), _i, _i, _i, r, r, r, r, _vp, _vp, _sz, _vp]),
        "wan_attention_packed_bwd": (_i, [c, P(Documents), _i, _i, _i, r, r, r, r, _vp, r, r, r, r, _vp, _sz, _vp]),
        "wan_attention_packed_workspace_bytes": (_sz, [c, _i, _i, _i, _i, _i]),
    }


# ------------------------------------------------------------------ argument checks
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream, device):
    """The stream given, or the device's current one."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(device)


def _act(cfg):
    return _torch().bfloat16 if cfg.dtype == WAN_BF16 else _torch().float32


class _Args:
    """Collects the tensors of one call: their device must be one CUDA device."""
    __slots__ = ("where", "device")

    def __init__(self, where):
        self.where, self.device = where, -1

    def fail(self, what):
        raise ValueError(f"{self.where}: {what}")

    def _seen(self, t, name):
        d = t.get_device()  # -1 on the CPU
        if d != self.device or d < 0:
            if d < 0:
                self.fail(f"{name} is not on a CUDA device")
            if self.device >= 0:
                self.fail(f"{name} is on device {d}, the other tensors on {self.device}")
            self.device = d

    def array(self, t, name, dtype, shape, optional=False):
        """Pointer of a contiguous tensor of this type and shape."""
        if t is None:
            if not optional:
                self.fail(f"{name} is required")
            return None
        self._seen(t, name)
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            self.fail(f"{name} must be contiguous {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)} "
                      f"strides {t.stride()}")
        return t.data_ptr()

    def rows(self, t, name, dtype, n, width, optional=False):
        """wan_rows of a [n, width] tensor whose rows are dense (a column slice will do)."""
        if t is None:
            if not optional:
                self.fail(f"{name} is required")
            return None
        self._seen(t, name)
        st = t.stride()
        if t.dtype != dtype or t.shape != (n, width) or (st[1] != 1 and width > 1):
            self.fail(f"{name} must be {dtype} [{n}, {width}] with dense rows, got {t.dtype} {tuple(t.shape)} strides {st}")
        stride = st[0] if n > 1 else width  # the stride of a single row says nothing
        return ctypes.byref(Rows(t.data_ptr(), stride))

    def workspace(self, ws):
        if ws is None:
            return None, 0
        self._seen(ws, "ws")
        if not ws.is_contiguous():
            self.fail("ws must be contiguous")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def call(self, fn, stream, *args):
        f, torch, dev = getattr(_lib(), fn), _torch(), self.device
        if dev < 0:  # a call without tensors
            dev = torch.cuda.current_device()
        if dev == torch._C._cuda_getDevice():
            status = f(*args, _stream(stream, dev))
        else:
            with torch.cuda.device(dev):
                status = f(*args, _stream(stream, dev))
        if status != 0:
            _check(status, fn)


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


# ------------------------------------------------------------------ rotary positions
def rope(axes: Sequence[int], layout: str = "interleaved", theta: float = 10000.0, scaling: str = "none",
         factor: Sequence[float] = (), orig_len: Sequence[int] = (), fast: float = 32.0, slow: float = 1.0,
         amplitude: float = 1.0) -> RopeSpec:
    """Rotary positions over the first ``sum(axes)`` dims of every head, ``axes[a]`` of them
    turned by position axis a. ``scaling``: "linear" (frequencies / factor), "base" (theta
    raised so that the slowest pair is stretched by the factor), "ramp" (pairs with more
    than ``fast`` turns over ``orig_len`` positions keep their frequency, those with fewer
    than ``slow`` are stretched by the factor, a ramp between). The library checks values."""
    axes = [int(a) for a in axes]
    if not 1 <= len(axes) <= 3:
        raise ValueError(f"rope: 1 to 3 axes, got {len(axes)}")
    s = RopeSpec(_choice(LAYOUTS, layout, "layout"), _choice(SCALINGS, scaling, "scaling"), len(axes))
    if scaling != "none" and len(factor) != len(axes):
        raise ValueError("rope: a factor per axis")
    if scaling == "ramp" and len(orig_len) != len(axes):
        raise ValueError("rope: an orig_len per axis")
    for a, n in enumerate(axes):
        s.axis_dim[a] = n
        if scaling != "none":
            s.factor[a] = float(factor[a])
        if scaling == "ramp":
            s.orig_len[a] = int(orig_len[a])
    s.theta, s.fast, s.slow, s.amplitude = float(theta), float(fast), float(slow), float(amplitude)
    return s


def _qk_weights(a, cfg, norm, kv_heads, with_k, w_q, w_k):
    if norm == "none":
        return None, None
    nq, nk = (cfg.head_dim,) * 2 if norm == "head" else (cfg.heads * cfg.head_dim, kv_heads * cfg.head_dim)
    return (a.array(w_q, "w_q", _act(cfg), (nq,)), a.array(w_k, "w_k", _act(cfg), (nk,)) if with_k else None)


def qk_norm_rope_fwd(cfg, rope: RopeSpec, positions, q, k, q_out, k_out, kv_heads: Optional[int] = None,
                     norm: str = "none", w_q=None, w_k=None, stream=None):
    """q [rows, heads*d], k [rows, kv_heads*d] (both may be column slices; k and k_out None:
    q alone) -> q_out, k_out (may be q, k): norm ("none", "head", "width") and rotation by
    positions [rows, n_axes] int32."""
    a = _Args("qk_norm_rope_fwd")
    torch, act, kv = _torch(), _act(cfg), cfg.heads if kv_heads is None else int(kv_heads)
    nm, n, wq, wk = _choice(QK_NORMS, norm, "norm"), q.shape[0], cfg.heads * cfg.head_dim, kv * cfg.head_dim
    if (k is None) != (k_out is None):
        a.fail("k and k_out go together")
    pos = a.array(positions, "positions", torch.int32, (n, rope.n_axes))
    v = [a.rows(q, "q", act, n, wq), a.rows(k, "k", act, n, wk, optional=True)]
    o = [a.rows(q_out, "q_out", act, n, wq), a.rows(k_out, "k_out", act, n, wk, optional=True)]
    w = _qk_weights(a, cfg, norm, kv, k is not None, w_q, w_k)
    a.call("wan_qk_norm_rope_fwd", stream, ctypes.byref(cfg), ctypes.byref(rope), pos, n, kv, nm, *v, *w, *o)


def qk_norm_rope_workspace_bytes(cfg, rows: int, kv_heads: int, norm: str) -> int:
    return int(_lib().wan_qk_norm_rope_workspace_bytes(ctypes.byref(cfg), rows, kv_heads,
                                                       _choice(QK_NORMS, norm, "norm")))


def qk_norm_rope_bwd(cfg, rope: RopeSpec, positions, dq_out, dk_out, q, k, dq, dk, kv_heads: Optional[int] = None,
                     norm: str = "none", w_q=None, w_k=None, dw_q=None, dw_k=None, ws=None, stream=None):
    """Gradients of q_out, k_out -> dq, dk (dq may be dq_out) and, with a norm, dw_q, dw_k
    float32 (optional). q, k: the forward's inputs (None allowed for norm "none")."""
    a = _Args("qk_norm_rope_bwd")
    torch, act, kv = _torch(), _act(cfg), cfg.heads if kv_heads is None else int(kv_heads)
    nm, n, wq, wk = _choice(QK_NORMS, norm, "norm"), dq_out.shape[0], cfg.heads * cfg.head_dim, kv * cfg.head_dim
    if (dk_out is None) != (dk is None):
        a.fail("dk_out and dk go together")
    with_k, plain = dk is not None, norm == "none"
    pos = a.array(positions, "positions", torch.int32, (n, rope.n_axes))
    g = [a.rows(dq_out, "dq_out", act, n, wq), a.rows(dk_out, "dk_out", act, n, wk, optional=True)]
    x = [None, None] if plain else [a.rows(q, "q", act, n, wq), a.rows(k, "k", act, n, wk, optional=not with_k)]
    w = _qk_weights(a, cfg, norm, kv, with_k, w_q, w_k)
    o = [a.rows(dq, "dq", act, n, wq), a.rows(dk, "dk", act, n, wk, optional=True)]
    if plain and (dw_q is not None or dw_k is not None):
        a.fail("there are no norm weights")
    dw = [None, None]
    if not plain:
        nq, nk = (cfg.head_dim,) * 2 if norm == "head" else (wq, wk)
        dw = [a.array(dw_q, "dw_q", torch.float32, (nq,), optional=True),
              a.array(dw_k, "dw_k", torch.float32, (nk,), optional=True)]
    a.call("wan_qk_norm_rope_bwd", stream, ctypes.byref(cfg), ctypes.byref(rope), pos, n, kv, nm, *g, *x, *w, *o, *dw,
           *a.workspace(ws))


# ------------------------------------------------------------------ gated residual + norm
def residual_norm(pre: str = "layer", post: str = "none", gate: int = -1, chunk: int = -1,
                  residual_scale: float = 1.0, w_pre=None, b_pre=None, w_post=None) -> ResidualNormSpec:
    """x' = residual_scale x + gate_d post(y) w_post; h = (pre(x') w_pre + b_pre)(1 + scale_d)
    + shift_d. ``gate``: row of e (0..5) or -1; ``chunk``: shift and scale rows 3 chunk and
    3 chunk + 1 of e, or -1."""
    s = ResidualNormSpec(_choice(NORMS, pre, "pre"), _choice(NORMS, post, "post"), int(gate), int(chunk),
                         float(residual_scale))
    s.weights = (w_pre, b_pre, w_post)
    return s


def _spec_pointers(a, cfg, op):
    D, act = cfg.dim, _act(cfg)
    for name, t in zip(("w_pre", "b_pre", "w_post"), op.weights):
        setattr(op, name, a.array(t, name, act, (D,), optional=True))


def _docs_of(a, cu, name="cu"):
    if cu is None or cu.dim() != 1 or cu.numel() < 1:
        a.fail(f"{name} must hold n_docs + 1 offsets")
    return cu.numel() - 1


def _residual_args(a, cfg, op, x, y, e, mod_bias, cu):
    torch, D, n = _torch(), cfg.dim, x.shape[0]
    docs = _docs_of(a, cu)
    _spec_pointers(a, cfg, op)
    uses_e = op.gate >= 0 or op.chunk >= 0
    return [a.array(x, "x", torch.float32, (n, D)), a.array(y, "y", _act(cfg), (n, D)),
            a.array(e, "e", torch.float32, (docs, 6, D), optional=not uses_e or docs == 0),
            a.array(mod_bias, "mod_bias", torch.float32, (6, D), optional=True),
            a.array(cu, "cu", torch.int32, (docs + 1,)), docs, n]


def gated_residual_norm_fwd(cfg, op: ResidualNormSpec, x, y, e, mod_bias, cu, x_out, h_out, stream=None):
    """x [rows, D] float32, y [rows, D] act, e [n_docs, 6, D] float32 -> x_out (may be x),
    h_out act (may be y). Rows of no document are not written."""
    a = _Args("gated_residual_norm_fwd")
    args = _residual_args(a, cfg, op, x, y, e, mod_bias, cu)
    out = [a.array(x_out, "x_out", _torch().float32, x.shape), a.array(h_out, "h_out", _act(cfg), x.shape)]
    a.call("wan_gated_residual_norm_fwd", stream, ctypes.byref(cfg), ctypes.byref(op), *args, *out)


def gated_residual_norm_workspace_bytes(cfg, rows: int, n_docs: int) -> int:
    return int(_lib().wan_gated_residual_norm_workspace_bytes(ctypes.byref(cfg), rows, n_docs))


def gated_residual_norm_bwd(cfg, op: ResidualNormSpec, x_out, y, e, mod_bias, cu, dh, dx_out, dx, dy, ws=None, de=None,
                            dmod_bias=None, dw_pre=None, db_pre=None, dw_post=None, stream=None):
    """x_out: the forward's result, y its branch input; dh act the gradient of h, dx_out
    float32 (or None: 0) that of x_out -> dx (may be dx_out), dy (may be dh) and the sums
    asked for, all float32: de [n_docs, 6, D] (only the rows in use are written), dmod_bias
    [6, D] (the same rows), dw_pre, db_pre, dw_post [D]."""
    a = _Args("gated_residual_norm_bwd")
    torch, act, D = _torch(), _act(cfg), cfg.dim
    args = _residual_args(a, cfg, op, x_out, y, e, mod_bias, cu)
    n, docs = x_out.shape[0], args[5]
    args += [a.array(dh, "dh", act, (n, D)), a.array(dx_out, "dx_out", torch.float32, (n, D), optional=True),
             a.array(dx, "dx", torch.float32, (n, D)), a.array(dy, "dy", act, (n, D))]
    if op.post == 0 and dw_post is not None:
        a.fail("dw_post needs a norm of y")
    g = ResidualNormGrads(a.array(de, "de", torch.float32, (docs, 6, D), optional=True),
                          a.array(dmod_bias, "dmod_bias", torch.float32, (6, D), optional=True),
                          *[a.array(t, name, torch.float32, (D,), optional=True)
                            for name, t in (("dw_pre", dw_pre), ("db_pre", db_pre), ("dw_post", dw_post))])
    a.call("wan_gated_residual_norm_bwd", stream, ctypes.byref(cfg), ctypes.byref(op), *args, ctypes.byref(g),
           *a.workspace(ws))


# ------------------------------------------------------------------ attention in documents
def documents(cu_q, cu_k=None, prefix=None, causal_block: int = 0, cap: float = 0.0, slopes=None,
              scale: float = 0.0) -> Documents:
    """Documents of attention_packed_*: offsets of their query and key rows (cu_k None: the
    same), an optional int32 prefix per document, the causal block (0: every key is seen;
    g: blocks of g rows in order), tanh cap of the scores (0: none), a float32 distance
    slope per head, and the score scale (0: 1/sqrt(head_dim))."""
    s = Documents()
    s.n_docs, s.causal_block, s.scale, s.cap = int(cu_q.numel()) - 1, int(causal_block), float(scale), float(cap)
    s.tensors = (cu_q, cu_q if cu_k is None else cu_k, prefix, slopes)
    return s


def _docs_pointers(a, cfg, s):
    torch = _torch()
    cu_q, cu_k, prefix, slopes = s.tensors
    n = _docs_of(a, cu_q, "cu_q")
    s.cu_q = a.array(cu_q, "cu_q", torch.int32, (n + 1,))
    s.cu_k = a.array(cu_k, "cu_k", torch.int32, (n + 1,))
    s.prefix = a.array(prefix, "prefix", torch.int32, (n,), optional=True) or None
    s.slopes = a.array(slopes, "slopes", torch.float32, (cfg.heads,), optional=True)


def attention_packed_workspace_bytes(cfg, q_rows: int, k_rows: int, n_docs: int, kv_heads: int,
                                     backward: bool = False) -> int:
    """Bytes of the forward's workspace (optional there: it lets few query rows over many
    keys be split over the keys) or of the gradient's; one buffer may serve both."""
    return int(_lib().wan_attention_packed_workspace_bytes(ctypes.byref(cfg), q_rows, k_rows, n_docs, kv_heads,
                                                           1 if backward else 0))


def attention_packed_fwd(cfg, docs: Documents, q, k, v, o, lse=None, kv_heads: Optional[int] = None, ws=None,
                         stream=None):
    """q [q_rows, heads*d], k and v [k_rows, kv_heads*d] (column slices will do) -> o as q,
    lse [heads, q_rows] float32 (optional). Rows of no document are not written."""
    a = _Args("attention_packed_fwd")
    act, kv, nq, nk = _act(cfg), cfg.heads if kv_heads is None else int(kv_heads), q.shape[0], k.shape[0]
    wq, wk = cfg.heads * cfg.head_dim, kv * cfg.head_dim
    _docs_pointers(a, cfg, docs)
    t = [a.rows(q, "q", act, nq, wq), a.rows(k, "k", act, nk, wk), a.rows(v, "v", act, nk, wk),
         a.rows(o, "o", act, nq, wq)]
    ls = a.array(lse, "lse", _torch().float32, (cfg.heads, nq), optional=True)
    a.call("wan_attention_packed_fwd", stream, ctypes.byref(cfg), ctypes.byref(docs), nq, nk, kv, *t, ls,
           *a.workspace(ws))


def attention_packed_bwd(cfg, docs: Documents, q, k, v, o, lse, do, dq, dk, dv, kv_heads: Optional[int] = None,
                         ws=None, stream=None):
    """o, lse: the forward's results, do the gradient of o -> dq, dk, dv. Keys that no query
    sees get 0; rows of no document are not written."""
    a = _Args("attention_packed_bwd")
    act, kv, nq, nk = _act(cfg), cfg.heads if kv_heads is None else int(kv_heads), q.shape[0], k.shape[0]
    wq, wk = cfg.heads * cfg.head_dim, kv * cfg.head_dim
    _docs_pointers(a, cfg, docs)
    t = [a.rows(q, "q", act, nq, wq), a.rows(k, "k", act, nk, wk), a.rows(v, "v", act, nk, wk),
         a.rows(o, "o", act, nq, wq)]
    ls = a.array(lse, "lse", _torch().float32, (cfg.heads, nq))
    g = [a.rows(do, "do", act, nq, wq), a.rows(dq, "dq", act, nq, wq), a.rows(dk, "dk", act, nk, wk),
         a.rows(dv, "dv", act, nk, wk)]
    a.call("wan_attention_packed_bwd", stream, ctypes.byref(cfg), ctypes.byref(docs), nq, nk, kv, *t, ls, *g,
           *a.workspace(ws))
