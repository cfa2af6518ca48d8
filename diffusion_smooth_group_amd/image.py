"""ctypes binding of the operators of an image model's conditioned blocks
(include/svdq_image.h): what runs between the 4-bit linears where an encoder's
states enter.

    y = group_norm(x, groups, weight, bias, act="silu")      x [samples, height, width, channels]
    o = cross_attention(q, k, v, mask=mask)                  q, k, v [requests, tokens, heads, D]

Argument marshalling only, as in ``kv.py``, whose conventions hold: a call runs
on the current stream or, with stream=, as if made under
``torch.cuda.stream(stream)``; all its tensors are on one device, which need not
be the current one; a wrong argument raises ValueError here or SvdqError with
the library's status.

Maps are channels last: the last dimension has unit stride and the dimensions
between the first and the last are one run of pixels (views of wider rows are
taken as they are; a torch ``channels_last`` tensor is passed as
``x.permute(0, 2, 3, 1)``).  ``*_autograd`` are the operators under
torch.autograd; their gradients can not be differentiated again (torch raises an
error).
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import kv
from . import svdq as S
from .kv import SvdqError, _code, _on, _scratch, _size, _stream, svdq_heads  # noqa: F401

ACT = {None: 0, "silu": 1, "gelu": 2}

_P, _I64, _I32, _F, _SZ = C.c_void_p, C.c_int64, C.c_int32, C.c_float, C.c_size_t


class svdq_map(C.Structure):
    _fields_ = [("data", _P), ("sample_stride", _I64), ("pixel_stride", _I64)]


class svdq_norm_desc(C.Structure):
    _fields_ = [("samples", _I64), ("pixels", _I64), ("channels", _I32), ("groups", _I32), ("dtype", _I32), ("act", _I32), ("eps", _F),
                ("weight", _P), ("bias", _P)]


class svdq_cross_desc(C.Structure):
    _fields_ = [("requests", _I64), ("tokens", _I64), ("states", _I64), ("head_dim", _I32), ("dtype", _I32), ("max_q", _I32),
                ("max_k", _I32), ("scale", _F), ("q_start", _P), ("k_start", _P), ("mask", _P)]


_NP, _MP, _XP, _HP = C.POINTER(svdq_norm_desc), C.POINTER(svdq_map), C.POINTER(svdq_cross_desc), C.POINTER(svdq_heads)
_SIGS = {
    "svdq_group_norm_workspace": [_NP, C.POINTER(_SZ)],
    "svdq_group_norm": [_NP, _MP, _MP, _P, _P, _SZ, _P],
    "svdq_group_norm_backward_workspace": [_NP, C.POINTER(_SZ)],
    "svdq_group_norm_backward": [_NP, _MP, _MP, _P, _MP, _P, _P, _P, _SZ, _P],
    "svdq_cross_attention_workspace": [_XP, _I32, _I32, C.POINTER(_SZ)],
    "svdq_cross_attention": [_XP, _HP, _HP, _HP, _HP, _P, _P, _SZ, _P],
    "svdq_cross_attention_backward_workspace": [_XP, _I32, _I32, C.POINTER(_SZ)],
    "svdq_cross_attention_backward": [_XP, _HP, _HP, _HP, _HP, _P, _HP, _HP, _HP, _HP, _P, _SZ, _P],
}
_FN = {}


def _fn(name):
    fn = _FN.get(name)
    if fn is None:
        fn = getattr(S.lib_handle(), name)
        fn.argtypes, fn.restype = _SIGS[name], C.c_int
        _FN[name] = fn
    return fn


def _call(name, *args):
    rc = _fn(name)(*args)
    if rc != 0:
        raise SvdqError(name, rc)


def _call_with_workspace(name, like, ws, size_of, before, stream, likely):
    """The call with the caller's workspace, or with one of its own where it needs
    one.  size_of: the arguments that tell its size.  Where a call is not `likely` to
    need one it goes without first (it says so before anything is launched), so that
    small calls are spared the question: 1 us of 9.5."""
    if ws is not None:
        _call(name, *before, *_scratch(ws, like.get_device()), stream)
        return
    if not likely:
        rc = _fn(name)(*before, None, 0, stream)
        if rc == 0:
            return
    need = _SZ(0)
    _call(name + "_workspace", *size_of, need)
    if need.value == 0:
        if not likely:
            raise SvdqError(name, rc)
        _call(name, *before, None, 0, stream)
        return
    ws = like.new_empty(need.value, dtype=torch.uint8)
    _call(name, *before, ws.data_ptr(), need.value, stream)


def _address(ws):
    return None if ws is None else ws.data_ptr()


# ------------------------------------------------------------------ group norm
def _run(t):
    """Stride between the pixels of t [samples, ..., channels], None where they are not one run."""
    step = None
    for n, s in zip(t.shape[-2:0:-1], t.stride()[-2:0:-1]):
        if n == 1:
            continue
        if step is None:
            step, span = s, s * n
        elif s != span:
            return None
        else:
            span *= n
    return 0 if step is None else step


def _map(t, name, like, dev):
    shape = like.shape
    if t.is_contiguous():
        c = shape[-1]
        step, first = c, (t.numel() // shape[0] if shape[0] > 1 else 0)
    else:
        step, first = _run(t), (t.stride(0) if shape[0] > 1 else 0)
        if step is None or t.stride(-1) != 1:
            raise ValueError(f"{name}: channels last with unit stride and one run of pixels is needed, got {tuple(t.shape)} with strides {t.stride()}")
    if t is not like and t.shape != shape or t.dtype is not like.dtype or t.get_device() != dev:
        raise ValueError(f"{name}: a {like.dtype} tensor {tuple(shape)} on cuda:{dev} is needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return svdq_map(t.data_ptr(), first, step)


def _new_map(like, view, dev):
    """An output like `like`, channels last, and its view for the call; view: like's."""
    t = torch.empty_like(like)
    if t.stride() == like.stride():
        return t, svdq_map(t.data_ptr(), view.sample_stride, view.pixel_stride)
    if not t.is_contiguous() and (t.stride(-1) != 1 or _run(t) is None):
        t = like.new_empty(like.shape)
    return t, _map(t, "out", like, dev)


def _norm_desc(x, groups, weight, bias, eps, act, dev):
    if x.dim() < 2:
        raise ValueError(f"x: [samples, ..., channels] is needed, got {tuple(x.shape)}")
    if act not in ACT:
        raise ValueError(f"act: one of {list(ACT)} is needed, got {act!r}")
    n, c = x.shape[0], x.shape[-1]
    dtype = x.dtype
    return svdq_norm_desc(n, math.prod(x.shape[1:-1]), _size(c, "channels"), _size(groups, "groups"), _code(dtype), ACT[act], eps,
                          kv._weight(weight, "weight", c, dtype, dev), kv._weight(bias, "bias", c, dtype, dev))


def group_norm(x, groups: int, weight=None, bias=None, eps: float = 1e-5, act: Optional[str] = None, out=None, ws=None,
               return_stats: bool = False, stream=None):
    """act((x - mean) / sqrt(var + eps) * weight + bias) over the pixels and the
    channels / groups channels of each group of x [samples, ..., channels].
    weight, bias [channels] (None: ones, zeros); act: None, "silu" or "gelu".
    out=x works in place.  Returns out, or (out, stats): mean and 1 / sqrt(var +
    eps), fp32 [samples, groups, 2]."""
    with _on(stream, x):
        dev = kv._current_device()
        d = _norm_desc(x, groups, weight, bias, eps, act, dev)
        mx = _map(x, "x", x, dev)
        if out is None:
            out, mo = _new_map(x, mx, dev)
        else:
            mo = _map(out, "out", x, dev)
        stats = x.new_empty((x.shape[0], groups, 2), dtype=torch.float32) if return_stats else None
        _call_with_workspace("svdq_group_norm", x, ws, (d,), (d, mx, mo, _address(stats)), _stream(x),
                             d.pixels * d.channels > 65536 * d.groups)
        return (out, stats) if return_stats else out


def group_norm_backward(g, x, stats, groups: int, weight=None, bias=None, act: Optional[str] = None, dx=None, ws=None, stream=None):
    """Gradient of ``group_norm`` from g (with respect to its output), its input
    and its stats.  Returns (dx, dw, db), the sums over samples and pixels fp32
    [channels].  dx=g and dx=x work in place."""
    with _on(stream, x):
        dev = kv._current_device()
        d = _norm_desc(x, groups, weight, bias, 0.0, act, dev)
        mx, mg = _map(x, "x", x, dev), _map(g, "g", x, dev)
        if dx is None:
            dx, md = _new_map(x, mx, dev)
        else:
            md = _map(dx, "dx", x, dev)
        if stats.dtype is not torch.float32 or stats.shape != (x.shape[0], groups, 2) or not stats.is_contiguous() or stats.get_device() != dev:
            raise ValueError(f"stats: a contiguous float32 tensor {(x.shape[0], groups, 2)} on cuda:{dev} is needed, "
                             f"got {stats.dtype} {tuple(stats.shape)} on {stats.device}")
        dw, db = x.new_empty((2, x.shape[-1]), dtype=torch.float32).unbind()
        _call_with_workspace("svdq_group_norm_backward", x, ws, (d,), (d, mx, mg, stats.data_ptr(), md, dw.data_ptr(), db.data_ptr()), _stream(x),
                             d.samples > 2 or d.pixels * d.channels > 16384 * d.groups)
        return dx, dw, db


def _as_map(t):
    """t as the library takes a map; what it does not (a gradient that is
    broadcast over pixels) is written out."""
    step = _run(t)
    fits = t.stride(-1) == 1 and step is not None and step % 8 == 0 and t.stride(0) % 8 == 0 and t.data_ptr() % 16 == 0 \
        and (step >= t.shape[-1] or math.prod(t.shape[1:-1]) <= 1)
    return t if fits else t.contiguous()


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, act):
        x = _as_map(x)
        y, stats = group_norm(x, groups, weight, bias, eps, act, return_stats=True)
        ctx.save_for_backward(x, stats, weight, bias)
        ctx.how = groups, act
        return y

    @staticmethod
    @once_differentiable        # a second derivative raises: without this it would be missing without a word
    def backward(ctx, g):
        x, stats, weight, bias = ctx.saved_tensors
        groups, act = ctx.how
        dx, dw, db = group_norm_backward(_as_map(g), x, stats, groups, weight, bias, act)
        return dx, None if weight is None else dw.to(weight.dtype), None if bias is None else db.to(bias.dtype), None, None, None


def group_norm_autograd(x, weight, bias, groups: int, eps: float = 1e-5, act: Optional[str] = None):
    """``group_norm`` under torch.autograd: gradients of x, weight and bias."""
    return _GroupNorm.apply(x, weight, bias, groups, eps, act)


# ------------------------------------------------------------- cross attention
def _stride(t):
    """Stride between the tokens of t [tokens, heads, D] or [requests, tokens,
    heads, D], None where they are not one run."""
    s = t.stride()
    if len(s) == 3:
        return s[0]
    b, n = t.shape[:2]
    return s[0] if n <= 1 else s[1] if b == 1 or s[0] == n * s[1] else None


def _rows(t, name, b, n, dim, dtype, dev):
    """t as rows of heads: [n, heads, dim], or [b, n, heads, dim] where b is not None."""
    s = t.stride()
    if b is None:
        (m, h, d), (step, wide, one) = t.shape, s
        fits = m == n
    else:
        (r, m, h, d), (far, step, wide, one) = t.shape, s
        fits = r == b and m == n
        if n <= 1:
            step = far
        elif b > 1 and far != n * step:
            fits = False
    if not fits or d != dim or one != 1 or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name}: a {dtype} tensor {(n, 'heads', dim) if b is None else (b, n, 'heads', dim)} on cuda:{dev} with unit stride in the "
                         f"last dimension and one run of tokens is needed, got {t.dtype} {tuple(t.shape)} with strides {s} on {t.device}")
    return svdq_heads(t.data_ptr(), step if n * (b or 1) > 1 else 0, wide if h > 1 else 0, h)


def _out(t, name, like, view, b, n, dim, dtype, dev):
    """An output like `like`, a new one where t is None, and its view for the call;
    view: like's."""
    if t is None:
        t = torch.empty_like(like)
        if t.stride() == like.stride():
            return t, svdq_heads(t.data_ptr(), view.token_stride, view.head_stride, view.heads)
        if not t.is_contiguous() and (t.stride(-1) != 1 or _stride(t) is None):
            t = like.new_empty(like.shape)
    elif t.shape != like.shape:
        raise ValueError(f"{name}: {tuple(like.shape)} is needed, got {tuple(t.shape)}")
    return t, _rows(t, name, b, n, dim, dtype, dev)


def _cross_desc(q, k, v, q_start, k_start, max_q, max_k, mask, scale, dev):
    """The call's descriptor, and (requests or None, tokens, states) as _rows takes them."""
    dims = q.dim(), k.dim(), v.dim()
    if dims == (4, 4, 4):
        if q_start is not None or k_start is not None or max_q is not None or max_k is not None:
            raise ValueError("q_start, k_start, max_q and max_k go with rows [tokens, heads, D]")
        b, n, _, dim = q.shape
        m = k.shape[1]
        requests, max_q, max_k, tokens, states, qs, ks = b, n, m, b * n, b * m, None, None
    elif dims == (3, 3, 3):
        if q_start is None or k_start is None or max_q is None or max_k is None:
            raise ValueError("rows [tokens, heads, D] need q_start, k_start, max_q and max_k")
        b, (n, _, dim), m = None, q.shape, k.shape[0]
        requests, tokens, states = q_start.numel() - 1, n, m
        if requests < 0:
            raise ValueError("q_start: [requests + 1] is needed, got no entry")
        qs, ks = kv._int32(q_start, "q_start", requests + 1, dev), kv._int32(k_start, "k_start", requests + 1, dev)
    else:
        raise ValueError(f"q, k, v: all [tokens, heads, D] or all [requests, tokens, heads, D] are needed, got {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    pm = None
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8) or mask.shape != k.shape[:-2] or not mask.is_contiguous() or mask.get_device() != dev:
            raise ValueError(f"mask: a contiguous bool tensor {tuple(k.shape[:-2])} on cuda:{dev} is needed, got {mask.dtype} {tuple(mask.shape)} on {mask.device}")
        pm = mask.data_ptr()
    d = svdq_cross_desc(requests, tokens, states, _size(dim, "head_dim"), _code(q.dtype), _size(max_q, "max_q"), _size(max_k, "max_k"),
                        (1.0 / math.sqrt(dim) if dim else 1.0) if scale is None else scale, qs, ks, pm)
    return d, b, n, m, dim


def cross_attention(q, k, v, q_start=None, k_start=None, max_q: Optional[int] = None, max_k: Optional[int] = None, mask=None,
                    scale: Optional[float] = None, out=None, ws=None, return_lse: bool = False, stream=None):
    """softmax(scale q k^T) v of queries over an encoder's keys and values.

    q [requests, tokens, heads, D], k and v [requests, states, k_heads, D]; or
    requests of different lengths one after the other: q [tokens, heads, D], rows
    q_start[r] .. q_start[r + 1] are request r's, k and v [states, k_heads, D]
    with k_start (int32 [requests + 1] both), and max_q, max_k, which bound a
    request's rows and states.  k_heads divides heads.  mask: bool or uint8, of
    k's shape without heads and D; false (0): the state is not seen.  scale: 1 /
    sqrt(D) by default.  A row that sees nothing gives zeros; a row of no
    request is not written.  Returns out, or (out, lse): lse fp32, q's shape
    without D."""
    with _on(stream, q):
        dev = kv._current_device()
        d, b, n, m, dim = _cross_desc(q, k, v, q_start, k_start, max_q, max_k, mask, scale, dev)
        dtype = q.dtype
        hq, hk, hv = _rows(q, "q", b, n, dim, dtype, dev), _rows(k, "k", b, m, dim, dtype, dev), _rows(v, "v", b, m, dim, dtype, dev)
        out, ho = _out(out, "out", q, hq, b, n, dim, dtype, dev)
        lse = q.new_empty(q.shape[:-1], dtype=torch.float32) if return_lse else None
        _call_with_workspace("svdq_cross_attention", q, ws, (d, hq.heads, hk.heads), (d, hq, hk, hv, ho, _address(lse)), _stream(q), False)
        return (out, lse) if return_lse else out


def cross_attention_backward(g, q, k, v, out, lse, q_start=None, k_start=None, max_q: Optional[int] = None, max_k: Optional[int] = None,
                             mask=None, scale: Optional[float] = None, dq=None, dk=None, dv=None, ws=None, stream=None):
    """Gradient of ``cross_attention`` from g (with respect to its output), its
    inputs, its output and lse.  Returns (dq, dk, dv).  States that the mask
    hides get zeros; rows and states of no request are not written."""
    with _on(stream, q):
        dev = kv._current_device()
        d, b, n, m, dim = _cross_desc(q, k, v, q_start, k_start, max_q, max_k, mask, scale, dev)
        dtype = q.dtype
        hq, ho, hg = _rows(q, "q", b, n, dim, dtype, dev), _rows(out, "out", b, n, dim, dtype, dev), _rows(g, "g", b, n, dim, dtype, dev)
        hk, hv = _rows(k, "k", b, m, dim, dtype, dev), _rows(v, "v", b, m, dim, dtype, dev)
        if lse.dtype is not torch.float32 or lse.shape != q.shape[:-1] or not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError(f"lse: a contiguous float32 tensor {tuple(q.shape[:-1])} on cuda:{dev} is needed, got {lse.dtype} {tuple(lse.shape)} on {lse.device}")
        dq, hdq = _out(dq, "dq", q, hq, b, n, dim, dtype, dev)
        dk, hdk = _out(dk, "dk", k, hk, b, m, dim, dtype, dev)
        dv, hdv = _out(dv, "dv", v, hv, b, m, dim, dtype, dev)
        _call_with_workspace("svdq_cross_attention_backward", q, ws, (d, hq.heads, hk.heads),
                             (d, hq, hk, hv, ho, lse.data_ptr(), hg, hdq, hdk, hdv), _stream(q), True)
        return dq, dk, dv


def _as_rows(t, group=1):
    """t as the library takes rows; what it does not (states that requests
    share by a stride of 0, a gradient that is broadcast over heads, strides that its
    32-bit offsets do not hold) is written out.  group: heads that share a key head."""
    step, h = _stride(t), t.stride(-2)
    fits = t.stride(-1) == 1 and step is not None and step >= 0 and step % 8 == 0 and h % 8 == 0 and (h >= t.shape[-1] or t.shape[-2] == 1) \
        and step < 1 << 23 and (group == 1 or h * group < 1 << 28) and t.data_ptr() % 16 == 0
    return t if fits else t.contiguous()


class _CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_start, k_start, max_q, max_k, mask, scale):
        group = q.shape[-2] // max(k.shape[-2], 1)
        q, k, v = _as_rows(q, group), _as_rows(k), _as_rows(v)
        out = None if q_start is None else q.new_zeros(q.shape)     # rows of no request are defined here
        out, lse = cross_attention(q, k, v, q_start, k_start, max_q, max_k, mask, scale, out=out, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, q_start, k_start, mask)
        ctx.how = max_q, max_k, scale, group
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        q, k, v, out, lse, q_start, k_start, mask = ctx.saved_tensors
        max_q, max_k, scale, group = ctx.how
        dq = dk = dv = None
        if q_start is not None:
            dq, dk, dv = (t.new_zeros(t.shape) for t in (q, k, v))
        grads = cross_attention_backward(_as_rows(g, group), q, k, v, out, lse, q_start, k_start, max_q, max_k, mask, scale, dq, dk, dv)
        return *grads, *[None] * 6


def cross_attention_autograd(q, k, v, q_start=None, k_start=None, max_q: Optional[int] = None, max_k: Optional[int] = None, mask=None,
                             scale: Optional[float] = None):
    """``cross_attention`` under torch.autograd: gradients of q, k and v.
    States shared by ``expand`` are taken (and written out); rows of no request
    are zeros."""
    return _CrossAttention.apply(q, k, v, q_start, k_start, max_q, max_k, mask, scale)
