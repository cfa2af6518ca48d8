"""ctypes binding of the 4-bit key/value cache operators (include/svdq_kv.h).

Argument marshalling only, like ``svdq.py``: torch tensors in and out, the
work is done by the library's kernels on the current (or the given) stream.
What runs between a QKV projection and the attention output:

    step = plan(past, fresh, table, free_pages, free_count, page_size, tokens)
    q = cache.append(k, v, step.slots, q=q, cos=cos, sin=sin, wq=wq, wk=wk, norm=True,
                     positions=step.positions)
    out = attention(q, cache, step.block_table, step.q_start, step.kv_len, max_q, max_kv)

Tensors of heads are [tokens, heads, D] with unit stride in D (views of a
fused QKV row are taken as they are).  A wrong argument raises ValueError
here or SvdqError with the library's status.

A call runs on the current stream.  With stream= (a torch stream or a raw
handle) it is as if made under ``torch.cuda.stream(stream)``: outputs and
workspaces that it allocates belong to that stream, too, so its memory goes to
nobody else while its kernels run.  All tensors of a call are on one device,
which need not be the current one.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import svdq as S
from .svdq import FMT_INT4_G64, FMT_MXFP4_G32, SvdqError  # noqa: F401  (part of this module's interface)

QK_NORM, QK_ROPE, QK_ROPE_HALVES = 1, 2, 4
ATTN_CAUSAL = 1
MAX_REQUESTS = 8192
GROUP = {FMT_MXFP4_G32: 32, FMT_INT4_G64: 64}
SCALE_DTYPE = {FMT_MXFP4_G32: torch.uint8, FMT_INT4_G64: torch.float16}

_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle, without building a Stream
_current_device = torch._C._cuda_getDevice         # the current device's index
_DTYPES = {torch.float16: S.F16, torch.bfloat16: S.BF16}
_P, _I64, _I32, _U, _F, _SZ = C.c_void_p, C.c_int64, C.c_int32, C.c_uint, C.c_float, C.c_size_t


class svdq_heads(C.Structure):
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64), ("heads", _I32)]


class svdq_qk_desc(C.Structure):
    _fields_ = [("tokens", _I64), ("head_dim", _I32), ("dtype", _I32), ("flags", _U), ("eps", _F), ("wq", _P),
                ("wk", _P), ("cos", _P), ("sin", _P), ("n_positions", _I64), ("positions", _P)]


class svdq_kv_cache(C.Structure):
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("n_pages", _I64),
                ("page_size", _I32), ("heads", _I32), ("head_dim", _I32), ("fmt", _I32)]


class svdq_attn_desc(C.Structure):
    _fields_ = [("requests", _I64), ("tokens", _I64), ("q_heads", _I32), ("dtype", _I32), ("max_q", _I32),
                ("max_kv", _I32), ("window", _I32), ("flags", _U), ("scale", _F), ("q_start", _P), ("kv_len", _P),
                ("block_table", _P), ("table_stride", _I64)]


_HP, _QP, _CP, _AP = C.POINTER(svdq_heads), C.POINTER(svdq_qk_desc), C.POINTER(svdq_kv_cache), C.POINTER(svdq_attn_desc)
_SIGS = {
    "svdq_qk_norm_rope": [_QP, _HP, _HP, _HP, _HP, _P],
    "svdq_qk_backward_workspace": [_QP, _I32, _I32, C.POINTER(_SZ)],
    "svdq_qk_norm_rope_backward": [_QP, _HP, _HP, _HP, _HP, _HP, _HP, _P, _P, _P, _SZ, _P],
    "svdq_kv_cache_size": [_I64, _I32, _I32, _I32, C.c_int, C.POINTER(_SZ), C.POINTER(_SZ)],
    "svdq_kv_append": [_QP, _HP, _HP, _HP, _HP, _CP, _P, _P],
    "svdq_kv_read": [_CP, _P, _I64, C.c_int, _HP, _HP, _P],
    "svdq_kv_plan": [_P, _P, _I64, _I32, _I64, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P],
    "svdq_kv_release": [_P, _I64, _I32, _P, _I64, _P, _P, _P, _I64, _P],
    "svdq_kv_attention_workspace": [_AP, _CP, C.POINTER(_SZ)],
    "svdq_kv_attention": [_AP, _HP, _CP, _HP, _P, _P, _SZ, _P],
}
_FN = {}


def _call(name, *args):
    fn = _FN.get(name)
    if fn is None:
        fn = getattr(S.lib_handle(), name)
        fn.argtypes, fn.restype = _SIGS[name], C.c_int
        _FN[name] = fn
    rc = fn(*args)
    if rc != 0:
        raise SvdqError(name, rc)


def _size(v, name, bits=32):
    """v, if the library's integer holds it (ctypes keeps the low bits of any)."""
    if -1 << bits - 1 <= v < 1 << bits - 1:
        return v
    raise ValueError(f"{name}: {v} is no {bits}-bit integer")


def _heads(t, name, tokens, dim, dtype, dev):
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if n != tokens or d != dim or s2 != 1 or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name}: a {dtype} tensor [{tokens}, heads, {dim}] on cuda:{dev} with unit stride in the last dimension is needed, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return svdq_heads(t.data_ptr(), s0 if n > 1 else 0, s1 if h > 1 else 0, h)


def _new(like):
    """An output of like's shape and type, and its view for the call."""
    t = torch.empty_like(like)
    s0, s1, _ = t.stride()
    n, h, _ = t.shape
    return t, svdq_heads(t.data_ptr(), s0 if n > 1 else 0, s1 if h > 1 else 0, h)


def _int32(t, name, n, dev):
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} entries on cuda:{dev} is needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, b, dev):
    if t.dim() != 2 or t.shape[0] != b:
        raise ValueError(f"block_table: [{b}, pages] is needed, got {tuple(t.shape)}")
    return _int32(t, "block_table", t.numel(), dev)


def _weight(w, name, dim, dtype, dev):
    if w is None:
        return None
    if w.dtype is not dtype or w.numel() != dim or not w.is_contiguous() or w.get_device() != dev:
        raise ValueError(f"{name}: a contiguous {dtype} tensor of {dim} on cuda:{dev} is needed")
    return w.data_ptr()


def _scratch(ws, dev):
    """Address and bytes of a workspace."""
    if not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError(f"ws: a contiguous tensor on cuda:{dev} is needed, got strides {ws.stride()} on {ws.device}")
    n = ws.numel() * ws.element_size()
    return ws.data_ptr() if n else None, n


def _code(dtype):
    c = _DTYPES.get(dtype)
    if c is None:
        raise ValueError(f"float16 or bfloat16 rows are needed, got {dtype}")
    return c


_HERE = contextlib.nullcontext()


def _on(stream, t):
    """The context of a call: `stream` is the current stream in it, for the
    allocator as for the launch, and the device of t, a tensor of the call, the
    current device, to which a launch goes."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"GPU tensors are needed, got one on {t.device}")
    if stream is None:
        return _HERE if index == _current_device() else torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device) if stream else torch.cuda.default_stream(t.device)
    return torch.cuda.stream(stream)


def _stream(t):
    return _raw_stream(t.get_device())


def _desc(tokens, dim, dtype, cos, sin, wq, wk, eps, norm, halves, positions, dev):
    flags = pq = pk = pc = ps = pp = n = 0
    if norm:
        flags, pq, pk = QK_NORM, _weight(wq, "wq", dim, dtype, dev), _weight(wk, "wk", dim, dtype, dev)
    if cos is not None:
        flags |= QK_ROPE | QK_ROPE_HALVES if halves else QK_ROPE
        n = cos.shape[0]
        f32, shape = torch.float32, (n, dim // 2)
        if sin is None or cos.dtype is not f32 or sin.dtype is not f32 or cos.shape != shape or sin.shape != shape \
                or not (cos.is_contiguous() and sin.is_contiguous() and cos.get_device() == sin.get_device() == dev):
            raise ValueError(f"cos, sin: contiguous float32 tables [positions, {dim} / 2] on cuda:{dev} are needed")
        pc, ps = cos.data_ptr(), sin.data_ptr()
        if positions is not None:
            pp = _int32(positions, "positions", tokens, dev)
    elif sin is not None:
        raise ValueError("cos and sin go together")
    return svdq_qk_desc(tokens, dim, _code(dtype), flags, eps, pq, pk, pc, ps, n, pp)


# ------------------------------------------------------------ norm and rotation
def qk_norm_rope(q, k, cos=None, sin=None, wq=None, wk=None, eps: float = 1e-6, norm: bool = True, halves: bool = False,
                 positions=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q and k (``norm``; weights wq, wk [D], None for
    ones) and rotation by the tables cos, sin [positions, D / 2] (None: no
    rotation), at positions [tokens] (int32, None: 0, 1, ...).  halves: pairs
    (i, i + D/2), else (2i, 2i + 1).  Returns (q_out, k_out); q_out=q, k_out=k
    work in place."""
    with _on(stream, q):
        dev = _current_device()
        tokens, _, dim = q.shape
        dtype = q.dtype
        d = _desc(tokens, dim, dtype, cos, sin, wq, wk, eps, norm, halves, positions, dev)
        hq, hk = _heads(q, "q", tokens, dim, dtype, dev), _heads(k, "k", tokens, dim, dtype, dev)
        if q_out is None:
            q_out, hqo = _new(q)
        else:
            hqo = _heads(q_out, "q_out", tokens, dim, dtype, dev)
        if k_out is None:
            k_out, hko = _new(k)
        else:
            hko = _heads(k_out, "k_out", tokens, dim, dtype, dev)
        _call("svdq_qk_norm_rope", d, hq, hk, hqo, hko, _stream(q))
        return q_out, k_out


def qk_norm_rope_backward(gq, gk, q, k, cos=None, sin=None, wq=None, wk=None, eps: float = 1e-6, norm: bool = True,
                          halves: bool = False, positions=None, dq=None, dk=None, ws=None, stream=None):
    """Gradient of ``qk_norm_rope`` from gq, gk (with respect to its outputs)
    and its inputs.  Returns (dq, dk, dwq, dwk), the weight gradients fp32 [D]
    (zero without ``norm``)."""
    with _on(stream, q):
        dev = _current_device()
        tokens, _, dim = q.shape
        dtype = q.dtype
        d = _desc(tokens, dim, dtype, cos, sin, wq, wk, eps, norm, halves, positions, dev)
        h = [_heads(t, n, tokens, dim, dtype, dev) for t, n in ((q, "q"), (k, "k"), (gq, "gq"), (gk, "gk"))]
        for t, like, n in ((dq, q, "dq"), (dk, k, "dk")):
            h.append(_new(like) if t is None else (t, _heads(t, n, tokens, dim, dtype, dev)))
        (dq, hdq), (dk, hdk) = h[4:]
        dwq, dwk = dw = q.new_empty((2, dim), dtype=torch.float32).unbind()
        if ws is None:
            need = _SZ(0)
            _call("svdq_qk_backward_workspace", d, q.shape[1], k.shape[1], need)
            ws = q.new_empty(need.value, dtype=torch.uint8)
        _call("svdq_qk_norm_rope_backward", d, *h[:4], hdq, hdk, dwq.data_ptr(), dwk.data_ptr(), *_scratch(ws, dev),
              _stream(q))
        return dq, dk, *dw


def _rows(g):
    """g as the library takes rows; a gradient that is the same for all heads
    (stride 0, from a sum over heads) is written out."""
    t, h, d = g.stride()
    fits = d == 1 and t >= 0 and t % 8 == 0 and h % 8 == 0 and (h >= g.shape[2] or g.shape[1] == 1) and g.data_ptr() % 16 == 0
    return g if fits else g.contiguous()


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, eps, halves, positions, norm):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.how = eps, halves, norm
        return qk_norm_rope(q, k, cos, sin, wq, wk, eps, norm, halves, positions)

    @staticmethod
    @once_differentiable        # a second derivative raises: without this it would be missing without a word
    def backward(ctx, gq, gk):
        q, k, wq, wk, cos, sin, positions = ctx.saved_tensors
        eps, halves, norm = ctx.how
        dq, dk, dwq, dwk = qk_norm_rope_backward(_rows(gq), _rows(gk), q, k, cos, sin, wq, wk, eps, norm, halves, positions)
        return dq, dk, None if wq is None else dwq.to(wq.dtype), None if wk is None else dwk.to(wk.dtype), *[None] * 6


def qk_norm_rope_autograd(q, k, wq, wk, cos, sin, eps: float = 1e-6, halves: bool = False, positions=None, norm: bool = True):
    """``qk_norm_rope`` under torch.autograd: gradients of q, k, wq and wk
    (zero for the weights without ``norm``).  They can not be differentiated
    again (torch raises an error)."""
    return _QKNormRope.apply(q, k, wq, wk, cos, sin, eps, halves, positions, norm)


# ----------------------------------------------------------------------- cache
class KVCache:
    """The paged 4-bit cache of one layer: codes [pages, heads, page_size, D / 2]
    and scales [pages, heads, page_size, D / G] of K and of V."""

    def __init__(self, n_pages: int, page_size: int, heads: int, head_dim: int, fmt: int, device="cuda"):
        code, scale = _SZ(0), _SZ(0)
        _call("svdq_kv_cache_size", _size(n_pages, "n_pages", 64), _size(page_size, "page_size"), _size(heads, "heads"),
              _size(head_dim, "head_dim"), fmt, code, scale)
        shape = (n_pages, heads, page_size)
        codes = [torch.zeros((*shape, head_dim // 2), dtype=torch.uint8, device=device) for _ in "kv"]
        scales = [torch.zeros((*shape, head_dim // GROUP[fmt]), dtype=SCALE_DTYPE[fmt], device=device) for _ in "kv"]
        self._hold(codes[0], scales[0], codes[1], scales[1], fmt)

    @classmethod
    def wrap(cls, k_codes, k_scales, v_codes, v_scales, fmt):
        """A cache in buffers that the caller has.  fmt: FMT_MXFP4_G32,
        FMT_INT4_G64, or "mxfp4_g32", "int4_g64"."""
        fmt = S.FMT_CODES.get(fmt, fmt)
        if fmt not in GROUP or k_codes.dim() != 4:
            raise ValueError(f"codes [pages, heads, page_size, D / 2] of a 4-bit format are needed, got {fmt!r} {tuple(k_codes.shape)}")
        shape, dim = k_codes.shape[:3], 2 * k_codes.shape[3]
        for t, kind, last in ((k_codes, torch.uint8, dim // 2), (v_codes, torch.uint8, dim // 2),
                              (k_scales, SCALE_DTYPE[fmt], dim // GROUP[fmt]), (v_scales, SCALE_DTYPE[fmt], dim // GROUP[fmt])):
            if not t.is_cuda or t.device != k_codes.device or not t.is_contiguous() or t.dtype is not kind or t.shape != (*shape, last):
                raise ValueError(f"a contiguous {kind} GPU tensor {(*shape, last)} is needed, all four on one device, "
                                 f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        self = cls.__new__(cls)
        self._hold(k_codes, k_scales, v_codes, v_scales, fmt)
        return self

    def _hold(self, k_codes, k_scales, v_codes, v_scales, fmt):
        self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.fmt = k_codes, k_scales, v_codes, v_scales, fmt
        self.n_pages, self.heads, self.page_size = k_codes.shape[:3]
        self.head_dim = 2 * k_codes.shape[3]
        self.device, self.index = k_codes.device, k_codes.get_device()
        self.c = svdq_kv_cache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                               self.n_pages, self.page_size, self.heads, self.head_dim, fmt)

    def _here(self, dev):
        if self.index != dev:
            raise ValueError(f"the cache is on {self.device}, the call's tensors on cuda:{dev}")

    def append(self, k, v, slots, q=None, cos=None, sin=None, wq=None, wk=None, eps: float = 1e-6, norm: bool = False,
               halves: bool = False, positions=None, q_out=None, stream=None):
        """Quantizes k and v [tokens, heads, D] into slots [tokens] (int32, a
        negative one is skipped).  With norm and / or cos, sin: k is normed and
        rotated on the way (and q into q_out, which is returned)."""
        with _on(stream, k):
            dev = _current_device()
            self._here(dev)
            tokens, _, dim = k.shape
            d = _desc(tokens, dim, k.dtype, cos, sin, wq, wk, eps, norm, halves, positions, dev)
            hq = ho = None
            if q is not None:
                hq = _heads(q, "q", tokens, dim, k.dtype, dev)
                if q_out is None:
                    q_out, ho = _new(q)
                else:
                    ho = _heads(q_out, "q_out", tokens, dim, k.dtype, dev)
            _call("svdq_kv_append", d, hq, _heads(k, "k", tokens, dim, k.dtype, dev), _heads(v, "v", tokens, dim, k.dtype, dev), ho, self.c,
                  _int32(slots, "slots", tokens, dev), _stream(k))
            return q_out

    def read(self, slots, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
        """(k, v) [len(slots), heads, D]: the cached values of the slots, zero
        for slots outside the cache."""
        with _on(stream, slots):
            dev = _current_device()
            self._here(dev)
            n = slots.numel()
            code, at, hd = _code(dtype), _int32(slots, "slots", n, dev), self.head_dim
            if k_out is None:
                k_out = self.k_codes.new_empty((n, self.heads, hd), dtype=dtype)
            if v_out is None:
                v_out = self.k_codes.new_empty((n, self.heads, hd), dtype=dtype)
            _call("svdq_kv_read", self.c, at, n, code, _heads(k_out, "k_out", n, hd, dtype, dev), _heads(v_out, "v_out", n, hd, dtype, dev),
                  _stream(slots))
            return k_out, v_out


# ------------------------------------------------------------------- step tables
class Plan(NamedTuple):
    block_table: torch.Tensor   # [requests, pages], the caller's, new pages entered
    q_start: torch.Tensor       # [requests + 1]
    kv_len: torch.Tensor        # [requests]
    slots: torch.Tensor         # [tokens]
    positions: torch.Tensor     # [tokens]
    free_count: torch.Tensor    # [1] pages left
    missing: torch.Tensor       # [1] pages that were wanted and not there


def plan(past, fresh, block_table, free_pages, free_count, page_size: int, tokens: int, stream=None) -> Plan:
    """Block tables, slots and positions of a step: past [requests] cached
    tokens, fresh [requests] new ones, pages from the end of free_pages
    (free_count [1] of them are free).  tokens: length of the slot map, at
    least the sum of fresh (the rest is -1)."""
    with _on(stream, past):
        dev = _current_device()
        b = past.numel()
        out = past.new_empty(2 * b + 3 + 2 * tokens)
        at = out.data_ptr()
        cuts = (b + 1, b, tokens, tokens, 1, 1)
        q_start, kv_len, slots, positions, left, missing = out.split(cuts)
        p, ptr = [], at
        for n in cuts:
            p.append(ptr)
            ptr += 4 * n
        room = free_pages.numel()
        _call("svdq_kv_plan", _int32(past, "past", b, dev), _int32(fresh, "fresh", b, dev), b,
              _size(page_size, "page_size"), tokens,
              _int32(free_pages, "free_pages", room, dev), _int32(free_count, "free_count", 1, dev), room, _table(block_table, b, dev),
              block_table.shape[1], *p, _stream(past))
        return Plan(block_table, q_start, kv_len, slots, positions, left, missing)


def release(done, block_table, kv_len, free_pages, free_count, page_size: int, stream=None):
    """Gives the pages of the requests with done != 0 back to free_pages (in
    place: free_pages, free_count, block_table and kv_len)."""
    with _on(stream, done):
        dev = _current_device()
        b = done.numel()
        room = free_pages.numel()
        _call("svdq_kv_release", _int32(done, "done", b, dev), b, _size(page_size, "page_size"), _table(block_table, b, dev), block_table.shape[1],
              _int32(kv_len, "kv_len", b, dev), _int32(free_pages, "free_pages", room, dev), _int32(free_count, "free_count", 1, dev), room,
              _stream(done))


# --------------------------------------------------------------------- attention
def attention_workspace_size(requests: int, tokens: int, q_heads: int, cache: KVCache, max_q: int, max_kv: int) -> int:
    """Bytes of workspace that ``attention`` calls with at most these requests,
    tokens, max_q and max_kv need."""
    d = svdq_attn_desc(_size(requests, "requests", 64), _size(tokens, "tokens", 64), _size(q_heads, "q_heads"), S.BF16,
                       _size(max_q, "max_q"), _size(max_kv, "max_kv"), 0, ATTN_CAUSAL, 1.0)
    need = _SZ(0)
    _call("svdq_kv_attention_workspace", d, cache.c, need)
    return need.value


def attention_workspace(requests: int, tokens: int, q_heads: int, cache: KVCache, max_q: int, max_kv: int,
                        device=None) -> torch.Tensor:
    """A workspace for ``attention`` calls of these bounds and smaller ones, on the cache's
    device.  One stream at a time may use it."""
    return torch.empty(attention_workspace_size(requests, tokens, q_heads, cache, max_q, max_kv), dtype=torch.uint8,
                       device=cache.device if device is None else device)


def attention(q, cache: KVCache, block_table, q_start, kv_len, max_q: int, max_kv: int, causal: bool = True, window: int = 0,
              scale: Optional[float] = None, out=None, ws=None, return_lse: bool = False, stream=None):
    """softmax(scale q k^T) v over the cached tokens, request by request: rows
    q_start[r] .. q_start[r + 1] of q [tokens, q_heads, D] are request r's, the
    last of them at position kv_len[r] - 1.  causal: keys up to the row's
    position; window > 0: only the last `window` of them.  max_q, max_kv bound
    the rows and cached tokens of a request.  scale: 1 / sqrt(D) by default.
    A row that sees nothing gives zeros; a row of no request is not written.
    Returns out, or (out, lse)."""
    with _on(stream, q):
        dev = _current_device()
        cache._here(dev)
        tokens, hq, dim = q.shape
        if dim != cache.head_dim:
            raise ValueError(f"q: heads of {dim} over a cache of heads of {cache.head_dim}")
        b = kv_len.numel()
        hin = _heads(q, "q", tokens, dim, q.dtype, dev)
        if out is None:
            out, hout = _new(q)
        else:
            hout = _heads(out, "out", tokens, dim, q.dtype, dev)
        lse = q.new_empty((tokens, hq), dtype=torch.float32) if return_lse else None
        d = svdq_attn_desc(b, tokens, hq, _code(q.dtype), _size(max_q, "max_q"), _size(max_kv, "max_kv"), _size(window, "window"),
                           ATTN_CAUSAL if causal else 0,
                           1.0 / math.sqrt(dim) if scale is None else scale, _int32(q_start, "q_start", b + 1, dev),
                           _int32(kv_len, "kv_len", b, dev), _table(block_table, b, dev), block_table.shape[1])
        if ws is None:
            need = _SZ(0)
            _call("svdq_kv_attention_workspace", d, cache.c, need)
            ws = q.new_empty(need.value, dtype=torch.uint8)
        _call("svdq_kv_attention", d, hin, cache.c, hout,
              None if lse is None else lse.data_ptr(), *_scratch(ws, dev), _stream(q))
        return (out, lse) if return_lse else out
