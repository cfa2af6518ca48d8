"""An attention layer served over a 4-bit cache: two SVDQuant linears and, between
them, the operators of ``kv.py``.

    qkv = W_qkv x                               4-bit GEMM
    q, cache <- norm, rotation, quantization    one launch (KVCache.append)
    o = attention(q, cache)
    y = W_out o                                 4-bit GEMM

The step's tables (``kv.plan``) are shared by all layers of a model: plan once a
step, then call every layer.
"""
from __future__ import annotations

import torch

from . import kv
from .svdq import SVDQLinear, workspace_size


class SVDQAttention:
    """qkv: SVDQLinear K -> (q_heads + 2 k_heads) D, rows q heads, k heads, v
    heads; out: SVDQLinear q_heads D -> N; wq, wk: norm weights [D] or None; cos,
    sin: rotation tables [positions, D / 2]; cache: this layer's KVCache;
    causal, window: which keys a token sees (causal=False: all of its request,
    as in an image transformer, whose request is an image's tokens in one step).

    A call keeps nothing.  Its workspaces come from torch's allocator, under the
    current stream (or into the pool of the graph that is being captured), so
    that calls on several streams and captured ones do not share any.  What they
    do share is the cache; its order is the caller's."""

    def __init__(self, qkv: SVDQLinear, out: SVDQLinear, q_heads: int, cache: kv.KVCache, cos, sin, wq=None, wk=None,
                 eps: float = 1e-6, norm: bool = True, halves: bool = False, window: int = 0,
                 causal: bool = True):
        rows = (q_heads + 2 * cache.heads) * cache.head_dim
        if qkv.N != rows or out.K != q_heads * cache.head_dim:
            raise ValueError(f"{q_heads} query heads of {cache.head_dim} over {cache.heads} cache heads need a projection to {rows} "
                             f"and one from {q_heads * cache.head_dim}, got {qkv.N} and {out.K}")
        self.qkv, self.out, self.q_heads, self.cache = qkv, out, q_heads, cache
        self.how = dict(cos=cos, sin=sin, wq=wq, wk=wk, eps=eps, norm=norm, halves=halves)
        self.window, self.causal = window, causal

    def workspace(self, requests: int, tokens: int, max_q: int, max_kv: int):
        """A workspace for the attention of calls of these bounds, for callers
        that keep one (for one stream, and as long as a graph that holds it)."""
        return kv.attention_workspace(requests, tokens, self.q_heads, self.cache, max_q, max_kv)

    def _linear(self, linear: SVDQLinear, x):
        ws = torch.empty(workspace_size(linear.layer, x.shape[0]), dtype=torch.uint8, device=x.device)
        return linear.forward(x, ws=ws)

    def forward(self, x, step: kv.Plan, max_q: int, max_kv: int, ws=None):
        """x [tokens, K]: the new tokens of all requests, request after request;
        step: the plan that gave them their slots; max_q, max_kv: bounds on a
        request's new and cached tokens.  Rows past the last request's (a padded
        step) come out as the projection of zeros.  ws: the attention's workspace, or None
        for one of the call's own."""
        with kv._on(None, x):           # the linears, too, launch on the current device
            tokens, d, hq, hk = x.shape[0], self.cache.head_dim, self.q_heads, self.cache.heads
            rows = self._linear(self.qkv, x).view(tokens, hq + 2 * hk, d)
            q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
            self.cache.append(k, v, step.slots, q=q, q_out=q, positions=step.positions, **self.how)
            o = torch.zeros((tokens, hq, d), dtype=x.dtype, device=x.device)
            kv.attention(q, self.cache, step.block_table, step.q_start, step.kv_len, max_q, max_kv, causal=self.causal,
                         window=self.window, out=o, ws=ws)
            return self._linear(self.out, o.view(tokens, hq * d))

    __call__ = forward
