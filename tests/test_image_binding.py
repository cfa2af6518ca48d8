"""CPU tests of the binding of the group norm and the cross attention: what it
makes of its arguments before the library is called.  The tensors are the
host's; the device, the stream and the call are stand-ins."""
import contextlib

import pytest
import torch

from diffusion_smooth_group_amd import image, kv


@pytest.fixture
def calls(monkeypatch):
    """The library's calls: name and arguments.  They need a workspace of 64 bytes."""
    seen = []

    def fn(name):
        def call(*args):
            seen.append((name, args))
            if name.endswith("_workspace"):
                args[-1].value = 64
                return 0
            return 0 if args[-2] == 64 else 1
        return call
    monkeypatch.setattr(image, "_on", lambda stream, t: contextlib.nullcontext())
    monkeypatch.setattr(image, "_stream", lambda t: 17)
    monkeypatch.setattr(kv, "_current_device", lambda: -1)
    monkeypatch.setattr(image, "_fn", fn)
    return seen


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_maps_are_taken_as_they_lie(calls):
    x = half(3, 5, 7, 64)
    image.group_norm(x, 8)
    d, mx, my, stats, ws, size, stream = calls[-1][1]
    assert (d.samples, d.pixels, d.channels, d.groups, d.act, d.weight, d.bias) == (3, 35, 64, 8, 0, None, None)
    assert (mx.data, mx.sample_stride, mx.pixel_stride) == (x.data_ptr(), 35 * 64, 64) and stats is None and size == 64 and stream == 17
    wide = half(3, 5, 7, 160)
    view = wide[..., 32:96]
    y = image.group_norm(view, 8, act="gelu", out=view)
    d, mx, my, *_ = calls[-1][1]
    assert y is view and d.act == 2 and (mx.data, mx.sample_stride, mx.pixel_stride) == (view.data_ptr(), 35 * 160, 160) == (my.data, my.sample_stride, my.pixel_stride)
    rows = wide[:, ::2][..., :64]                       # rows of pixels with gaps: no single run
    with pytest.raises(ValueError, match="one run"):
        image.group_norm(rows, 8)
    image.group_norm(half(4, 64), 8)                    # one pixel a sample
    assert calls[-1][1][0].pixels == 1
    first = half(2, 64, 5, 7)
    with pytest.raises(ValueError, match="channels last"):
        image.group_norm(first.permute(0, 2, 3, 1), 8)
    last = first.to(memory_format=torch.channels_last)
    image.group_norm(last.permute(0, 2, 3, 1), 8)
    assert calls[-1][1][1].pixel_stride == 64


@pytest.mark.parametrize("change,match", [
    (dict(act="relu"), "act"), (dict(weight=half(32)), "weight"), (dict(weight=torch.zeros(64)), "weight"), (dict(bias=half(128)[::2]), "bias"),
    (dict(out=half(3, 5, 8, 64)), "out"), (dict(out=half(3, 5, 7, 64).bfloat16()), "out"), (dict(groups=1 << 31), "groups")])
def test_norm_refusals(calls, change, match):
    with pytest.raises(ValueError, match=match):
        image.group_norm(half(3, 5, 7, 64), **(dict(groups=8) | change))
    assert not calls
    with pytest.raises(ValueError):
        image.group_norm(half(64), 8)
    with pytest.raises(ValueError):
        image.group_norm(torch.zeros(2, 4, 64), 8)      # 32-bit maps


def test_norm_gradient(calls):
    x, stats = half(3, 5, 7, 64), torch.zeros(3, 8, 2)
    dx, dw, db = image.group_norm_backward(x, x, stats, 8, act="silu")
    assert dx.shape == x.shape and dw.shape == db.shape == (64,) and dw.dtype == db.dtype == torch.float32
    for bad in (torch.zeros(3, 8), torch.zeros(3, 8, 2, dtype=torch.float64), torch.zeros(3, 8, 4)[..., ::2]):
        with pytest.raises(ValueError, match="stats"):
            image.group_norm_backward(x, x, bad, 8)
    with pytest.raises(ValueError, match="g:"):
        image.group_norm_backward(half(3, 5, 6, 64), x, stats, 8)


def test_dense_rows(calls):
    qkv = half(2, 9, 12, 64)
    q, k, v = half(2, 5, 8, 64), qkv[:, :, 4:8], qkv[:, :, 8:]
    out, lse = image.cross_attention(q, k, v, return_lse=True, mask=torch.ones(2, 9, dtype=torch.bool))
    assert out.shape == q.shape and lse.shape == (2, 5, 8)
    d, hq, hk, hv, ho, at, ws, size, stream = calls[-1][1]
    assert (d.requests, d.tokens, d.states, d.head_dim, d.max_q, d.max_k, d.scale) == (2, 10, 18, 64, 5, 9, 0.125)
    assert d.q_start is None and d.k_start is None and d.mask is not None and at == lse.data_ptr() and stream == 17
    assert (hk.data, hk.token_stride, hk.head_stride, hk.heads) == (k.data_ptr(), 12 * 64, 64, 4) and hv.data == v.data_ptr()
    one = half(2, 1, 8, 64)                             # one token a request: its stride is the request's
    image.cross_attention(half(2, 3, 8, 64)[:, :1], k, v)
    assert calls[-1][1][1].token_stride == 3 * 8 * 64 and one.stride(0) == 8 * 64


def starts(*n):
    return torch.tensor(n, dtype=torch.int32)


def test_ragged_rows(calls):
    q, k = half(10, 8, 64), half(18, 4, 64)
    image.cross_attention(q, k, k, starts(0, 3, 10), starts(0, 9, 18), 7, 9, scale=2.0)
    d = calls[-1][1][0]
    assert (d.requests, d.tokens, d.states, d.max_q, d.max_k, d.scale) == (2, 10, 18, 7, 9, 2.0) and d.q_start and d.k_start


@pytest.mark.parametrize("args,change,match", [
    ("dense", dict(max_q=5), "go with rows"), ("dense", dict(q_start=starts(0, 1, 2)), "go with rows"), ("dense", dict(mask=torch.ones(2, 8, dtype=torch.bool)), "mask"),
    ("dense", dict(mask=torch.ones(2, 9)), "mask"), ("dense", dict(mask=torch.ones(9, 2, dtype=torch.bool)), "mask"), ("dense", dict(mask=torch.ones(2, 18, dtype=torch.bool)[:, ::2]), "mask"),
    ("dense", dict(k=half(3, 9, 4, 64)), "k:"), ("dense", dict(v=half(2, 8, 4, 64)), "v:"), ("dense", dict(v=half(2, 9, 4, 32)), "v:"),
    ("dense", dict(k=half(2, 9, 4, 64).bfloat16()), "k:"), ("dense", dict(k=half(1, 9, 4, 64).expand(2, -1, -1, -1)), "k:"),
    ("dense", dict(k=half(2, 18, 4, 64)[:, :9]), "k:"), ("dense", dict(q=half(2, 5, 8, 128)[..., ::2]), "q:"), ("dense", dict(out=half(2, 5, 4, 64)), "out"),
    ("dense", dict(k=half(18, 4, 64)), "all"), ("ragged", dict(q_start=None), "need"), ("ragged", dict(max_k=None), "need"),
    ("ragged", dict(q_start=torch.tensor([0, 3, 10])), "q_start"), ("ragged", dict(k_start=starts(0, 18)), "k_start"), ("ragged", dict(q_start=starts()), "q_start"),
    ("ragged", dict(max_q=1 << 31), "max_q"), ("ragged", dict(max_k=(1 << 32) + 8), "max_k"), ("ragged", dict(v=half(17, 4, 64)), "v:")])
def test_cross_refusals(calls, args, change, match):
    a = dict(q=half(2, 5, 8, 64), k=half(2, 9, 4, 64), v=half(2, 9, 4, 64)) if args == "dense" else \
        dict(q=half(10, 8, 64), k=half(18, 4, 64), v=half(18, 4, 64), q_start=starts(0, 3, 10), k_start=starts(0, 9, 18), max_q=7, max_k=9)
    with pytest.raises(ValueError, match=match):
        image.cross_attention(**(a | change))
    assert not calls


def test_gradient_outputs(calls):
    q, k, lse = half(2, 5, 8, 64), half(2, 9, 4, 64), torch.zeros(2, 5, 8)
    dq, dk, dv = image.cross_attention_backward(q, q, k, k, q, lse)
    assert dq.shape == q.shape and dk.shape == dv.shape == k.shape
    for bad in (torch.zeros(2, 5, 4), torch.zeros(2, 5, 8, dtype=torch.float64), torch.zeros(2, 8, 5).transpose(1, 2)):
        with pytest.raises(ValueError, match="lse"):
            image.cross_attention_backward(q, q, k, k, q, bad)
    with pytest.raises(ValueError, match="dk"):
        image.cross_attention_backward(q, q, k, k, q, lse, dk=half(2, 9, 8, 64))


def test_workspaces(calls):
    x = half(3, 5, 7, 64)
    image.group_norm(x, 8)
    assert [n for n, _ in calls] == ["svdq_group_norm", "svdq_group_norm_workspace", "svdq_group_norm"]
    ws = torch.zeros(64, dtype=torch.uint8)
    image.group_norm(x, 8, ws=ws)
    assert len(calls) == 4 and calls[-1][1][-3:-1] == (ws.data_ptr(), 64)
    with pytest.raises(kv.SvdqError):                   # a workspace that is too small stays the caller's matter
        image.group_norm(x, 8, ws=ws[:32])
    assert len(calls) == 5
    with pytest.raises(ValueError, match="ws"):
        image.group_norm(x, 8, ws=torch.zeros(128, dtype=torch.uint8)[::2])


def test_strides_that_32_bits_do_not_hold_are_written_out():
    """Where the library takes no such strides the autograd form makes a copy, as of any other it does not take (here of tensors
    without memory)."""
    far = lambda *strides: torch.empty_strided((1, 5, 8, 64), strides, dtype=torch.float16, device="meta")
    near, tokens, heads = far(0, 1 << 22, 64, 1), far(0, 1 << 23, 64, 1), far(0, 64, 1 << 26, 1)
    assert image._as_rows(near, 8) is near and image._as_rows(heads) is heads and image._as_rows(heads, 2) is heads
    assert image._as_rows(tokens).is_contiguous() and image._as_rows(heads, 4).is_contiguous()


@pytest.mark.parametrize("name", ["x", "k", "v", "weight", "bias"])
def test_layer_refuses_to_lose_a_gradient(monkeypatch, calls, name):
    """A 4-bit linear has none: where one would be asked of the layer, it says so, and does not give a result without it."""
    from diffusion_smooth_group_amd import attention_layer as layers
    monkeypatch.setattr(kv, "_on", lambda stream, t: contextlib.nullcontext())
    linear = type("Linear", (), {"N": 64, "K": 64})()
    monkeypatch.setattr(layers, "_linear", lambda linear, x: x)
    a = dict(x=half(2, 3, 3, 64), k=half(2, 9, 1, 64), v=half(2, 9, 1, 64), weight=half(64), bias=half(64))
    layer = layers.SVDQCrossAttention(linear, linear, 1, groups=8, weight=a["weight"], bias=a["bias"])
    assert layer(a["x"], a["k"], a["v"]).shape == a["x"].shape
    a[name].requires_grad_()
    n = len(calls)
    with pytest.raises(ValueError, match="no gradient"):
        layer(a["x"], a["k"], a["v"])
    assert len(calls) == n
    with torch.no_grad():
        assert layer(a["x"], a["k"], a["v"]).shape == a["x"].shape


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="GPU"):
        image.group_norm(half(2, 5, 64), 8)
    with pytest.raises(ValueError, match="GPU"):
        image.cross_attention(half(2, 5, 8, 64), half(2, 9, 4, 64), half(2, 9, 4, 64))
