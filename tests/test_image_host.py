"""CPU tests of the C ABI of the group norm and the cross attention: exported
symbols, sizes and the refusal of every wrong argument before anything is
launched."""
import ctypes as C
import os
import re

import pytest

from diffusion_smooth_group_amd import image, kv
from diffusion_smooth_group_amd import svdq as S

HDR = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "svdq_image.h")
OK, INVALID, SHAPE, UNSUPPORTED, CAPACITY = 0, 1, 2, 3, 4
P = C.c_void_p(4096)         # aligned, never dereferenced: every call here is refused or has nothing to do
ODD = C.c_void_p(4104)


def fn(name):
    f = getattr(S.lib_handle(), name)
    f.argtypes, f.restype = image._SIGS[name], C.c_int
    return f


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"^svdq_status\s+(svdq_\w+)\s*\(", open(HDR).read(), re.M))
    assert names == set(image._SIGS)
    for n in names:
        assert hasattr(S.lib_handle(), n)


# ------------------------------------------------------------------ group norm
def norm(**kw):
    d = image.svdq_norm_desc(2, 100, 320, 32, S.BF16, 1, 1e-5, P, P)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fmap(data=P, sample=320 * 10 ** 6, pixel=320):
    return image.svdq_map(data, sample, pixel)


BAD_NORM = [(dict(samples=-1), INVALID), (dict(pixels=-1), INVALID), (dict(pixels=0), INVALID), (dict(channels=0), INVALID),
            (dict(groups=0), INVALID), (dict(dtype=2), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(eps=-1.0), INVALID),
            (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(channels=324), SHAPE), (dict(groups=33), SHAPE),
            (dict(channels=64, groups=128), SHAPE), (dict(weight=ODD), SHAPE), (dict(bias=ODD), SHAPE),
            (dict(channels=8200, groups=1), UNSUPPORTED), (dict(samples=1 << 31), UNSUPPORTED), (dict(samples=1 << 62, pixels=1 << 62), UNSUPPORTED),
            (dict(samples=1 << 30, pixels=1 << 30), UNSUPPORTED), (dict(samples=1 << 26), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", BAD_NORM)
def test_norm_desc_refusals(change, status):
    d, size = norm(**change), C.c_size_t()
    assert fn("svdq_group_norm_workspace")(d, size) == status
    assert fn("svdq_group_norm_backward_workspace")(d, size) == status
    assert fn("svdq_group_norm")(d, fmap(), fmap(), None, P, 1 << 40, None) == status
    assert fn("svdq_group_norm_backward")(d, fmap(), fmap(), P, fmap(), P, P, P, 1 << 40, None) == status


def test_norm_operand_refusals():
    big = norm(pixels=1 << 16)
    size = C.c_size_t()
    assert fn("svdq_group_norm_workspace")(big, None) == INVALID
    assert fn("svdq_group_norm_workspace")(big, size) == OK and size.value > 0
    need = size.value
    f, b = fn("svdq_group_norm"), fn("svdq_group_norm_backward")
    assert f(None, fmap(), fmap(), None, P, need, None) == INVALID
    assert f(big, None, fmap(), None, P, need, None) == INVALID
    assert f(big, fmap(), None, None, P, need, None) == INVALID
    for bad, status in ((fmap(data=None), INVALID), (fmap(data=ODD), SHAPE), (fmap(pixel=324), SHAPE), (fmap(pixel=312), SHAPE),
                        (fmap(pixel=-320), SHAPE), (fmap(sample=4), SHAPE), (fmap(sample=-320), SHAPE)):
        assert f(big, bad, fmap(), None, P, need, None) == status
        assert f(big, fmap(), bad, None, P, need, None) == status
        for at in range(3):
            maps = [fmap(), fmap(), fmap()]
            maps[at] = bad
            assert b(big, maps[0], maps[1], P, maps[2], P, P, P, 1 << 40, None) == status
    for lies_on_itself in (fmap(sample=0), fmap(sample=320), fmap(sample=320 * ((1 << 16) - 1)), fmap(sample=640, pixel=320)):
        assert f(big, fmap(), lies_on_itself, None, P, need, None) == SHAPE
        assert b(big, fmap(), fmap(), P, lies_on_itself, P, P, P, 1 << 40, None) == SHAPE
    assert f(big, fmap(), fmap(), None, None, need, None) == INVALID
    assert f(big, fmap(), fmap(), None, P, need - 1, None) == CAPACITY
    assert f(big, fmap(), fmap(), None, ODD, need, None) == INVALID
    assert b(big, fmap(), fmap(), None, fmap(), P, P, P, 1 << 40, None) == INVALID
    assert fn("svdq_group_norm_backward_workspace")(big, size) == OK
    assert b(big, fmap(), fmap(), P, fmap(), P, P, P, size.value - 1, None) == CAPACITY


@pytest.mark.parametrize("samples,pixels,channels,groups", [(1, 64, 1280, 32), (3, 1, 64, 8), (2, 16384, 320, 32), (1, 1 << 20, 8, 1),
                                                            (7, 1023, 960, 32), (1, 5000, 8192, 8192), (300, 70000, 16, 4)])
def test_norm_sizes(samples, pixels, channels, groups):
    d, size, back = norm(samples=samples, pixels=pixels, channels=channels, groups=groups, weight=None, bias=None), C.c_size_t(), C.c_size_t()
    assert fn("svdq_group_norm_workspace")(d, size) == OK and fn("svdq_group_norm_backward_workspace")(d, back) == OK
    # at most one chunk for each of 256 workgroups and sample: partial sums of groups (and channels)
    chunks = max(256, samples)
    assert size.value <= 8 * chunks * groups and back.value <= 8 * chunks * (groups + channels)


def test_norm_without_samples():
    d, size = norm(samples=0, pixels=0), C.c_size_t(7)
    assert fn("svdq_group_norm_workspace")(d, size) == OK and size.value == 0
    assert fn("svdq_group_norm")(d, fmap(data=None), fmap(data=None), None, None, 0, None) == OK
    assert fn("svdq_group_norm_backward")(d, fmap(data=None), fmap(data=None), None, fmap(data=None), None, None, None, 0, None) == OK


# ------------------------------------------------------------- cross attention
def cross(**kw):
    d = image.svdq_cross_desc(2, 200, 154, 64, S.BF16, 100, 77, 0.125, None, None, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def heads(n=8, token=1024, head=64, data=P):
    return kv.svdq_heads(data, token, head, n)


BAD_CROSS = [(dict(requests=-1), INVALID), (dict(tokens=-1), INVALID), (dict(states=-1), INVALID), (dict(dtype=2), INVALID), (dict(max_q=-1), INVALID),
             (dict(max_k=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(head_dim=0), SHAPE),
             (dict(head_dim=-8), SHAPE), (dict(head_dim=68), SHAPE), (dict(head_dim=136), UNSUPPORTED), (dict(tokens=199), SHAPE), (dict(states=155), SHAPE),
             (dict(max_q=99), SHAPE), (dict(max_k=78), SHAPE), (dict(tokens=(1 << 31) - 512, q_start=P), UNSUPPORTED),
             (dict(states=(1 << 31) - 512, k_start=P), UNSUPPORTED), (dict(requests=1 << 30, q_start=P, k_start=P), UNSUPPORTED),
             (dict(states=(1 << 30) + 1, max_k=(1 << 30) + 1, k_start=P), UNSUPPORTED),
             (dict(requests=1 << 20, tokens=1 << 30, max_q=1 << 30, q_start=P, k_start=P), UNSUPPORTED)]


def run_forward(d, q=None, k=None, v=None, out=None, lse=None, ws=P, size=1 << 50):
    return fn("svdq_cross_attention")(d, q or heads(), k or heads(4), v or heads(4), out or heads(), lse, ws, size, None)


def run_backward(d, ws=P, size=1 << 50, lse=P, **other):
    o = dict(q=heads(), k=heads(4), v=heads(4), out=heads(), g=heads(), dq=heads(), dk=heads(4), dv=heads(4)) | other
    return fn("svdq_cross_attention_backward")(d, o["q"], o["k"], o["v"], o["out"], lse, o["g"], o["dq"], o["dk"], o["dv"], ws, size, None)


@pytest.mark.parametrize("change,status", BAD_CROSS)
def test_cross_desc_refusals(change, status):
    d, size = cross(**change), C.c_size_t()
    assert fn("svdq_cross_attention_workspace")(d, 8, 4, size) == status
    assert fn("svdq_cross_attention_backward_workspace")(d, 8, 4, size) == status
    assert run_forward(d) == status
    assert run_backward(d) == status


def test_cross_operand_refusals():
    d, size = cross(), C.c_size_t()
    for name in ("svdq_cross_attention_workspace", "svdq_cross_attention_backward_workspace"):
        f = fn(name)
        assert f(None, 8, 4, size) == INVALID and f(d, 8, 4, None) == INVALID
        assert f(d, 0, 4, size) == INVALID and f(d, 8, 0, size) == INVALID and f(d, 8, 3, size) == SHAPE
    assert run_forward(d, k=heads(3), v=heads(3)) == SHAPE
    assert run_forward(d, v=heads(2)) == SHAPE
    assert run_forward(d, out=heads(4)) == SHAPE
    bad = [(dict(data=None), INVALID), (dict(data=ODD), SHAPE), (dict(token=1028), SHAPE), (dict(token=-8), SHAPE), (dict(head=60), SHAPE), (dict(head=56), SHAPE)]
    for change, status in bad:
        for name, n in (("q", 8), ("k", 4), ("v", 4), ("out", 8)):
            assert run_forward(d, **{name: heads(n, **change)}) == status, name
        for name, n in (("q", 8), ("k", 4), ("v", 4), ("out", 8), ("g", 8), ("dq", 8), ("dk", 4), ("dv", 4)):
            assert run_backward(d, **{name: heads(n, **change)}) == status, name
    for name in ("q", "out", "g", "dq"):
        assert run_backward(d, **{name: heads(4)}) == SHAPE
    for name in ("v", "dk", "dv"):
        assert run_backward(d, **{name: heads(8)}) == SHAPE
    for stride in (0, 56):              # results whose rows lie on each other
        assert run_forward(d, out=heads(8, token=stride)) == SHAPE
        for name, n in (("dq", 8), ("dk", 4), ("dv", 4)):
            assert run_backward(d, **{name: heads(n, token=stride)}) == SHAPE
    # strides whose offsets 32 bits do not hold
    far = 1 << 23
    assert run_forward(d, k=heads(4, token=far)) == UNSUPPORTED and run_forward(d, v=heads(4, token=far)) == UNSUPPORTED
    for name in "qg":
        assert run_backward(d, **{name: heads(8, token=far)}) == UNSUPPORTED
        assert run_backward(d, **{name: heads(8, head=1 << 27)}) == UNSUPPORTED
    assert run_backward(d, lse=None) == INVALID


def test_cross_workspaces():
    size = C.c_size_t()
    d = cross(requests=1, tokens=1, max_q=1, states=100000, max_k=100000)
    assert fn("svdq_cross_attention_workspace")(d, 8, 4, size) == OK and size.value > 0
    need = size.value
    assert run_forward(d, ws=None) == INVALID and run_forward(d, size=need - 1) == CAPACITY and run_forward(d, ws=ODD, size=need) == INVALID
    assert fn("svdq_cross_attention_backward_workspace")(d, 8, 4, size) == OK and size.value > 0
    need = size.value
    assert run_backward(d, ws=None) == INVALID and run_backward(d, size=need - 1) == CAPACITY and run_backward(d, ws=ODD, size=need) == INVALID
    assert fn("svdq_cross_attention_workspace")(cross(requests=64, tokens=64 * 4096, states=64 * 77, max_q=4096), 8, 4, size) == OK and size.value == 0


@pytest.mark.parametrize("requests,max_q,max_k,hq,hk,dim", [(1, 1, 1, 1, 1, 8), (64, 1, 4096, 32, 8, 128), (1, 4608, 4096, 24, 24, 128), (5, 1023, 2049, 32, 8, 128),
                                                            (1, 1, 1 << 30, 1, 1, 128), (1, 1 << 22, 77, 8, 8, 64), (300, 3, 0, 4, 4, 64), (2, 0, 9, 4, 4, 64)])
def test_cross_sizes(requests, max_q, max_k, hq, hk, dim):
    """Partial rows are as many as fill the chip, not more the longer a call is."""
    d, size = cross(requests=requests, tokens=requests * max_q, states=requests * max_k, max_q=max_q, max_k=max_k, head_dim=dim), C.c_size_t()
    assert fn("svdq_cross_attention_workspace")(d, hq, hk, size) == OK
    cus = 256
    assert size.value <= 4 * (dim + 2) * 2 * cus * 128
    assert fn("svdq_cross_attention_backward_workspace")(d, hq, hk, size) == OK
    assert size.value <= 4 * (requests * max_q * hq + 64 + dim * 2 * cus * 128 + 64 + 2 * dim * 2 * cus * 128)


def test_cross_with_nothing_to_do():
    assert run_forward(cross(requests=0, tokens=0, states=0), ws=None, size=0) == OK
    assert run_backward(cross(requests=0, tokens=0, states=0), ws=None, size=0) == OK
    assert run_forward(cross(tokens=0, max_q=0), ws=None, size=0, q=heads(data=None), out=heads(data=None)) == OK


# (token, head) strides of results of 64 columns: the first head of a later token is another head of token 0, or half of it, or the last
# token's is
@pytest.mark.parametrize("token,head", [(64, 64), (128, 256), (64, 128), (96, 64), (64, 64 * 153), (192, 128)])
@pytest.mark.parametrize("name", ["out", "dq", "dk", "dv"])
def test_cross_results_whose_heads_lie_on_other_rows(name, token, head):
    d, n = cross(), 8 if name in ("out", "dq") else 4
    bad = heads(n, token=token, head=head)
    if name == "out":
        assert run_forward(d, out=bad, ws=None) == SHAPE
    else:
        assert run_backward(d, **{name: bad}) == SHAPE


def test_cross_results_in_any_order_of_dimensions():
    """What views of dense tensors look like passes the check (the workspace's, behind it, refuses the call)."""
    d = cross(requests=1, tokens=300, states=100000, max_q=300, max_k=100000)
    size = C.c_size_t()
    assert fn("svdq_cross_attention_backward_workspace")(d, 8, 4, size) == OK and size.value > 0
    for token, head in ((512, 64), (64, 64 * 100000), (2 * 512, 2 * 64), (96, 96 * 100000), (4 * 64, 64)):
        for name, n in (("dq", 8), ("dk", 4), ("dv", 4)):
            if n == 8 and token == 256:
                continue                # eight heads in the place of four
            assert run_backward(d, ws=None, **{name: heads(n, token=token, head=head)}) == INVALID, (name, token, head)
    one = cross(requests=1, tokens=1, states=100000, max_q=1, max_k=100000)
    assert run_forward(one, ws=None, out=heads(8, token=0, head=64)) == INVALID        # one token: its stride says nothing


# samples, pixels, channels, groups, and the most samples a launch of fewer than 2^32 threads takes: in one launch (64 threads a
# group of 40 channels of one pixel), forward and gradient; in two (1024 threads a sample), of which the gradient's second has one more
@pytest.mark.parametrize("pixels,channels,groups,forward,backward", [(1, 1280, 32, (1 << 21) - 1, (1 << 21) - 1), (96 * 96, 32, 32, (1 << 22) - 1, (1 << 22) - 2),
                                                                     (1, 8, 1, (1 << 26) - 1, (1 << 26) - 1)])
def test_most_samples(pixels, channels, groups, forward, backward):
    for name, most in (("svdq_group_norm_workspace", forward), ("svdq_group_norm_backward_workspace", backward)):
        for samples, status in ((4092, OK), (200000, OK), (most, OK), (most + 1, UNSUPPORTED)):
            d, size = norm(samples=samples, pixels=pixels, channels=channels, groups=groups, weight=None, bias=None), C.c_size_t()
            assert fn(name)(d, size) == status, (name, samples)
