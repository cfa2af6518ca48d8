"""GPU tests of the group norm over channels-last maps and its gradient against
64-bit formulas."""
import math

import pytest

pytestmark = pytest.mark.gpu

# half a step of a 16-bit value, relative, and half the smallest step
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}
ACTS = [None, "silu", "gelu"]

# samples, sides, channels, groups: one launch (few pixels a group) and two; groups narrower than 8 channels, of widths that
# 8 does not divide, one group, as many as channels; one pixel; the widest
SIZES = [(1, (8, 8), 1280, 32), (2, (33, 31), 480, 32), (3, (), 64, 8), (3, (1, 1), 64, 8), (2, (5, 7), 40, 5), (1, (16, 16), 32, 32),
         (2, (64, 64), 320, 32), (1, (128, 96), 128, 1), (1, (3, 5), 8192, 32), (2, (40, 41), 8, 4), (1, (37,), 8, 1), (5, (3, 211), 24, 3),
         (2, (130, 129), 96, 4), (1, (61, 67), 8192, 8192), (1, (257, 255), 16, 16), (1, (100, 99), 8192, 8192)]


def _torch():
    import torch

    from diffusion_smooth_group_amd import image
    return torch, image


def _dtype(name):
    torch, _ = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _inputs(seed, dtype, n, sides, c, mean=1.0):
    torch, _ = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (r(n, *sides, c) * torch.exp(0.5 * r(c)) + mean * r(c)).to(_dtype(dtype))
    return x, (1 + 0.3 * r(c)).to(_dtype(dtype)), (0.3 * r(c)).to(_dtype(dtype)), r(n, *sides, c).to(_dtype(dtype))


def _act64(z, act):
    torch, _ = _torch()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def _forward64(x, groups, w, b, eps, act):
    """(y, mean, rstd, xh, z, slope) of the definition; x as [N, pixels, C]."""
    torch, _ = _torch()
    n, c = x.shape[0], x.shape[-1]
    y = x.double().reshape(n, -1, groups, c // groups)
    var, mean = torch.var_mean(y, dim=(1, 3), unbiased=False, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = ((y - mean) * rstd).reshape(n, -1, c)
    z = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    out, slope = _act64(z, act)
    return out, mean.reshape(n, groups), rstd.reshape(n, groups), xh, z, slope


def _spread(t, groups, c):
    """[N, groups] as [N, 1, C]."""
    return t.repeat_interleave(c // groups, dim=1)[:, None]


def _check(got, want, tol, what):
    torch, _ = _torch()
    assert not torch.isnan(got).any(), what
    worst = float(((got.double() - want).abs() / tol).max()) if want.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3f} of the tolerance"


# z in fp32: mean and deviation from sums of deviations over at most 64 serial terms, 128 rows of LDS, a tree and 512 chunks
# (each at most 512 roundings of 2^-24 of the deviations' size, which xh and 1 bound), x - mean to 2^-24 of |mean| rstd.
def _z_error(xh, z, w, mean, rstd, groups, c):
    far = _spread(mean.abs() * rstd, groups, c)
    wide = 1.0 if w is None else w.double().abs()
    return wide * (2.0 ** -15 * (1 + xh.abs()) + 2.0 ** -22 * far) + 2.0 ** -22 * z.abs()


def _check_forward(x, groups, w, b, eps, act, got, stats, dtype, what=""):
    n, c = x.shape[0], x.shape[-1]
    want, mean, rstd, xh, z, _ = _forward64(x, groups, w, b, eps, act)
    # |act'| <= 1.13; exponential, reciprocal and erf to 2^-20 of z
    tol = ULP[dtype] * want.abs() * 1.01 + 1.2 * _z_error(xh, z, w, mean, rstd, groups, c) + 2.0 ** -20 * z.abs() + TINY[dtype]
    _check(got.reshape(n, -1, c), want, tol, "y " + what)
    if stats is not None:
        _check(stats[..., 0], mean, 2.0 ** -15 / rstd + 2.0 ** -23 * mean.abs(), "mean " + what)
        _check(stats[..., 1], rstd, 2.0 ** -15 * rstd, "rstd " + what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,sides,c,groups", SIZES)
def test_forward(n, sides, c, groups, act, dtype):
    _, image = _torch()
    x, w, b, _ = _inputs(c + n, dtype, n, sides, c)
    y, stats = image.group_norm(x, groups, w, b, eps=1e-5, act=act, return_stats=True)
    assert y.shape == x.shape and y.dtype == x.dtype and stats.shape == (n, groups, 2)
    _check_forward(x, groups, w, b, 1e-5, act, y, stats, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,sides,c,groups", SIZES)
def test_gradient(n, sides, c, groups, act, dtype):
    torch, image = _torch()
    x, w, b, g = _inputs(c + n + 7, dtype, n, sides, c)
    _, stats = image.group_norm(x, groups, w, b, act=act, return_stats=True)
    dx, dw, db = image.group_norm_backward(g, x, stats, groups, w, b, act=act)
    _check_gradient(x, g, stats, groups, w, b, act, dx, dw, db, dtype)


def _check_gradient(x, g, stats, groups, w, b, act, dx, dw, db, dtype):
    torch, _ = _torch()
    n, c = x.shape[0], x.shape[-1]
    mean, rstd = stats[..., 0].double(), stats[..., 1].double()
    xs, gs = x.double().reshape(n, -1, c), g.double().reshape(n, -1, c)
    r = _spread(rstd, groups, c)
    xh = (xs - _spread(mean, groups, c)) * r
    wd = 1.0 if w is None else w.double()
    z = xh * wd + (0.0 if b is None else b.double())
    _, slope = _act64(z, act)
    dz = gs * slope
    u = dz * wd
    cut = lambda t: t.reshape(n, -1, groups, c // groups)
    m1, m2 = (_spread(cut(t).mean((1, 3)), groups, c) for t in (u, u * xh))
    a1, a2 = (_spread(cut(t.abs()).mean((1, 3)), groups, c) for t in (u, u * xh))
    want = r * (u - m1 - xh * m2)
    # dz: xh to a few roundings, the slope (its own slope is at most 0.7) to 2^-20 beside the error of z; sums of up to 512 roundings
    e_dz = gs.abs() * (2.0 ** -19 + 2.0 ** -21 * z.abs()) + dz.abs() * 2.0 ** -21
    e_u = e_dz * (wd if w is None else wd.abs())
    e1, e2 = (_spread(cut(t).mean((1, 3)), groups, c) for t in (e_u, e_u * xh.abs()))
    tol = ULP[dtype] * want.abs() * 1.01 + TINY[dtype] + r * (
        e_u + e1 + xh.abs() * e2 + 2.0 ** -15 * (a1 + xh.abs() * a2) + 2.0 ** -21 * (u.abs() + m1.abs() + (xh * m2).abs()))
    _check(dx.reshape(n, -1, c), want, tol, "dx")
    _check(db, dz.sum((0, 1)), 2.0 ** -15 * dz.abs().sum((0, 1)) + e_dz.sum((0, 1)) + 1e-30, "db")
    _check(dw, (dz * xh).sum((0, 1)), 2.0 ** -15 * (dz * xh).abs().sum((0, 1)) + (e_dz * xh.abs()).sum((0, 1)) + 1e-30, "dw")


@pytest.mark.parametrize("sides", [(7, 9), (70, 90)])
def test_gradient_against_differences(sides):
    """The formula's gradient along a direction, of the 64-bit definition's difference."""
    torch, image = _torch()
    x, w, b, g = _inputs(5, "f16", 2, sides, 48)
    _, stats = image.group_norm(x, 6, w, b, act="silu", return_stats=True)
    dx, dw, db = image.group_norm_backward(g, x, stats, 6, w, b, act="silu")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for which, t, grad in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        d = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
        h, values = 1e-4, []
        for s in (h, -h):
            a = {"x": x.double(), "w": w.double(), "b": b.double()}
            a[which] = a[which] + s * d
            y = _forward64(a["x"], 6, a["w"], a["b"], 1e-5, "silu")[0]
            values.append((y * g.double().reshape(y.shape)).sum())
        want, got = (values[0] - values[1]) / (2 * h), (grad.double() * d).sum()
        size = torch.sqrt((grad.double() * d).square().sum())       # roundings of 2^-11 add up like a random walk
        assert abs(float(got - want)) <= 2.0 ** -11 * 6 * float(size) + 1e-5 * abs(float(want)), which


@pytest.mark.parametrize("sides", [(9, 7), (80, 81)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_views_in_place_and_no_weights(sides, dtype):
    torch, image = _torch()
    x, w, b, g = _inputs(11, dtype, 2, sides, 96)
    want = image.group_norm(x, 8, w, b, act="silu")
    wide = torch.zeros((2, *sides, 160), dtype=x.dtype, device="cuda")
    view = wide[..., 32:128]
    view.copy_(x)
    assert torch.equal(image.group_norm(view, 8, w, b, act="silu"), want)
    out = torch.full_like(wide, 3.0)
    assert image.group_norm(view, 8, w, b, act="silu", out=out[..., 32:128]) is not None
    assert torch.equal(out[..., 32:128], want) and bool((out[..., :32] == 3).all()) and bool((out[..., 128:] == 3).all())
    _, stats = image.group_norm(x, 8, w, b, act="silu", return_stats=True)
    grads = image.group_norm_backward(g, x, stats, 8, w, b, act="silu")
    g2 = g.clone()
    again = image.group_norm_backward(g2, view, stats, 8, w, b, act="silu", dx=g2)
    assert all(torch.equal(a, c) for a, c in zip(grads, again)) and again[0] is g2
    image.group_norm(view, 8, w, b, act="silu", out=view)
    assert torch.equal(view, want) and bool((wide[..., :32] == 0).all())
    y, stats = image.group_norm(x, 8, return_stats=True)
    _check_forward(x, 8, None, None, 1e-5, None, y, stats, dtype)
    _check_gradient(x, g, stats, 8, None, None, None, *image.group_norm_backward(g, x, stats, 8), dtype)


@pytest.mark.parametrize("sides", [(8, 8), (72, 64)])
def test_a_mean_far_from_zero(sides):
    """Deviations of a 256th of the mean: sums of squares would lose all of them."""
    torch, image = _torch()
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (512 + 2 * torch.randn((2, *sides, 64), generator=g, device="cuda")).half()
    y, stats = image.group_norm(x, 4, return_stats=True)
    _check_forward(x, 4, None, None, 1e-5, None, y, stats, "f16")
    x[:, 0] = 0                                             # a border that lies far from the rest
    y, stats = image.group_norm(x, 4, return_stats=True)
    _check_forward(x, 4, None, None, 1e-5, None, y, stats, "f16")


@pytest.mark.parametrize("sides", [(8, 8), (72, 64)])
def test_constant_maps_and_values_that_are_not_finite(sides):
    torch, image = _torch()
    x = torch.full((3, *sides, 64), 2.5, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(64, device="cuda").bfloat16(), torch.full((64,), 0.75, device="cuda").bfloat16()
    y, stats = image.group_norm(x, 4, w, b, eps=1e-5, return_stats=True)
    assert bool((y == 0.75).all()) and torch.equal(stats[..., 0], torch.full((3, 4), 2.5, device="cuda"))
    good = image.group_norm(x, 4, w, b)
    flat = x.view(3, -1, 64)
    flat[1, 5, 17] = float("nan")
    flat[2, 3, 60] = float("inf")
    y = image.group_norm(x, 4, w, b).view(3, -1, 64)
    assert torch.equal(y[0], good.view(3, -1, 64)[0])
    assert bool(torch.isnan(y[1, :, 16:32]).all()) and bool((y[1, :, :16] == 0.75).all()) and bool((y[1, :, 32:] == 0.75).all())
    assert bool(torch.isnan(y[2, :, 48:]).all()) and bool((y[2, :, :48] == 0.75).all())


def test_no_samples():
    torch, image = _torch()
    x = torch.empty((0, 4, 4, 64), device="cuda", dtype=torch.bfloat16)
    y, stats = image.group_norm(x, 4, return_stats=True)
    assert y.shape == x.shape and stats.shape == (0, 4, 2)
    _, dw, db = image.group_norm_backward(x, x, stats, 4)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("sides", [(9, 7), (80, 81)])
def test_autograd(sides):
    torch, image = _torch()
    x, w, b, g = _inputs(21, "bf16", 2, sides, 96)
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    y = image.group_norm_autograd(x, w, b, 8, act="silu")
    y.backward(g)
    _, stats = image.group_norm(x.detach(), 8, w.detach(), b.detach(), act="silu", return_stats=True)
    dx, dw, db = image.group_norm_backward(g, x.detach(), stats, 8, w.detach(), b.detach(), act="silu")
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw.bfloat16()) and torch.equal(b.grad, db.bfloat16())
    # a gradient that is one value for all, and a map that lies channels first
    x.grad = None
    image.group_norm_autograd(x, w, b, 8).sum().backward()
    first = x.detach().permute(0, 3, 1, 2).contiguous().permute(0, 2, 3, 1).requires_grad_()
    image.group_norm_autograd(first, w, b, 8).sum().backward()
    assert torch.equal(x.grad, first.grad)
    with pytest.raises(RuntimeError):
        y = image.group_norm_autograd(x, w, b, 8)
        torch.autograd.grad(torch.autograd.grad(y.sum(), x, create_graph=True)[0].sum(), x)


@pytest.mark.parametrize("sides", [(8, 8), (80, 80)])
def test_captured_and_replayed(sides):
    torch, image = _torch()
    x, w, b, g = _inputs(31, "f16", 2, sides, 128)

    def both():
        y, stats = image.group_norm(x, 32, w, b, act="silu", return_stats=True)
        return y, *image.group_norm_backward(g, x, stats, 32, w, b, act="silu")
    both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (1, 2, 3):
        new = _inputs(seed, "f16", 2, sides, 128)
        x.copy_(new[0])
        g.copy_(new[3])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(held, both()))


def test_two_streams_at_once():
    torch, image = _torch()
    sets = [_inputs(s, "bf16", 2, (64, 64), 320) for s in (41, 42)]
    want = [image.group_norm(x, 32, w, b, act="silu") for x, w, b, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (x, w, b, _) in enumerate(sets):
            got[i].append(image.group_norm(x, 32, w, b, act="silu", stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in (0, 1) for y in got[i])


def test_offsets_past_32_bits():
    """Pixels 2^17 elements apart: 2^31 elements and more in all."""
    torch, image = _torch()
    x, w, b, g = _inputs(51, "bf16", 1, (17000,), 64)
    wide = torch.empty((1, 17000, 1 << 17), dtype=torch.bfloat16, device="cuda")
    far, far_g = wide[..., :64], wide[..., 64:128]
    far.copy_(x)
    far_g.copy_(g)
    want, stats = image.group_norm(x, 8, w, b, act="silu", return_stats=True)
    assert torch.equal(image.group_norm(far, 8, w, b, act="silu"), want)
    grads = image.group_norm_backward(g, x, stats, 8, w, b, act="silu")
    again = image.group_norm_backward(far_g, far, stats, 8, w, b, act="silu", dx=wide[..., 128:192])
    assert all(torch.equal(a, c) for a, c in zip(grads, again))
