"""GPU tests of the group norm over long maps and many samples, where a sum has
many terms and one value far from the rest may be what deviations are taken from,
and of an activation's far ends."""
import math

import pytest

from tests import test_gpu_image_norm as base

pytestmark = pytest.mark.gpu


def _stats64(x, groups):
    """Mean and inverse deviation of every group in 64 bits, a few samples at a time."""
    torch, _ = base._torch()
    n, c = x.shape[0], x.shape[-1]
    step = max(1, (1 << 28) // (x[0].numel()))
    mean, rstd = [], []
    for i in range(0, n, step):
        y = x[i:i + step].double().reshape(min(step, n - i), -1, groups, c // groups)
        var, mu = torch.var_mean(y, dim=(1, 3), unbiased=False)
        mean.append(mu)
        rstd.append(1 / torch.sqrt(var + 1e-5))
    return torch.cat(mean), torch.cat(rstd)


# Square deviations are sums of terms that are not negative: at most 32 a run of a thread and 8 runs, 64 rows of pixels and 4
# steps of a tree, 128 channels and 6 steps, and the chunks' (64 and 32): below 2^9 roundings of 2^-24 each, 2^-15 of the
# variance and 2^-16 of rstd.  The mean: as many of the deviations', and its own.
def _check_stats(x, groups, stats):
    mean, rstd = _stats64(x, groups)
    base._check(stats[..., 0], mean, 2.0 ** -15 / rstd + 2.0 ** -23 * mean.abs(), "mean")
    base._check(stats[..., 1], rstd, 2.0 ** -15 * rstd, "rstd")


@pytest.mark.parametrize("far", ["first", "some", "rows", "channel"])
@pytest.mark.parametrize("n,sides,c,groups", [(256, (256, 256), 8, 1), (32, (512, 512), 64, 4), (256, (64, 64), 2048, 8), (2, (64, 64), 8192, 1), (1, (1500, 1400), 16, 1),
                                              (3, (16, 16), 1280, 4), (2, (30, 30), 320, 32)])
def test_values_far_from_the_rest(n, sides, c, groups, far):
    """512 +- 2 but for one pixel, a few, the upper rows of a map or one channel of a group, which are 0."""
    torch, image = base._torch()
    g = torch.Generator(device="cuda").manual_seed(n + c)
    x = torch.empty((n, *sides, c), device="cuda", dtype=torch.float16)
    for i in range(0, n, 16):
        x[i:i + 16] = 512 + 2 * torch.randn((min(16, n - i), *sides, c), generator=g, device="cuda")
    pixels = x.view(n, -1, c)
    if far == "first":
        pixels[:, 0] = 0
    elif far == "some":
        for at in (0, 1, 2, 4):             # the corner, and what lies a quarter of the map on
            pixels[:, at * pixels.shape[1] // 4 if at < 4 else -1] = 0
    elif far == "rows":
        x[:, :max(1, sides[0] // 40)] = 0
    else:
        x[..., ::c // groups] = 0
    y, stats = image.group_norm(x, groups, return_stats=True)
    _check_stats(x, groups, stats)
    few = x[-1:]
    base._check_forward(few, groups, None, None, 1e-5, None, y[-1:], stats[-1:], "f16")


@pytest.mark.parametrize("n,sides,c", [(1000003, (), 8), (70001, (3,), 40)])
def test_gradient_sums_over_many_samples(n, sides, c):
    """dw and db are sums over all samples.  Weights of zero make every term of db the same, whose roundings all go one way.  A
    sum of n equal terms is off by 2^-24 n / 2 at most: runs of 256, as many as there are (489), and eight walks, below 2^-15."""
    torch, image = base._torch()
    g = torch.Generator(device="cuda").manual_seed(c)
    x = torch.randn((n, *sides, c), generator=g, device="cuda").bfloat16()
    w, b = torch.zeros(c, device="cuda").bfloat16(), torch.ones(c, device="cuda").bfloat16()
    grad = torch.ones_like(x)
    _, stats = image.group_norm(x, 1, w, b, act="silu", return_stats=True)
    grads = image.group_norm_backward(grad, x, stats, 1, w, b, act="silu")
    base._check_gradient(x, grad, stats, 1, w, b, "silu", *grads, "bf16")


@pytest.mark.parametrize("sides", [(8, 8), (72, 64)])
def test_gelu_far_below_zero(sides):
    """z Phi(z) for z from -8 to -4 to a result's own rounding: weights of zero make z the bias.  Beside the rounding erfc's
    argument counts (2^-24 of it, 64 times as much of the result) and erfc itself (16 steps), below 2^-17 in all; the slope's
    exponent likewise (46 roundings of 2^-24), and its sum of equal terms (256 and 64 one after the other): 2^-15 is above both."""
    torch, image = base._torch()
    n, c = 2, 64
    x = torch.randn((n, *sides, c), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    w, b = torch.zeros(c, device="cuda").bfloat16(), torch.linspace(-8, -4, c, device="cuda").bfloat16()
    y, stats = image.group_norm(x, 8, w, b, act="gelu", return_stats=True)
    z = b.double()
    phi = 0.5 * torch.erfc(-z / math.sqrt(2))
    want = (z * phi).expand_as(x)
    base._check(y, want, (2.0 ** -8 * 1.01 + 2.0 ** -15) * want.abs(), "y")
    dx, dw, db = image.group_norm_backward(torch.ones_like(x), x, stats, 8, w, b, act="gelu")
    want = x.numel() // c * (phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    base._check(db, want, 2.0 ** -15 * want.abs(), "db")
    assert bool((dx == 0).all())


@pytest.mark.parametrize("n,sides,c,groups", [(200001, (), 1280, 32), (4501, (50, 50), 32, 1)])
def test_many_samples(n, sides, c, groups):
    torch, image = base._torch()
    x, w, b, g = base._inputs(n, "bf16", n, sides, c)
    y, stats = image.group_norm(x, groups, w, b, act="silu", return_stats=True)
    _check_stats(x, groups, stats)
    part = slice(n - 1000, n)
    base._check_forward(x[part], groups, w, b, 1e-5, "silu", y[part], stats[part], "bf16")
    grads = image.group_norm_backward(g, x, stats, groups, w, b, act="silu")
    few = image.group_norm_backward(g[part], x[part], stats[part], groups, w, b, act="silu")
    base._check_gradient(x[part], g[part], stats[part], groups, w, b, "silu", *few, "bf16")
    assert torch.equal(few[0], grads[0][part])
    # dw and db in all: fewer than 2^9 terms one after the other on the way, so within 2^-15 of the terms' absolute values
    total = [torch.zeros(c, device="cuda", dtype=torch.float64) for _ in range(4)]
    for i in range(0, n, 2000):
        at = slice(i, min(i + 2000, n))
        xs, gs, st = x[at].double().reshape(-1, math.prod(sides), c), g[at].double().reshape(-1, math.prod(sides), c), stats[at].double()
        xh = (xs - base._spread(st[..., 0], groups, c)) * base._spread(st[..., 1], groups, c)
        dz = gs * base._act64(xh * w.double() + b.double(), "silu")[1]
        for t, v in zip(total, (dz * xh, dz, (dz * xh).abs(), (gs * (1 + xh.abs())).abs())):
            t += v.sum((0, 1))
    # each term's own error: the slope to 2^-19 of g (and of g xh)
    base._check(grads[1], total[0], 2.0 ** -15 * total[2] + 2.0 ** -18 * total[3], "dw")
    base._check(grads[2], total[1], 2.0 ** -15 * total[3], "db")
