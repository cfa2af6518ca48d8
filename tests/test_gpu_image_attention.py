"""GPU tests of the cross attention and its gradient against 64-bit formulas."""
import math

import pytest

pytestmark = pytest.mark.gpu

# half a step of a 16-bit value, relative, and half the smallest step
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def _torch():
    import torch

    from diffusion_smooth_group_amd import image
    return torch, image


def _dtype(name):
    torch, _ = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


class Case:
    """Operands of requests with rows[i] queries over keys[i] states each; `extra` rows and states of no request behind them."""

    def __init__(self, rows, keys, hq, hk, d, dtype, seed=0, mask=None, extra=0, size=1.0, grad=1.0):
        torch, _ = _torch()
        g = torch.Generator(device="cuda").manual_seed(seed + 1000 * d + hq)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.rows, self.keys, self.hq, self.hk, self.d, self.dtype = rows, keys, hq, hk, d, dtype
        n, m = sum(rows) + extra, sum(keys) + extra
        t = _dtype(dtype)
        self.q = (1.2 * size * r(n, hq, d)).to(t)
        kv = ((r(m, 2 * hk, d) + 0.2 * r(2 * hk, d)) * torch.exp(0.3 * r(2 * hk, d))).to(t)
        self.k, self.v = kv[:, :hk], kv[:, hk:]
        self.g = (grad * r(n, hq, d)).to(t)
        self.mask = None
        if mask == "random":
            self.mask = torch.rand(m, generator=g, device="cuda") < 0.6
        elif mask == "tail":            # the last third of each request's states, all of the last request's
            self.mask = torch.cat([torch.arange(k, device="cuda") < k - k // 3 for k in keys] + [torch.ones(extra, device="cuda", dtype=torch.bool)])
            if len(keys) > 1:
                self.mask[sum(keys[:-1]):sum(keys)] = False
        starts = lambda c: torch.tensor([0] + [sum(c[:i + 1]) for i in range(len(c))], dtype=torch.int32, device="cuda")
        self.where = dict(q_start=starts(rows), k_start=starts(keys), max_q=max(rows), max_k=max(keys), mask=self.mask)
        self.scale = None

    def heads(self):
        """(rows, kept states, query head, key head) slices of every request and head that has rows."""
        torch, _ = _torch()
        r0 = k0 = 0
        for n, m in zip(self.rows, self.keys):
            at = torch.arange(k0, k0 + m, device="cuda")
            if self.mask is not None:
                at = at[self.mask[k0:k0 + m]]
            for h in range(self.hq if n else 0):
                yield slice(r0, r0 + n), at, h, h // (self.hq // self.hk)
            r0, k0 = r0 + n, k0 + m


def _logits(c, rows, at, h, hk):
    scale = 1 / math.sqrt(c.d) if c.scale is None else c.scale
    q, k = c.q[rows, h].double(), c.k[at, hk].double()
    # error of a logit: D products and sums of 2^-24 each way of what is added up, and the exponent's own rounding at its size
    size = abs(scale) * (q.abs() @ k.abs().T)
    s = scale * (q @ k.T)
    return q, k, s, (c.d + 16) * 2.0 ** -24 * size + 2.0 ** -22 * s.abs() + 2.0 ** -20


def check_forward(c, out, lse=None, what=""):
    torch, _ = _torch()
    u = ULP[c.dtype]
    for rows, at, h, hk in c.heads():
        got = out[rows, h].double()
        if at.numel() == 0:
            assert bool((got == 0).all()), what
            assert lse is None or bool((lse[rows, h] == -math.inf).all()), what
            continue
        _, _, s, e = _logits(c, rows, at, h, hk)
        v = c.v[at, hk].double()
        p = torch.softmax(s, -1)
        want, size = p @ v, p @ v.abs()
        # p rounded to 16 bits, each logit's error (twice: the sum has it, too), the result's rounding; f16: probabilities 2^-31
        # of the largest and less are held to 2^-31 of it
        tol = (u * (size + want.abs()) * 1.01 + 2 * e.amax(-1, keepdim=True) * size + TINY[c.dtype]
               + (2.0 ** -30 * v.abs().sum(0) if c.dtype == "f16" else 0.0))
        worst = float(((got - want).abs() / tol).nan_to_num(nan=1e9).max())
        assert worst <= 1, f"{what} head {h}: {worst:.3f} of the tolerance"
        if lse is not None:
            want = torch.logsumexp(s, -1)
            tol = e.amax(-1) + 2.0 ** -22 * want.abs() + 2.0 ** -20 + at.numel() * 2.0 ** -24
            assert float(((lse[rows, h].double() - want).abs() / tol).max()) <= 1, f"lse {what}"


def check_backward(c, out, lse, dq, dk, dv, what=""):
    torch, _ = _torch()
    u, scale = ULP[c.dtype], 1 / math.sqrt(c.d) if c.scale is None else c.scale
    wk, wv, ek, ev = (torch.zeros((c.k.shape[0], c.hk, c.d), dtype=torch.float64, device="cuda") for _ in range(4))
    for rows, at, h, hk in c.heads():
        got = dq[rows, h].double()
        if at.numel() == 0:
            assert bool((got == 0).all()), what
            continue
        q, k, s, e = _logits(c, rows, at, h, hk)
        v, g, o = c.v[at, hk].double(), c.g[rows, h].double(), out[rows, h].double()
        # the definition, from the given lse and output
        p = torch.exp(s - lse[rows, h].double()[:, None])
        e = e + 2.0 ** -21 * (1 + lse[rows, h].double().abs()[:, None])
        dp = g @ v.T
        # up to 128 states: delta of the probabilities themselves
        delta = (p * dp).sum(-1, keepdim=True) if c.where["max_k"] <= 128 else (g * o).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        near = (c.d + 16) * 2.0 ** -24 * (g.abs() @ v.abs().T + (g * o).abs().sum(-1, keepdim=True))
        if c.where["max_k"] <= 128:     # the error of each probability and product, and of a sum of up to 128
            near = near + (p * ((e + 128 * 2.0 ** -24) * dp.abs() + near)).sum(-1, keepdim=True)
        # ds: rounded to 16 bits, p's error, the products' errors; f16 under its gain: to 2^-30 of the largest of its row
        # (or state), which `least` bounds for either sum
        least = 2.0 ** -30 * torch.maximum(ds.abs().amax(-1, keepdim=True), ds.abs().amax(0, keepdim=True)) if c.dtype == "f16" else 0.0
        e_ds = (u * 1.01 + e) * ds.abs() + p * (1 + e) * near + least
        want = scale * ds @ k
        tol = abs(scale) * e_ds @ k.abs() + u * want.abs() * 1.01 + TINY[c.dtype] + 2.0 ** -20 * abs(scale) * ds.abs() @ k.abs()
        worst = float(((got - want).abs() / tol).nan_to_num(nan=1e9).max()) if got.numel() else 0.0
        assert worst <= 1, f"dq {what} head {h}: {worst:.3f} of the tolerance"
        wk[at, hk] += scale * ds.T @ q
        ek[at, hk] += abs(scale) * (e_ds.T @ q.abs() + 2.0 ** -20 * ds.abs().T @ q.abs())
        wv[at, hk] += p.T @ g
        # f16: p is held at 2^10 of its size, so to 2^-35 of 1 (2^-35 of each g)
        ev[at, hk] += ((u * 1.01 + e + 2.0 ** -20) * p).T @ g.abs() + (2.0 ** -34 * g.abs().sum(0) if c.dtype == "f16" else 0.0)
    n = sum(c.keys)
    for got, want, err, name in ((dk, wk, ek, "dk"), (dv, wv, ev, "dv")):
        tol = err[:n] + u * want[:n].abs() * 1.01 + TINY[c.dtype]
        worst = float(((got[:n].double() - want[:n]).abs() / tol).nan_to_num(nan=1e9).max()) if n else 0.0
        assert worst <= 1, f"{name} {what}: {worst:.3f} of the tolerance"
        if c.mask is not None:
            assert bool((got[:n][~c.mask[:n]] == 0).all()), f"{name} {what}: states that are not seen"


# rows, states, heads, head dimensions; few rows and tiles of 128, one and many chunks, grouped heads, empty requests
FORMS = [
    ([1], [1], 1, 1, 64), ([1, 1, 1], [1500, 7, 33], 20, 20, 64), ([1] * 5, [129, 1, 64, 2000, 31], 32, 8, 128), ([3, 0, 16, 1], [5, 70, 0, 600], 4, 2, 72),
    ([130, 1, 64], [77, 300, 65], 5, 5, 40), ([257, 31], [64, 1], 2, 1, 128), ([100, 0, 7], [63, 5, 0], 8, 2, 96), ([65], [4100], 1, 1, 128),
    ([2, 1], [9000, 4], 2, 1, 80), ([129, 300], [513, 1025], 3, 3, 8), ([400], [77], 10, 10, 64), ([33], [33], 6, 3, 120),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("mask", [None, "random", "tail"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forward(form, mask, dtype):
    _, image = _torch()
    c = Case(*FORMS[form], dtype, seed=form, mask=mask)
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    check_forward(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("mask", [None, "random", "tail"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_gradient(form, mask, dtype):
    torch, image = _torch()
    c = Case(*FORMS[form], dtype, seed=form, mask=mask)
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    dq, dk, dv = image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where)
    check_backward(c, out, lse, dq, dk, dv)
    again = image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), again))


@pytest.mark.parametrize("d", range(8, 129, 8))
def test_every_head_dimension(d):
    _, image = _torch()
    for rows, keys in (([3], [70]), ([140], [70])):
        c = Case(rows, keys, 2, 2, d, "f16" if d % 16 else "bf16", seed=d)
        out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
        check_forward(c, out, lse, f"D {d}")
        check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where), f"D {d}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 200])
def test_dense_requests_are_the_ragged_ones(rows, dtype):
    torch, image = _torch()
    c = Case([rows] * 3, [90] * 3, 6, 3, 64, dtype, mask="random")
    want = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    q, k, v, g = (t.unflatten(0, (3, -1)) for t in (c.q, c.k, c.v, c.g))
    got = image.cross_attention(q, k, v, mask=c.mask.view(3, 90), return_lse=True)
    assert got[0].shape == q.shape and got[1].shape == q.shape[:3]
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, want))
    grads = image.cross_attention_backward(g, q, k, v, *got, mask=c.mask.view(3, 90))
    again = image.cross_attention_backward(c.g, c.q, c.k, c.v, *want, **c.where)
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(grads, again))
    assert torch.equal(image.cross_attention(q, k, v, mask=c.mask.view(3, 90).to(torch.uint8)), got[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hk,d", [(6, 2, 64), (5, 1, 128), (14, 2, 72), (33, 1, 40), (64, 1, 64), (80, 1, 96), (7, 7, 64), (24, 8, 128)])
def test_heads_in_groups_of_any_size(hq, hk, d, dtype):
    """Rows of a pair are (token, head of the group): groups that divide a stage of rows, that do not, and larger ones."""
    _, image = _torch()
    for rows, keys in (([1, 1], [70, 9]), ([37, 2, 5], [150, 300, 40])):
        c = Case(rows, keys, hq, hk, d, dtype, seed=hq, mask="random")
        out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
        check_forward(c, out, lse, f"{hq}/{hk}")
        check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where), f"{hq}/{hk}")


@pytest.mark.parametrize("rows", [1, 20])
def test_many_requests(rows):
    _, image = _torch()
    n = 203
    c = Case([rows + i % 3 for i in range(n)], [(7 * i) % 90 for i in range(n)], 3, 3, 64, "bf16", mask="random")
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    check_forward(c, out, lse)
    check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where))


@pytest.mark.parametrize("rows", [[2, 1], [150, 40]])
def test_what_is_of_no_request_is_left(rows):
    torch, image = _torch()
    c = Case(rows, [70, 30], 4, 2, 64, "bf16", extra=9)
    out, lse = torch.full_like(c.q, 7.0), None
    image.cross_attention(c.q, c.k, c.v, out=out, **c.where)
    n, m = sum(rows), 100
    assert bool((out[n:] == 7).all())
    _, lse = image.cross_attention(c.q, c.k, c.v, out=out, return_lse=True, **c.where)
    check_forward(c, out, lse)
    grads = [torch.full_like(t, 5.0) for t in (c.q, c.k, c.v)]
    image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, dq=grads[0], dk=grads[1], dv=grads[2], **c.where)
    assert bool((grads[0][n:] == 5).all()) and all(bool((t[m:] == 5).all()) for t in grads[1:])
    check_backward(c, out, lse, *grads)


@pytest.mark.parametrize("rows", [[2], [150]])
def test_bounds_cut_rows_and_states(rows):
    torch, image = _torch()
    c = Case(rows, [300], 2, 2, 64, "bf16")
    c.where |= dict(max_q=rows[0] - 1, max_k=129)
    out, lse = torch.full_like(c.q, 7.0), None
    _, lse = image.cross_attention(c.q, c.k, c.v, out=out, return_lse=True, **c.where)
    assert bool((out[-1] == 7).all())
    small = Case(rows, [300], 2, 2, 64, "bf16")
    small.rows, small.keys = [rows[0] - 1], [129]
    check_forward(small, out, lse)
    grads = [torch.full_like(t, 5.0) for t in (c.q, c.k, c.v)]
    image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, dq=grads[0], dk=grads[1], dv=grads[2], **c.where)
    assert bool((grads[0][-1] == 5).all()) and all(bool((t[129:] == 5).all()) for t in grads[1:])
    check_backward(small, out, lse, *grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [[1], [140]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_masked_states_hold_does_not_matter(rows, bad, dtype):
    torch, image = _torch()
    c = Case(rows, [333], 4, 4, 64, dtype, mask="random")
    run = lambda: image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    want = run()
    grads = image.cross_attention_backward(c.g, c.q, c.k, c.v, *want, **c.where)
    for t in (c.k, c.v):
        t[~c.mask] = bad
    got = run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = image.cross_attention_backward(c.g, c.q, c.k, c.v, *got, **c.where)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("rows", [[2], [140]])
def test_scales(rows, scale, dtype):
    _, image = _torch()
    c = Case(rows, [150], 2, 2, 40, dtype, mask="random")
    c.scale = scale
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, scale=scale, **c.where)
    check_forward(c, out, lse)
    check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, scale=scale, **c.where))


@pytest.mark.parametrize("rows", [[2], [140]])
@pytest.mark.parametrize("grad", [2.0 ** -20, 2.0 ** -8, 2.0 ** 8])
def test_f16_gradients_of_any_size(rows, grad):
    """Small and large gradients keep f16's digits as far as the results hold them."""
    _, image = _torch()
    c = Case(rows, [700], 2, 2, 64, "f16", grad=grad)
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [[2], [140]])
def test_logits_that_rise_and_fall(rows, dtype):
    """States whose logits grow to many times a reference's slack, then fall."""
    torch, image = _torch()
    c = Case(rows, [900], 2, 2, 64, dtype)
    grow = torch.cat((torch.linspace(0, 6, 450), torch.linspace(6, 0, 450))).cuda()
    c.k.mul_(grow[:, None, None].to(c.k.dtype))
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    check_forward(c, out, lse)
    check_backward(c, out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where))


@pytest.mark.parametrize("rows", [[3], [140]])
def test_gradient_against_differences(rows):
    """Along a direction, against the 64-bit definition's difference."""
    torch, image = _torch()
    c = Case(rows, [90], 4, 2, 64, "f16", mask="random")
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    grads = dict(zip("qkv", image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where)))
    gen = torch.Generator(device="cuda").manual_seed(3)

    def loss(q, k, v):
        total = 0.0
        for at_r, at, h, hk in c.heads():
            w = torch.softmax(q[at_r, h] @ k[at, hk].T / math.sqrt(c.d), -1)
            total = total + ((w @ v[at, hk]) * c.g[at_r, h].double()).sum()
        return float(total)
    for name in "qkv":
        a = {n: getattr(c, n).double() for n in "qkv"}
        d = torch.randn(a[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = loss(**{**a, name: a[name] + h * d}), loss(**{**a, name: a[name] - h * d})
        got = float((grads[name].double() * d).sum())
        size = float((grads[name].double() * d).square().sum().sqrt())  # roundings of about 2^-10 in all add up like a random walk
        assert abs(got - (up - down) / (2 * h)) <= 8 * 2.0 ** -10 * size, name


def test_strides_and_outputs():
    torch, image = _torch()
    c = Case([70, 3], [90, 40], 4, 4, 72, "bf16")
    want, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    wide = torch.zeros((73, 12, 96), dtype=c.q.dtype, device="cuda")
    q = wide[:, 2:10:2, 8:80]
    q.copy_(c.q)
    out = torch.full_like(wide, 3.0)
    o = out[:, 4:8, 16:88]
    assert image.cross_attention(q, c.k, c.v, out=o, **c.where) is o
    assert torch.equal(o, want)
    o.fill_(3.0)
    assert bool((out == 3).all())
    grads = image.cross_attention_backward(c.g, c.q, c.k, c.v, want, lse, **c.where)
    again = image.cross_attention_backward(c.g, q, c.k, c.v, want, lse, dq=o, **c.where)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("shared", [False, True])
def test_autograd(shared):
    torch, image = _torch()
    c = Case([60] * 2, [77] * 2, 4, 2, 64, "bf16")
    q, k, v, g = (t.unflatten(0, (2, -1)).contiguous() for t in (c.q, c.k, c.v, c.g))
    if shared:
        k, v = k[:1], v[:1]
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    kk, vv = (t.expand(2, -1, -1, -1) if shared else t for t in leaves[1:])
    image.cross_attention_autograd(leaves[0], kk, vv).backward(g)
    kk, vv = (t.detach().contiguous() for t in (kk, vv))
    out, lse = image.cross_attention(q, kk, vv, return_lse=True)
    dq, dk, dv = image.cross_attention_backward(g, q, kk, vv, out, lse)
    assert torch.equal(leaves[0].grad, dq)
    for leaf, want in zip(leaves[1:], (dk, dv)):
        assert torch.equal(leaf.grad, want.sum(0, keepdim=True) if shared else want)


def test_autograd_of_ragged_rows():
    torch, image = _torch()
    c = Case([20, 5], [30, 0], 4, 2, 64, "bf16", extra=3)
    leaves = [t.clone().requires_grad_() for t in (c.q, c.k, c.v)]
    out = image.cross_attention_autograd(*leaves, **c.where)
    assert bool((out[20:] == 0).all())
    out.sum().backward()                # one gradient for all heads and rows, broadcast
    assert bool((leaves[0].grad[20:] == 0).all()) and bool((leaves[1].grad[30:] == 0).all()) and bool((leaves[2].grad[30:] == 0).all())
    c.g = torch.ones_like(c.g)
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    check_backward(c, out, lse, *[t.grad for t in leaves])
    with pytest.raises(RuntimeError):
        y = image.cross_attention_autograd(*leaves, **c.where)
        torch.autograd.grad(torch.autograd.grad(y.sum(), leaves[0], create_graph=True)[0].sum(), leaves[0])


@pytest.mark.parametrize("rows,keys", [(1, 3000), (130, 77), (130, 2000)])
def test_captured_and_replayed(rows, keys):
    torch, image = _torch()
    c = Case([rows] * 2, [keys] * 2, 4, 2, 64, "f16", mask="random")

    def both():
        out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
        return out, lse, *image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where)
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
        new = Case([rows] * 2, [keys] * 2, 4, 2, 64, "f16", seed=seed, mask="random")
        for t, n in ((c.q, new.q), (c.k, new.k), (c.v, new.v), (c.g, new.g), (c.mask, new.mask)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, both()))


def test_two_streams_at_once():
    torch, image = _torch()
    cases = [Case([1, 1], [3000, 2000], 8, 8, 64, "bf16", seed=s) for s in (1, 2)]
    want = [image.cross_attention(c.q, c.k, c.v, **c.where) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, c in enumerate(cases):
            got[i].append(image.cross_attention(c.q, c.k, c.v, stream=streams[i], **c.where))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in (0, 1) for y in got[i])


def test_no_requests_and_no_states():
    torch, image = _torch()
    q = torch.zeros((0, 5, 4, 64), device="cuda", dtype=torch.bfloat16)
    assert image.cross_attention(q, q, q).shape == q.shape
    q, k = torch.ones((2, 5, 4, 64), device="cuda", dtype=torch.bfloat16), torch.zeros((2, 0, 4, 64), device="cuda", dtype=torch.bfloat16)
    out, lse = image.cross_attention(q, k, k, return_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = image.cross_attention_backward(q, q, k, k, out, lse)
    assert bool((dq == 0).all()) and dk.shape == k.shape
    q = torch.zeros((2, 0, 4, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.ones((2, 7, 4, 64), device="cuda", dtype=torch.bfloat16)
    out, lse = image.cross_attention(q, k, k, return_lse=True)
    _, dk, dv = image.cross_attention_backward(q, q, k, k, out, lse)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("rows,keys", [(1, 9000), (9000, 150)])
def test_offsets_past_32_bits(rows, keys):
    """Operands whose tokens lie 2^18 elements apart: 2^31 elements and more in all."""
    torch, image = _torch()
    c = Case([rows], [keys], 2, 2, 64, "bf16")
    if rows > keys:
        far = torch.empty((rows, 1 << 18), dtype=torch.bfloat16, device="cuda")[:, :256].view(rows, 4, 64)
        q, g = far[:, :2], far[:, 2:]
        q.copy_(c.q)
        g.copy_(c.g)
        k, v = c.k, c.v
    else:
        far = torch.empty((keys, 1 << 18), dtype=torch.bfloat16, device="cuda")[:, :256].view(keys, 4, 64)
        k, v = far[:, :2], far[:, 2:]
        k.copy_(c.k)
        v.copy_(c.v)
        q, g = c.q, c.g
    out, lse = image.cross_attention(q, k, v, return_lse=True, **c.where)
    want, again = image.cross_attention(c.q, c.k, c.v, return_lse=True, **c.where)
    assert torch.equal(out, want) and torch.equal(lse, again)
    grads = image.cross_attention_backward(g, q, k, v, out, lse, **c.where)
    assert all(torch.equal(a, b) for a, b in zip(grads, image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **c.where)))
    far = torch.empty((max(rows, keys), 1 << 18), dtype=torch.bfloat16, device="cuda")[:, :128].view(-1, 2, 64)
    if rows > keys:
        assert torch.equal(image.cross_attention(q, k, v, out=far, **c.where), want)
    else:
        image.cross_attention_backward(g, q, k, v, out, lse, dk=far, **c.where)
        assert torch.equal(far, grads[1])
