"""GPU tests of the gradient of the cross attention over up to 128 states, which
has a form of its own (all states at once, delta from the probabilities), and of
both forms around that length."""
import math

import pytest

from tests import test_gpu_image_attention as base

pytestmark = pytest.mark.gpu


def _both(c, **how):
    _, image = base._torch()
    out, lse = image.cross_attention(c.q, c.k, c.v, return_lse=True, **how, **c.where)
    return out, lse, image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, **how, **c.where)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("keys", [1, 31, 32, 33, 63, 64, 65, 77, 96, 97, 127, 128, 129])
def test_every_length_of_the_form(keys, dtype):
    for mask in (None, "random"):
        c = base.Case([150, 3], [keys, keys // 2], 4, 2, 64, dtype, seed=keys, mask=mask)
        out, lse, grads = _both(c)
        base.check_forward(c, out, lse)
        base.check_backward(c, out, lse, *grads, f"{keys} {mask}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("rows,d", [([2], 40), ([140], 64), ([140], 96), ([140], 128)])
def test_scales(rows, d, scale, dtype):
    c = base.Case(rows, [77], 2, 2, d, dtype, mask="random")
    c.scale = scale
    out, lse, grads = _both(c, scale=scale)
    base.check_forward(c, out, lse)
    base.check_backward(c, out, lse, *grads)


@pytest.mark.parametrize("rows", [[2], [140]])
@pytest.mark.parametrize("grad", [2.0 ** -20, 2.0 ** -8, 2.0 ** 8])
def test_f16_gradients_of_any_size(rows, grad):
    c = base.Case(rows, [77], 2, 2, 64, "f16", grad=grad)
    out, lse, grads = _both(c)
    base.check_backward(c, out, lse, *grads)


@pytest.mark.parametrize("rows", [[2], [140]])
@pytest.mark.parametrize("keys", [77, 700])
def test_f16_rows_of_different_size(rows, keys):
    """Each row's ds has a power of two of its own in dq, each state's in dk."""
    torch, _ = base._torch()
    c = base.Case(rows, [keys], 2, 2, 64, "f16")
    c.g *= torch.exp2(torch.linspace(-12, 8, c.g.shape[0], device="cuda"))[:, None, None].half()
    out, lse, grads = _both(c)
    base.check_backward(c, out, lse, *grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [[2], [140]])
def test_logits_that_rise_and_fall(rows, dtype):
    torch, _ = base._torch()
    c = base.Case(rows, [120], 2, 2, 64, dtype)
    grow = torch.cat((torch.linspace(0, 6, 60), torch.linspace(6, 0, 60))).cuda()
    c.k.mul_(grow[:, None, None].to(c.k.dtype))
    out, lse, grads = _both(c)
    base.check_forward(c, out, lse)
    base.check_backward(c, out, lse, *grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [[1], [140]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_masked_states_hold_does_not_matter(rows, bad, dtype):
    torch, _ = base._torch()
    for keys in (77, 128):
        c = base.Case(rows, [keys], 4, 4, 64, dtype, mask="random")
        c.mask[:33] = False             # a tile of 32 that shows nothing
        out, lse, grads = _both(c)
        for t in (c.k, c.v):
            t[~c.mask] = bad
        again, lse2, grads2 = _both(c)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("keys", [77, 300])
def test_a_row_that_is_not_finite_stays_alone(keys, dtype):
    """A query or a gradient row of NaN spoils its own row's results and the sums over rows of its head, nothing else."""
    torch, image = base._torch()
    for which in ("q", "g"):
        c = base.Case([150, 20], [keys, keys], 4, 2, 64, dtype, mask="random")
        out, lse, (dq, dk, dv) = _both(c)
        getattr(c, which)[7, 1] = math.nan
        out2, lse2, grads2 = _both(c)
        good = torch.ones(170, 4, dtype=torch.bool, device="cuda")
        good[7, 1] = False
        if which == "q":
            assert torch.equal(out[good], out2[good]) and torch.equal(lse[good], lse2[good]) and bool(torch.isnan(out2[7, 1]).all())
        assert torch.equal(dq[good], grads2[0][good]) and bool(torch.isnan(grads2[0][7, 1]).all())
        for a, b in zip((dk, dv), grads2[1:]):
            assert torch.equal(a[keys:], b[keys:]) and torch.equal(a[:, 1], b[:, 1])        # the other request's, the other key head's
            assert bool((b[:keys][~c.mask[:keys]] == 0).all())


@pytest.mark.parametrize("keys", [77, 200])
def test_no_row_of_a_request(keys):
    """States of a request without rows get zeros, rows of one without states too."""
    c = base.Case([0, 130, 5], [keys, 0, keys], 4, 2, 64, "bf16")
    out, lse, grads = _both(c)
    base.check_forward(c, out, lse)
    base.check_backward(c, out, lse, *grads)
    assert bool((grads[1][:keys] == 0).all()) and bool((grads[2][:keys] == 0).all())


@pytest.mark.parametrize("keys", [77, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("offset,gap", [(8, 0), (32, 0), (64, 0), (0, 16), (0, 32)])
def test_results_at_any_place(offset, gap, d, keys):
    """Rows that are whole lines are stored in another way than rows that are not: the same values, and nothing beside them."""
    torch, image = base._torch()
    c = base.Case([150, 40], [keys, keys], 4, 2, d, "bf16")
    out, lse, grads = _both(c)
    n = 4 * d + 128 + gap
    wide = [torch.full((190, n), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    o, dq = (t[:, offset:offset + 4 * d].view(190, 4, d) for t in wide)
    image.cross_attention(c.q, c.k, c.v, out=o, **c.where)
    image.cross_attention_backward(c.g, c.q, c.k, c.v, out, lse, dq=dq, **c.where)
    assert torch.equal(o, out) and torch.equal(dq, grads[0])
    for t in (o, dq):
        t.fill_(3.0)
    assert all(bool((t == 3).all()) for t in wide)
