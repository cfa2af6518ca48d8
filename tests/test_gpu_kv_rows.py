"""GPU tests of the row operators around the 4-bit cache: norm and rotation of
q and k and its gradient against 64-bit formulas, the append bit for bit
against the oracle's quantizers, the read-back, and the tables of a step
against Python loops."""
import numpy as np
import pytest

import oracle as o

pytestmark = pytest.mark.gpu

DT = ["bf16", "f16"]
# half a unit in the last place of a 16-bit value, relative, and the smallest step
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def _torch():
    import torch

    from diffusion_smooth_group_amd import kv
    return torch, kv


def _dtype(name):
    torch, _ = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _rows(seed, dtype, *shape, size=1.0):
    torch, _ = _torch()
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(_dtype(dtype)).cuda()


def _tables(n, dim, seed=3):
    torch, _ = _torch()
    a = torch.rand((n, dim // 2), generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * 40
    return a.cos().float().cuda(), a.sin().float().cuda()


def _pairs(x, halves):
    if halves:
        a, b = x.chunk(2, -1)
        return a, b
    return x[..., 0::2], x[..., 1::2]


def _join(a, b, halves):
    torch, _ = _torch()
    return torch.cat((a, b), -1) if halves else torch.stack((a, b), -1).flatten(-2)


def _forward64(x, w, cos, sin, positions, eps, norm, halves):
    """The definition in 64 bits on the CPU, and the size of what is added up
    in each element (for the fp32 rounding errors)."""
    torch, _ = _torch()
    y = x.double().cpu()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double().cpu()
    if cos is None:
        return y, y.abs()
    at = torch.arange(x.shape[0]) if positions is None else positions.cpu().long()
    c, s = cos.double().cpu()[at][:, None], sin.double().cpu()[at][:, None]
    a, b = _pairs(y, halves)
    return (_join(a * c - b * s, a * s + b * c, halves),
            _join((a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs(), halves))


def _check16(got, want, size, dtype, what=""):
    """One rounding to 16 bits of a value whose fp32 error is at most 2^-19 of
    its terms' size (a mean of D squares in a tree: (log2 D + 16) roundings of
    2^-24; root, quotient, weight and rotation: 8 more)."""
    err = (got.double().cpu() - want).abs()
    tol = ULP[dtype] * want.abs() * 1.01 + 2.0 ** -19 * size + TINY[dtype]
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.3f} of the tolerance"


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim", [(1, 1, 1, 16), (3, 5, 2, 48), (65, 3, 1, 64), (17, 4, 4, 80), (9, 2, 2, 96),
                                             (130, 24, 8, 128), (33, 3, 3, 240), (7, 2, 1, 256)])
def test_norm_rope_against_64_bits(dtype, halves, tokens, hq, hk, dim):
    torch, kv = _torch()
    qkv = _rows(tokens + dim, dtype, tokens, hq + 2 * hk, dim, size=2.0)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]              # views of a fused row
    wq, wk = 1 + _rows(1, dtype, dim, size=0.3), 1 + _rows(2, dtype, dim, size=0.3)
    cos, sin = _tables(tokens + 9, dim)
    pos = torch.randperm(tokens + 9, generator=torch.Generator().manual_seed(4))[:tokens].int().cuda()
    for norm, rope, w, p in ((True, True, True, pos), (True, True, False, None), (True, False, True, None), (False, True, False, pos)):
        got = kv.qk_norm_rope(q, k, cos if rope else None, sin if rope else None, wq if w else None, wk if w else None,
                              eps=1e-5, norm=norm, halves=halves and rope, positions=p if rope else None)
        for x, y, ww in ((q, got[0], wq), (k, got[1], wk)):
            want, size = _forward64(x, ww if w else None, cos if rope else None, sin, p, 1e-5, norm, halves)
            _check16(y, want, size, dtype, f"{norm} {rope} {w}")


@pytest.mark.parametrize("dtype", DT)
def test_norm_rope_in_place_strided_and_other_layouts(dtype):
    torch, kv = _torch()
    x = _rows(11, dtype, 37, 5, 3, 64)                  # [T, H, q k v, D]: head stride 3 D
    q, k = x[:, :, 0], x[:, :, 1]
    cos, sin = _tables(37, 64)
    want = kv.qk_norm_rope(q.contiguous(), k.contiguous(), cos, sin)
    keep = x[:, :, 2].clone()
    kv.qk_norm_rope(q, k, cos, sin, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, 2], keep)
    wide = torch.full((37, 5, 80), 7.0, dtype=x.dtype, device="cuda")     # heads with a gap behind each
    q2 = _rows(12, dtype, 37, 5, 64)
    kv.qk_norm_rope(q2, q2, cos, sin, q_out=wide[..., :64], k_out=torch.empty_like(q2))
    assert torch.equal(wide[..., :64], kv.qk_norm_rope(q2, q2, cos, sin)[0]) and bool((wide[..., 64:] == 7).all())
    only_q, _ = kv.qk_norm_rope(q2, q2[:, :0], cos, sin)
    assert torch.equal(only_q, wide[..., :64])


def test_norm_rope_special_values():
    torch, kv = _torch()
    cos, sin = _tables(4, 64)
    q = _rows(5, "bf16", 6, 2, 64)
    q[1, 0] = 0                                          # a zero row: finite, zero
    q[2, 1, 3] = float("inf")
    q[3, 0, 5] = float("nan")
    pos = torch.tensor([0, 1, 2, 3, 4, -1], dtype=torch.int32, device="cuda")
    y, _ = kv.qk_norm_rope(q, q[:, :1], cos, sin, positions=pos)
    assert bool((y[1, 0] == 0).all())
    assert bool(y[2, 1].isnan().any()) and bool(y[2, 0].isfinite().all())
    assert bool(y[3, 0].isnan().all()) and bool(y[3, 1].isfinite().all())
    assert bool(y[4:].isnan().all()) and bool(y[0].isfinite().all())       # positions outside the table


def _backward64(g, x, w, cos, sin, positions, eps, norm, halves):
    torch, _ = _torch()
    g, x = g.double().cpu(), x.double().cpu()
    if cos is not None:
        at = torch.arange(x.shape[0]) if positions is None else positions.cpu().long()
        c, s = cos.double().cpu()[at][:, None], sin.double().cpu()[at][:, None]
        a, b = _pairs(g, halves)
        g = _join(a * c + b * s, b * c - a * s, halves)
    if not norm:
        return g, g.abs().amax(-1, keepdim=True) * 2, torch.zeros(x.shape[-1], dtype=torch.float64), torch.zeros(1)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = g if w is None else g * w.double().cpu()
    n = x * r
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    size = r * (u.abs().amax(-1, keepdim=True) * 2 + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    return dx, size, (g * n).sum((0, 1)), (g * n).abs().sum((0, 1))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim", [(1, 1, 1, 16), (5, 3, 1, 80), (257, 3, 2, 64), (1500, 24, 24, 128), (40, 2, 1, 256)])
def test_gradient_against_the_formula(dtype, halves, tokens, hq, hk, dim):
    torch, kv = _torch()
    x = _rows(tokens, dtype, tokens, hq + hk, dim, size=1.5)
    g = _rows(tokens + 1, dtype, tokens, hq + hk, dim)
    wq, wk = 1 + _rows(1, dtype, dim, size=0.3), 1 + _rows(2, dtype, dim, size=0.3)
    cos, sin = _tables(tokens, dim)
    for norm, rope in ((True, True), (True, False), (False, True)):
        t = (cos, sin) if rope else (None, None)
        got = kv.qk_norm_rope_backward(g[:, :hq], g[:, hq:], x[:, :hq], x[:, hq:], *t, wq, wk, norm=norm, halves=halves and rope)
        for part, w, dx, dw in ((slice(0, hq), wq, got[0], got[2]), (slice(hq, None), wk, got[1], got[3])):
            want, size, wdw, wsize = _backward64(g[:, part], x[:, part], w, *t, None, 1e-6, norm, halves)
            _check16(dx, want, size, dtype, f"dx {norm} {rope}")
            # fp32 sums over tokens and heads: at most 2^11 roundings deep each way
            assert bool(((dw.double().cpu() - wdw).abs() <= 2.0 ** -13 * wsize + 1e-30).all()), "dw"
    again = kv.qk_norm_rope_backward(g[:, :hq], g[:, hq:], x[:, :hq], x[:, hq:], cos, sin, wq, wk, halves=halves)
    once = kv.qk_norm_rope_backward(g[:, :hq], g[:, hq:], x[:, :hq], x[:, hq:], cos, sin, wq, wk, halves=halves)
    assert all(torch.equal(a, b) for a, b in zip(again, once))            # the same bits every time


@pytest.mark.parametrize("halves", [False, True])
def test_gradient_against_differences(halves):
    """Central differences of the 64-bit definition, step 1e-4: their error is
    the third derivative's, below 1e-5 of the gradient's size here."""
    torch, kv = _torch()
    x, g = _rows(21, "f16", 3, 2, 32), _rows(22, "f16", 3, 2, 32)
    w = 1 + _rows(23, "f16", 32, size=0.3)
    cos, sin = _tables(3, 32)
    dq, _, dwq, _ = kv.qk_norm_rope_backward(g, g, x, x, cos, sin, w, w, halves=halves)

    def loss(xx, ww):
        y = xx / torch.sqrt((xx * xx).mean(-1, keepdim=True) + 1e-6) * ww
        a, b = _pairs(y, halves)
        c, s = cos.double().cpu()[:, None], sin.double().cpu()[:, None]
        return (_join(a * c - b * s, a * s + b * c, halves) * g.double().cpu()).sum()
    x64, w64, e = x.double().cpu(), w.double().cpu(), 1e-4
    for i in range(0, x64.numel(), 5):
        d = torch.zeros(x64.numel(), dtype=torch.float64)
        d[i] = e
        num = (loss(x64 + d.view_as(x64), w64) - loss(x64 - d.view_as(x64), w64)) / (2 * e)
        assert abs(float(num) - float(dq.flatten()[i])) <= 2.0 ** -11 * abs(float(num)) + 2e-5
    for i in range(32):
        d = torch.zeros(32, dtype=torch.float64)
        d[i] = e
        num = (loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * e)
        assert abs(float(num) - float(dwq[i])) <= 2e-5


def test_autograd_function():
    torch, kv = _torch()
    q, k = _rows(31, "bf16", 9, 4, 64).requires_grad_(), _rows(32, "bf16", 9, 2, 64).requires_grad_()
    wq, wk = (_rows(33, "bf16", 64).requires_grad_() for _ in range(2))
    cos, sin = _tables(9, 64)
    yq, yk = kv.qk_norm_rope_autograd(q, k, wq, wk, cos, sin, halves=True)
    g = _rows(34, "bf16", 9, 4, 64)
    ((yq * g).sum() + yk.sum()).backward()                # yk's gradient arrives with zero strides
    dq, dk, dwq, dwk = kv.qk_norm_rope_backward(g, torch.ones_like(yk), q.detach(), k.detach(), cos, sin, wq.detach(), wk.detach(), halves=True)
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)
    assert torch.equal(wq.grad, dwq.bfloat16()) and torch.equal(wk.grad, dwk.bfloat16())


def test_gradient_of_no_tokens():
    torch, kv = _torch()
    z = torch.empty((0, 3, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    dq, dk, dwq, dwk = kv.qk_norm_rope_backward(z, z, z, z, wq=w, wk=w)
    assert dq.shape == dk.shape == (0, 3, 64) and bool((dwq == 0).all()) and bool((dwk == 0).all())


# ------------------------------------------------------------------------ cache
FMTS = {"mxfp4_g32": o.MXFP4, "int4_g64": o.INT4}


def _cache(pages, page, heads, dim, fmt, fill=None):
    _, kv = _torch()
    from diffusion_smooth_group_amd import svdq as S
    c = kv.KVCache(pages, page, heads, dim, S.FMT_CODES[fmt])
    if fill is not None:
        for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
            t.view(__import__("torch").uint8).fill_(fill)
    return c


def _oracle_codes(x, fmt):
    """Nibbles [T, H, D] and scale bits of rows x, by the oracle's quantizers."""
    v = x.float().cpu().numpy()
    grp = 32 if fmt == "mxfp4_g32" else 64
    q, s = (o.quant_mxfp4_g32 if grp == 32 else o.quant_int4_g64)(v.reshape(*v.shape[:-1], -1, grp))
    q = q.reshape(v.shape)
    if grp == 64:
        q = np.where(q < 0, 8 | -q, q)
    return q.astype(np.uint8), s


def _held(c, slots, which):
    codes, scales = (c.k_codes, c.k_scales) if which == 0 else (c.v_codes, c.v_scales)
    page, at = slots.long() // c.page_size, slots.long() % c.page_size
    b = codes[page, :, at].cpu().numpy()
    n = np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)
    s = scales[page, :, at].cpu().numpy()
    return n, s.view(np.uint16) if s.dtype == np.float16 else s


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (100, 3, 128, 64), (257, 8, 64, 32), (70, 2, 128, 256)])
def test_append_is_the_oracles_quantizer_and_read_returns_it(dtype, fmt, tokens, heads, dim, page):
    torch, kv = _torch()
    kvrow = _rows(tokens, dtype, tokens, 2 * heads, dim, size=2.0)
    kvrow[0, 0, :8] = 0
    kvrow[tokens // 2, heads] = 0                         # an all-zero row of V
    kvrow[tokens - 1, heads - 1] *= 2.0 ** -12            # small values
    k, v = kvrow[:, :heads], kvrow[:, heads:]
    pages = -(-tokens // page) + 2
    c = _cache(pages, page, heads, dim, fmt, fill=0xA5)
    before = c.k_codes.clone()
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(7))[:tokens].int().cuda()
    c.append(k, v, slots)
    for which, x in ((0, k), (1, v)):
        want, ws = _oracle_codes(x, fmt)
        got, gs = _held(c, slots, which)
        # a negative zero may be held as either zero
        same = (got == want) | (((got | want) & 7) == 0)
        assert same.all() and np.array_equal(gs, ws)
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots.cpu().long()] = False
    flat = lambda t: t.transpose(1, 2).reshape(pages * page, heads, dim // 2).cpu()[rest]   # noqa: E731
    assert torch.equal(flat(c.k_codes), flat(before))     # nothing else is written
    rk, rv = c.read(slots, dtype=_dtype(dtype))
    for x, r in ((k, rk), (v, rv)):
        q, s = _oracle_codes(x, fmt)
        grp = 32 if fmt == "mxfp4_g32" else 64
        table = np.array([0, .5, 1, 1.5, 2, 3, 4, 6]) if grp == 32 else np.arange(8.0)
        step = np.ldexp(1.0, s.astype(int) - 127) if grp == 32 else s.view(np.float16).astype(float)
        val = np.where(q >= 8, -1, 1) * table[q & 7] * np.repeat(step, grp, -1).reshape(q.shape)
        assert torch.equal(r.cpu(), torch.from_numpy(val).to(_dtype(dtype)))


def test_append_skips_slots_outside_and_read_gives_zeros_there():
    torch, kv = _torch()
    c = _cache(2, 16, 2, 64, "int4_g64", fill=0x11)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    x = _rows(3, "f16", 4, 2, 64)
    outside = torch.tensor([-1, 32, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    c.append(x, x, outside)
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)))
    k, v = c.read(outside, dtype=torch.float16)
    assert bool((k == 0).all()) and bool((v == 0).all())


@pytest.mark.parametrize("fmt", list(FMTS))
def test_append_holds_special_values_finite(fmt):
    torch, kv = _torch()
    c = _cache(1, 16, 1, 64, fmt)
    x = _rows(4, "bf16", 5, 1, 64)
    x[0, 0, 3], x[1, 0, 3], x[2, 0, 3] = float("nan"), float("inf"), float("-inf")
    x[3] = 3.0e38
    x[4] = 1e-38
    s = torch.arange(5, dtype=torch.int32, device="cuda")
    c.append(x, x, s)
    k, _ = c.read(s, dtype=torch.bfloat16)
    assert bool(k.isfinite().all())
    clean = x.clone()
    clean[0, 0, 3] = 0
    c.append(clean, clean, s)
    assert torch.equal(c.read(s, dtype=torch.bfloat16)[0][0], k[0])       # a NaN is a zero
    assert float(k[1, 0, 3]) == float(k[1].max()) > 1e4 and float(k[2, 0, 3]) < -1e4


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("halves", [False, True])
def test_fused_append_is_norm_rope_then_append(dtype, fmt, halves):
    torch, kv = _torch()
    t, hq, hk, dim = 51, 6, 3, 128
    qkv = _rows(8, dtype, t, hq + 2 * hk, dim)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wq, wk = 1 + _rows(1, dtype, dim, size=0.3), 1 + _rows(2, dtype, dim, size=0.3)
    cos, sin = _tables(t + 3, dim)
    pos = (torch.arange(t, dtype=torch.int32) + 2).cuda()
    slots = torch.randperm(64)[:t].int().cuda()
    a, b = _cache(4, 16, hk, dim, fmt), _cache(4, 16, hk, dim, fmt)
    args = dict(cos=cos, sin=sin, wq=wq, wk=wk, norm=True, halves=halves, positions=pos)
    q1 = a.append(k, v, slots, q=q, **args)
    q2, k2 = kv.qk_norm_rope(q, k, **args)
    b.append(k2, v, slots)
    assert torch.equal(q1, q2)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


# ------------------------------------------------------------------------- plan
def _plan_loops(past, fresh, table, free, count, page, tokens):
    table, taken, wanted = table.copy(), 0, 0
    q_start, kv_len, slots, positions = [0], [], [], []
    for r, (p, f) in enumerate(zip(past, fresh)):
        p, f = max(p, 0), max(f, 0)
        for col in range(-(-p // page), -(-(p + f) // page)):
            got = -1
            if wanted < count:
                got = free[count - 1 - wanted]
                taken += 1
            wanted += 1
            if col < table.shape[1]:
                table[r, col] = got
        for t in range(p, p + f):
            pg = table[r, t // page] if t // page < table.shape[1] else -1
            slots.append(-1 if pg < 0 else pg * page + t % page)
            positions.append(t)
        q_start.append(q_start[-1] + f)
        kv_len.append(p + f)
    slots = (slots + [-1] * tokens)[:tokens]
    positions = (positions + [0] * tokens)[:tokens]
    return table, q_start, kv_len, slots, positions, count - taken, max(0, wanted - count)


@pytest.mark.parametrize("requests,page,most_past,most_fresh,free,width,extra", [
    (1, 16, 0, 1, 5, 4, 0), (1, 64, 5000, 3000, 200, 200, 0), (5, 16, 40, 33, 100, 8, 7), (300, 32, 300, 1, 400, 12, 0),
    (257, 16, 100, 20, 90, 9, 3),          # the free list runs out
    (40, 16, 200, 60, 2000, 6, 0),         # tables too narrow
    (1023, 128, 2000, 5, 4000, 17, 100), (8192, 16, 50, 3, 9000, 5, 1)])
def test_plan_against_loops(requests, page, most_past, most_fresh, free, width, extra):
    torch, kv = _torch()
    rng = np.random.default_rng(requests + page)
    past = rng.integers(0, most_past + 1, requests)
    fresh = rng.integers(0 if requests > 1 else most_fresh, most_fresh + 1, requests)
    if requests > 4:
        past[3], fresh[1] = -5, -2                        # count as zero
    order = rng.permutation(free + 200000)
    pool = order[:free].astype(np.int32)
    table = np.full((requests, width), -1, np.int32)
    at = free
    for r in range(requests):
        n = min(width, -(-max(past[r], 0) // page))
        table[r, :n] = order[at:at + n]
        at += n
    count = max(0, free - 3)
    tokens = int(np.maximum(fresh, 0).sum()) + extra
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()   # noqa: E731
    want = _plan_loops(past, fresh, table, pool, count, page, tokens)
    got = kv.plan(dev(past), dev(fresh), dev(table), dev(pool), dev([count]), page, tokens)
    for g, w, name in zip(got, want, kv.Plan._fields):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name


def test_plan_without_requests_and_with_too_few_token_slots():
    torch, kv = _torch()
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.empty(0, **i32)
    p = kv.plan(none, none, torch.empty((0, 4), **i32), torch.arange(3, **i32), torch.tensor([3], **i32), 16, 5)
    assert p.q_start.tolist() == [0] and p.slots.tolist() == [-1] * 5 and p.free_count.tolist() == [3] and p.missing.tolist() == [0]
    p = kv.plan(torch.tensor([0, 0], **i32), torch.tensor([20, 20], **i32), torch.full((2, 2), -1, **i32), torch.arange(9, **i32),
                torch.tensor([9], **i32), 16, 25)          # 40 new tokens, a map of 25
    assert p.slots.tolist() == [128 + i for i in range(16)] + [112 + i for i in range(4)] + [96 + i for i in range(5)]
    assert p.block_table.tolist() == [[8, 7], [6, 5]] and p.q_start.tolist() == [0, 20, 40]


def test_release_returns_pages_in_order():
    torch, kv = _torch()
    rng = np.random.default_rng(5)
    requests, page, width, cap = 37, 16, 300, 9000
    lens = rng.integers(0, 300 * 16, requests)
    table = np.full((requests, width), -1, np.int32)
    pages = rng.permutation(8000).astype(np.int32)
    at = 0
    for r in range(requests):
        n = -(-lens[r] // page)
        table[r, :n] = pages[at:at + n]
        at += n
    table[4, 2] = -1                                       # a page that was missing
    done = rng.integers(0, 2, requests)
    done[4] = 1
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()   # noqa: E731
    for capacity in (cap, 50):
        t, kl, free, cnt = dev(table), dev(lens), dev(np.full(capacity, -7)), dev([11])
        kv.release(dev(done), t, kl, free, cnt, page)
        back = [int(p) for r in range(requests) if done[r] for p in table[r, :-(-lens[r] // page)] if p >= 0]
        room = min(len(back), capacity - 11)
        assert cnt.tolist() == [11 + room]
        assert free.tolist() == [-7] * 11 + back[:room] + [-7] * (capacity - 11 - room)
        for r in range(requests):
            assert int(kl[r]) == (0 if done[r] else lens[r])
            assert bool((t[r] == -1).all()) if done[r] else np.array_equal(t[r].cpu().numpy(), table[r])
