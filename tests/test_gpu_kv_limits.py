"""GPU tests of the cache operators at the limits of their arguments: bounds
that say "no bound", streams, workspaces, small scales."""
import pytest

from tests.test_gpu_kv_attention import _check, _mods, _reference, _setup, _values64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype,dim", [("mxfp4_g32", "bf16", 128), ("int4_g64", "f16", 64)])
@pytest.mark.parametrize("requests,heads,group,rows", [(1, 1, 2, 1), (300, 8, 2, 1), (600, 2, 1, 3), (12, 4, 2, 65)])
def test_max_kv_without_a_bound(fmt, dtype, dim, requests, heads, group, rows):
    """INT32_MAX as max_kv, with few and with more than enough work for one
    workgroup a row tile: bit for bit the result of the exact bound."""
    torch, kv, _ = _mods()
    lens = [rows + 17 * r % 90 for r in range(requests)]
    cache, table, slots, q, start, length = _setup(fmt, dtype, dim, 16, heads, group, [rows] * requests, lens)
    for causal, window in ((True, 0), (False, 0), (True, 20)):
        want, wl = kv.attention(q, cache, table, start, length, rows, max(lens), causal, window, return_lse=True)
        got, gl = kv.attention(q, cache, table, start, length, rows, (1 << 31) - 1, causal, window, return_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    every, _ = kv.attention(q, cache, table, start, length, rows, (1 << 31) - 1, True, (1 << 31) - 1, return_lse=True)
    assert torch.equal(every, kv.attention(q, cache, table, start, length, rows, max(lens)))
    k, v = _values64(cache, slots, fmt)
    few = min(requests, 4)
    n, keys = rows * few, sum(lens[:few])
    out, lse = kv.attention(q, cache, table, start, length, rows, (1 << 31) - 1, return_lse=True)
    ref = _reference(q[:n], k[:keys], v[:keys], [rows] * few, lens[:few], group, True, 0, dim ** -0.5)
    _check(out[:n], lse[:n], ref, dtype, dim)


def test_rows_before_the_first_token_under_the_widest_window():
    """More rows than tokens, no causal mask, a window of INT32_MAX: every row
    sees every key."""
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "bf16", 64, 16, 1, 1, [9, 120], [4, 50])
    want = kv.attention(q, cache, table, start, length, 120, 50, causal=False)
    assert torch.equal(kv.attention(q, cache, table, start, length, 120, 50, causal=False, window=(1 << 31) - 1), want)


def _scratch(monkeypatch, kv, name, at):
    """Where the calls of `name` had argument `at` (a pointer), in a list."""
    seen, call = [], kv._call

    def record(fn, *args):
        if fn == name:
            seen.append(args[at])
        return call(fn, *args)
    monkeypatch.setattr(kv, "_call", record)
    return seen


@pytest.mark.parametrize("raw", [False, True])
def test_scratch_and_outputs_belong_to_the_stream_of_the_call(monkeypatch, raw):
    """A call on another stream leaves no memory that the current stream's
    next allocations could take while its kernels still run."""
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "bf16", 128, 64, 2, 4, [1, 1], [8000, 5000])
    want, wl = kv.attention(q, cache, table, start, length, 1, 8000, return_lse=True)
    x, g = torch.randn((700, 6, 128), device="cuda").bfloat16(), torch.randn((700, 6, 128), device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    grads = kv.qk_norm_rope_backward(g, g, x, x, wq=w, wk=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = side.cuda_stream if raw else side
    taken = _scratch(monkeypatch, kv, "svdq_kv_attention", 5), _scratch(monkeypatch, kv, "svdq_qk_norm_rope_backward", 9)
    got, lse = kv.attention(q, cache, table, start, length, 1, 8000, return_lse=True, stream=stream)
    back = kv.qk_norm_rope_backward(g, g, x, x, wq=w, wk=w, stream=stream)
    sizes = (kv.attention_workspace_size(2, 2, 8, cache, 1, 8000), 2 * 132 * 128 * 4)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(20)]
    assert all(len(p) == 1 and p[0] for p in taken) and sizes[0] > 0
    for t in held:
        for p in taken:
            assert not t.data_ptr() <= p[0] < t.data_ptr() + t.numel()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, wl) and all(torch.equal(a, b) for a, b in zip(back, grads))


def test_every_call_takes_a_stream():
    torch, kv, S = _mods()
    i32 = dict(dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    cache = kv.KVCache(4, 16, 2, 64, S.FMT_MXFP4_G32)
    x = torch.randn((20, 2, 64), device="cuda").bfloat16()
    past, fresh, table = torch.zeros(1, **i32), torch.full((1,), 20, **i32), torch.full((1, 3), -1, **i32)
    free, count, done = torch.arange(4, **i32), torch.full((1,), 4, **i32), torch.ones(1, **i32)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        table.fill_(-1)
        torch.cuda.synchronize()
        p = kv.plan(past, fresh, table, free, count, 16, 20, stream=stream)
        cache.append(x, x, p.slots, stream=stream)
        k, v = cache.read(p.slots, stream=stream)
        out = kv.attention(x, cache, p.block_table, p.q_start, p.kv_len, 20, 20, stream=stream)
        y, _ = kv.qk_norm_rope(x, x, stream=stream)
        torch.cuda.synchronize()
        kv.release(done, p.block_table, p.kv_len, free, p.free_count, 16, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(k, v) and out.isfinite().all() and torch.equal(y, kv.qk_norm_rope(x, x)[0])
        assert sorted(free.tolist()) == [0, 1, 2, 3] and p.free_count.tolist() == [4] and p.block_table.tolist() == [[-1] * 3]
        free.copy_(torch.arange(4))


def test_workspaces_that_are_refused():
    torch, kv, _ = _mods()
    cache, table, _, q, start, length = _setup("mxfp4_g32", "bf16", 128, 64, 2, 4, [1], [5000])
    need = kv.attention_workspace_size(1, 1, 8, cache, 1, 5000)
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(need), torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            kv.attention(q, cache, table, start, length, 1, 5000, ws=ws)
    words = torch.empty(need // 4, dtype=torch.float32, device="cuda")        # bytes count, not elements
    assert torch.equal(kv.attention(q, cache, table, start, length, 1, 5000, ws=words), kv.attention(q, cache, table, start, length, 1, 5000))
    with pytest.raises(kv.SvdqError):
        kv.attention(q, cache, table, start, length, 1, 5000, ws=words[:-1])


def test_autograd_of_a_loss_over_all_heads():
    """The gradient of a sum over heads arrives with a head stride of 0."""
    torch, kv, _ = _mods()
    q, k = (torch.randn((9, h, 64), device="cuda").bfloat16().requires_grad_() for h in (4, 2))
    w, c = torch.rand(64, device="cuda").bfloat16(), torch.randn((9, 64), device="cuda").bfloat16()
    yq, yk = kv.qk_norm_rope_autograd(q, k, w, w, None, None)
    ((yq.sum(1) * c).sum() + (yk.sum(1) * c).sum()).backward()
    gq, gk = (c[:, None].expand(9, h, 64).contiguous() for h in (4, 2))
    dq, dk, _, _ = kv.qk_norm_rope_backward(gq, gk, q.detach(), k.detach(), wq=w, wk=w)
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)


@pytest.mark.parametrize("halves", [False, True])
def test_autograd_of_the_rotation_alone(halves):
    torch, kv, _ = _mods()
    q, k, gq = (torch.randn((9, h, 64), device="cuda").half() for h in (4, 2, 4))
    a = torch.rand((9, 32), device="cuda") * 6
    cos, sin = a.cos(), a.sin()
    q.requires_grad_(), k.requires_grad_()
    yq, yk = kv.qk_norm_rope_autograd(q, k, None, None, cos, sin, halves=halves, norm=False)
    want = kv.qk_norm_rope(q.detach(), k.detach(), cos, sin, norm=False, halves=halves)
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    ((yq * gq).sum() + yk.sum()).backward()
    dq, dk, _, _ = kv.qk_norm_rope_backward(gq, torch.ones_like(yk), q.detach(), k.detach(), cos, sin, norm=False, halves=halves)
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)


def test_one_workspace_serves_smaller_steps():
    """Sized once for prompts of many requests, used as they end."""
    torch, kv, _ = _mods()
    for requests, rows, length in ((1, 1, 8000), (3, 2, 5000), (1, 90, 2500), (2, 300, 3000)):
        cache, table, _, q, start, lens = _setup("mxfp4_g32", "bf16", 64, 64, 2, 4, [rows] * requests, [length] * requests)
        ws = kv.attention_workspace(300, 300 * 2048, 8, cache, 2048, 16384)
        want, wl = kv.attention(q, cache, table, start, lens, rows, length, return_lse=True)
        got, gl = kv.attention(q, cache, table, start, lens, rows, length, ws=ws, return_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_page_numbers_past_every_cache_give_no_slot(page):
    """Their slots would wrap to other requests' pages."""
    torch, kv, _ = _mods()
    i32 = dict(dtype=torch.int32, device="cuda")
    last = (1 << 31) // page - 1                           # its last slot is 2^31 - 1
    bad = [last + 1, 1 << 28, (1 << 28) + 5, (1 << 31) - 1]
    free = torch.tensor([*bad, last, 7], **i32)
    p = kv.plan(torch.zeros(6, **i32), torch.full((6,), 3, **i32), torch.full((6, 2), -1, **i32), free, torch.tensor([6], **i32), page, 18)
    slots = p.slots.view(6, 3).tolist()
    assert slots[0] == [7 * page + i for i in range(3)] and slots[1] == [last * page + i for i in range(3)]
    for row, number in zip(slots[2:], reversed(bad)):
        assert number > last and row == [-1] * 3
    held = p.block_table[:, 0].tolist()
    assert held == list(reversed(free.tolist()))           # the table has what the list had
    # the same for a page that the table held before
    table = torch.tensor([[1 << 28, -1]], **i32)
    p = kv.plan(torch.tensor([2], **i32), torch.tensor([3], **i32), table, free, torch.tensor([6], **i32), page, 3)
    assert p.slots.tolist() == [-1] * 3


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fresh,lens", [([1], [1]), ([1, 3], [40, 300]), ([1], [5200]), ([90], [400]), ([90], [2500]), ([200] * 20, [260] * 20)])
@pytest.mark.parametrize("which", ["small values", "small values in some keys", "small keys", "large keys", "large values", "all"])
def test_mxfp4_scales_that_f16_does_not_hold(dtype, dim, fresh, lens, which):
    """f16 has 40 binades, the cache's scales 253: values down to half an f16's
    last step and up to its end, keys under large and small queries, in all
    keys and in a few (so that some row tiles and chunks meet them and others
    do not)."""
    torch, kv, _ = _mods()
    group = 2 if len(fresh) < 3 else 3
    heads = 1 if len(fresh) < 3 else 7
    q_size = {"small keys": 20000.0, "large keys": 2.0 ** -17}.get(which, 1.5)
    cache, table, slots, q, start, length = _setup("mxfp4_g32", dtype, dim, 32, heads, group, fresh, lens, q_size=q_size)
    q.clamp_(-6e4, 6e4)
    at = slots.long()
    page, row = at // 32, at % 32
    ks, vs, vc = (t[page, :, row].clone() for t in (cache.k_scales, cache.v_scales, cache.v_codes))
    some = torch.arange(at.numel(), device="cuda") % 97 == 0
    some[:1] = True
    if which in ("small values", "all"):
        vs[:] = 127 - 21 - (torch.arange(dim // 32, device="cuda") % 4).byte()
    if which == "small values in some keys":
        vs[some] = 127 - 24
    if which in ("small keys", "all"):
        ks[:] -= 15 if which == "small keys" else 0
        ks[some] -= 10
    if which == "large keys":
        ks[:] += 17
    if which in ("large values", "all"):
        vs[some], vc[some] = 143, 0x91                     # 0.5 and -0.5 times 2^16
    cache.k_scales[page, :, row], cache.v_scales[page, :, row], cache.v_codes[page, :, row] = ks, vs, vc
    out, lse = kv.attention(q, cache, table, start, length, max(fresh), max(lens), return_lse=True)
    k, v = _values64(cache, slots, "mxfp4_g32")
    few = 1 if len(fresh) > 2 else len(fresh)
    n, keys = sum(fresh[:few]), sum(lens[:few])
    ref = _reference(q[:n], k[:keys], v[:keys], fresh[:few], lens[:few], group, True, 0, dim ** -0.5)
    _check(out[:n], lse[:n], ref, dtype, dim, which)


@pytest.mark.parametrize("rows", [1, 90])
def test_mxfp4_groups_of_zeros_and_scales_next_to_nothing(rows):
    """All-zero groups have the smallest scale there is, and stand beside
    ordinary ones."""
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "f16", 128, 32, 1, 2, [rows], [200])
    v = torch.randn((200, 1, 128), device="cuda").half()
    v[::3] = 0
    v[:, :, 32:64] = 0
    cache.append(v, v, slots)
    k64, v64 = _values64(cache, slots, "mxfp4_g32")
    out, lse = kv.attention(q, cache, table, start, length, rows, 200, return_lse=True)
    _check(out, lse, _reference(q, k64, v64, [rows], [200], 2, True, 0, 128 ** -0.5), "f16", 128)
    assert bool((out[..., 32:64] == 0).all())


def test_offsets_that_are_no_offsets():
    """Request 0 says that it has 2^30 rows: those there are stand before its
    first token and see nothing; request 1 has none."""
    torch, kv, _ = _mods()
    for rows in (2, 34):
        cache, table, _, q, _, length = _setup("mxfp4_g32", "bf16", 64, 16, 1, 2, [rows, 3], [90, 70])
        wild = torch.tensor([0, 1 << 30, -5], dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        _, lse = kv.attention(q, cache, table, wild, length, rows - 1, 90, out=out, return_lse=True)
        assert bool((out[:rows - 1] == 0).all()) and bool((out[rows - 1:] == 3.0).all())
        assert bool((lse[:rows - 1] == -float("inf")).all())
        for wild in ([-7, -3, 2], [rows + 3, rows + 9, 1 << 30], [5, 2, 2], [-(1 << 31), (1 << 31) - 1, (1 << 31) - 1]):
            out.fill_(3.0)
            kv.attention(q, cache, table, torch.tensor(wild, dtype=torch.int32, device="cuda"), length, rows, 90, out=out)
            assert bool((out == 3.0).all()), wild


ROWS = [([1], 300, 1), ([1], 5200, 1), ([90], 400, 1), ([90], 2500, 1), ([200] * 20, 260, 7)]


def _bf16_operands(fmt, dtype, fresh):
    """Of the second product: few rows but f16 over INT4, many in bf16 over MXFP4."""
    return (fmt, dtype) == ("mxfp4_g32", "bf16") or fresh == [1] and (fmt, dtype) != ("int4_g64", "f16")


SPREADS = [(f, t, d, k, e, *r) for f in ("mxfp4_g32", "int4_g64") for t in ("f16", "bf16") for d in (64, 128)
           for k in ("groups", "keys", "one key", "unlikely key") for e in (16, 21, 26, 31) for r in ROWS
           if e == 16 or _bf16_operands(f, t, r[0])]


@pytest.mark.parametrize("fmt,dtype,dim,kind,apart,fresh,length,heads", SPREADS)
def test_value_scales_far_apart(fmt, dtype, dim, kind, apart, fresh, length, heads):
    """Values 2^apart below others: of the other column groups, of most keys, of
    all keys but one, and beside one key of next to no probability whose values
    make up for it.  The result is as precise where they count: up to 2^16 in
    every form, and without a limit where the second product's operands are bf16."""
    torch, kv, _ = _mods()
    group = 2
    lens = [length] * len(fresh)
    cache, table, slots, q, start, kv_len = _setup(fmt, dtype, dim, 32, heads, group, fresh, lens)
    at = slots.long()
    page, row = at // 32, at % 32
    mx = fmt == "mxfp4_g32"
    vs = cache.v_scales[page, :, row].clone()              # [tokens, heads, groups]
    top, step = (138, lambda e: 138 - e) if mx else (2048.0, lambda e: 2048.0 * 2.0 ** -e)
    low = step(apart)
    if kind == "groups":
        vs[..., 0] = top
        vs[..., 1:] = low
    elif kind == "keys":
        vs[:] = low
        vs[::61] = top
    else:
        vs[:] = low
        vs[length // 3::length] = top
    if kind == "unlikely key":                             # keys against positive queries: about e^-16 of the others
        q.copy_(q.abs().clamp_(0.5, 2.0))
        ks, kc = cache.k_scales[page, :, row].clone(), cache.k_codes[page, :, row].clone()
        ks[length // 3::length] = 126 if mx else 0.25      # 2^-1 and -3, 1/4 and -6: -1.5 each
        kc[length // 3::length] = 0xDD if mx else 0xEE
        if dim == 64:
            ks[length // 3::length] = 127 if mx else 0.5
        cache.k_scales[page, :, row], cache.k_codes[page, :, row] = ks, kc
    cache.v_scales[page, :, row] = vs
    out, lse = kv.attention(q, cache, table, start, kv_len, max(fresh), length, return_lse=True)
    k, v = _values64(cache, slots, fmt)
    n = fresh[0]
    ref = _reference(q[:n], k[:length], v[:length], fresh[:1], lens[:1], group, True, 0, dim ** -0.5)
    _check(out[:n], lse[:n], ref, dtype, dim, kind)
