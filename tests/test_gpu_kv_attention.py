"""GPU tests of the attention over the 4-bit cache against the definition in
64 bits on the values that the cache holds."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _mods():
    import torch

    from diffusion_smooth_group_amd import kv
    from diffusion_smooth_group_amd import svdq as S
    return torch, kv, S


def _setup(fmt, dtype, dim, page, hk, group, fresh, lens, seed=1, k_size=1.0, q_size=1.5, spare=3):
    """A cache with rows appended through the library, in shuffled pages; slots
    that hold no token are filled with NaN scales."""
    torch, kv, S = _mods()
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    cache = kv.KVCache(pool, page, hk, dim, S.FMT_CODES[fmt])
    cache.k_codes.fill_(0x77), cache.v_codes.fill_(0x7F)
    for s in (cache.k_scales, cache.v_scales):
        s.fill_(255 if fmt == "mxfp4_g32" else float("nan"))
    order = torch.randperm(pool, generator=g).int()
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    slots = torch.cat([table[r].repeat_interleave(page)[:n] * page + torch.arange(n) % page for r, n in enumerate(lens)]
                      + [torch.empty(0, dtype=torch.int64)]).int().cuda()
    total = sum(lens)
    k = (torch.randn((total, hk, dim), generator=g) * k_size).to(dt).cuda()
    v = (torch.randn((total, hk, dim), generator=g) + 0.5).to(dt).cuda()
    if total:
        cache.append(k, v, slots)
    q = (torch.randn((sum(fresh), hk * group, dim), generator=g) * q_size).to(dt).cuda()
    start = torch.tensor(np.concatenate(([0], np.cumsum(fresh))), dtype=torch.int32).cuda()
    return cache, table.cuda(), slots, q, start, torch.tensor(lens, dtype=torch.int32).cuda()


def _values64(cache, slots, fmt):
    torch, _, _ = _mods()
    out = []
    page, at = slots.long() // cache.page_size, slots.long() % cache.page_size
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        b, s = codes[page, :, at].cpu(), scales[page, :, at].cpu()
        n = torch.stack((b & 15, b >> 4), -1).flatten(-2).long()
        mx = fmt == "mxfp4_g32"
        mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6] if mx else list(range(8)), dtype=torch.float64)
        val = torch.where(n >= 8, -mag[n & 7], mag[n & 7])
        step = 2.0 ** (s.double() - 127) if mx else s.double()
        out.append(val * step.repeat_interleave(32 if mx else 64, -1))
    return out


def _reference(q, k, v, fresh, lens, group, causal, window, scale):
    """out, lse, the sum of |p v| and the size of the logits' terms, 64 bits."""
    torch, _, _ = _mods()
    q = q.double().cpu()
    out, size, lse = torch.zeros_like(q), torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    terms = 0.0
    row = at = 0
    for n, length in zip(fresh, lens):
        for i in range(n):
            pos = length - n + i
            hi = min(pos + 1, length) if causal else length
            lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                continue
            kk, vv = k[at + lo:at + hi], v[at + lo:at + hi]
            for j in range(q.shape[1]):
                h = j // group
                x = kk[:, h] @ q[row + i, j] * scale
                terms = max(terms, float((kk[:, h].abs() @ q[row + i, j].abs()).max()) * abs(scale))
                p = torch.softmax(x, 0)
                out[row + i, j], size[row + i, j] = p @ vv[:, h], p @ vv[:, h].abs()
                lse[row + i, j] = torch.logsumexp(x, 0)
        row += n
        at += length
    return out, lse, size, terms


def _check(got, lse, ref, dtype, dim, what=""):
    """Probabilities and (INT4) values are rounded to 16 bits once each, the
    result once: 3 half-ulps of sum |p v|.  A logit is an fp32 sum of D products
    (error at most D 2^-24 of its terms' size), which moves p by as much, twice
    over in the quotient; exp2, sums and log2 add a few 2^-22."""
    out, want_lse, size, terms = ref
    logit = dim * 2.0 ** -24 * terms + 2.0 ** -18
    err = (got.double().cpu() - out).abs()
    tol = (3 * ULP[dtype] + 2 * logit) * size + 2.0 ** -24
    assert bool(got.isfinite().all()), what
    assert bool((err <= tol).all()), f"{what}: out at {float((err / tol.clamp(min=1e-30)).max()):.3f} of the tolerance"
    if lse is not None:
        lse = lse.double().cpu()
        empty = want_lse == -math.inf
        assert bool((lse[empty] == -math.inf).all()) and bool((got.cpu()[empty] == 0).all()), what
        e = (lse[~empty] - want_lse[~empty]).abs()
        assert bool((e <= logit + 2.0 ** -21 * want_lse[~empty].abs() + 2.0 ** -19).all()), f"{what}: lse {float(e.max())}"


def _run(fmt, dtype, dim, page, hk, group, fresh, lens, causal=True, window=0, scale=None, **kw):
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup(fmt, dtype, dim, page, hk, group, fresh, lens, **kw)
    out, lse = kv.attention(q, cache, table, start, length, max(fresh + [0]), max(lens + [0]), causal, window, scale,
                            return_lse=True)
    k, v = _values64(cache, slots, fmt)
    ref = _reference(q, k, v, fresh, lens, group, causal, window, 1 / math.sqrt(dim) if scale is None else scale)
    _check(out, lse, ref, dtype, dim, f"{fmt} {dtype} {dim} {page} {hk}x{group} {fresh} {lens} {causal} {window}")
    return out


FORMS = [(f, t, d) for f in ("mxfp4_g32", "int4_g64") for t in ("bf16", "f16") for d in (64, 128)]


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
@pytest.mark.parametrize("page,hk,group,fresh,lens", [
    (16, 1, 1, [1], [1]),
    (16, 2, 1, [1, 1, 1], [31, 32, 33]),
    (32, 2, 4, [1, 1, 1, 1], [5, 129, 64, 500]),
    (64, 1, 16, [1, 1], [127, 700]),
    (128, 3, 5, [2, 3], [130, 257]),
    (16, 1, 24, [1, 2], [65, 47]),              # more rows than one tile holds
    (256, 1, 1, [1], [3000]),                   # chunks that are joined
])
def test_few_rows(fmt, dtype, dim, page, hk, group, fresh, lens):
    _run(fmt, dtype, dim, page, hk, group, fresh, lens)


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
@pytest.mark.parametrize("fresh,lens,causal,window", [
    ([1, 1], [5200, 1025], True, 0),            # more than 16 chunks
    ([1], [70000], True, 0),                    # more than 256
    ([2, 1], [1024, 900], True, 0),             # one, of eight tiles a wave
    ([3, 1], [9000, 6000], True, 5000),
    ([3, 1], [9000, 100], False, 4200),
])
def test_few_rows_in_chunks(fmt, dtype, dim, fresh, lens, causal, window):
    _run(fmt, dtype, dim, 64, 1, 2, fresh, lens, causal, window)


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
@pytest.mark.parametrize("page,hk,group,fresh,lens,causal,window", [
    (16, 1, 2, [40], [40], True, 0),
    (64, 2, 1, [129], [129], False, 0),
    (32, 1, 4, [33, 64, 1], [100, 64, 200], True, 0),
    (16, 1, 3, [70, 5], [150, 90], True, 37),
    (64, 2, 2, [65], [300], False, 100),
    (128, 1, 1, [200], [333], True, 1),
])
def test_prompts(fmt, dtype, dim, page, hk, group, fresh, lens, causal, window):
    _run(fmt, dtype, dim, page, hk, group, fresh, lens, causal, window)


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 50)])
def test_many_requests_of_wide_tiles(fmt, dtype, dim, causal, window):
    """Tiles of 256 rows: enough requests and heads for half the compute units."""
    fresh = [81 + r % 3 * 40 for r in range(22)]
    _run(fmt, dtype, dim, 32, 3, 2, fresh, [n + 61 * (r % 4) for r, n in enumerate(fresh)], causal, window)


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
def test_wide_tiles_in_joined_chunks(fmt, dtype, dim):
    """Few requests and heads: tiles of 128 rows over chunks of a long cache,
    and rows just under what they take (tiles of 16)."""
    _run(fmt, dtype, dim, 64, 3, 4, [90], [2500])
    _run(fmt, dtype, dim, 16, 9, 2, [70], [1800], True, 1100)
    _run(fmt, dtype, dim, 64, 1, 1, [100], [2500])


@pytest.mark.parametrize("fmt,dtype", [("mxfp4_g32", "bf16"), ("int4_g64", "f16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 3)])
def test_requests_without_rows_tokens_or_visible_keys(fmt, dtype, causal, window):
    # no rows; no tokens at all; rows before the first cached token (they see
    # nothing when causal); one token
    _run(fmt, dtype, 64, 16, 2, 2, [0, 3, 9, 1, 40], [50, 0, 4, 1, 17], causal, window)


@pytest.mark.parametrize("fmt,dtype,dim", FORMS)
def test_scales_of_logits_and_of_values(fmt, dtype, dim):
    _run(fmt, dtype, dim, 16, 1, 2, [3], [200], scale=-0.3)                 # largest logits first under a negative scale
    _run(fmt, dtype, dim, 16, 1, 2, [3], [200], scale=0.0)                  # a plain mean
    _run(fmt, dtype, dim, 16, 1, 2, [40], [200], k_size=8.0, q_size=6.0)    # one key takes all
    _run(fmt, dtype, dim, 16, 1, 2, [1], [300], k_size=2.0 ** -9)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("f16", 64), ("f16", 128)])
@pytest.mark.parametrize("fresh", [[1], [90]])
def test_value_scales_near_the_end_of_f16(dtype, dim, fresh):
    """INT4 values past f16's range (7 x 65504) beside ones of ordinary size, in
    some keys of a tile and in whole tiles."""
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("int4_g64", dtype, dim, 16, 1, 2, fresh, [300])
    top = 65504.0 if dtype == "bf16" else 9000.0           # 7 x 9000 is what an f16 result holds
    s = cache.v_scales.view(-1, dim // 64)
    at = slots.long()
    for keys, scale in ((at[37], top), (at[150:155], 8191.0), (at[155:160], 8192.0), (at[192:256], top / 2)):
        s[keys] = scale
    assert torch.equal(cache.v_scales.view(-1, dim // 64)[at[37]], torch.full((dim // 64,), top, device="cuda").half())
    out, lse = kv.attention(q, cache, table, start, length, max(fresh), 300, return_lse=True)
    k, v = _values64(cache, slots, "int4_g64")
    assert float(v.abs().max()) > 50000
    _check(out, lse, _reference(q, k, v, fresh, [300], 2, True, 0, dim ** -0.5), dtype, dim)


@pytest.mark.parametrize("fresh", [[1, 1], [30, 4]])
def test_bounds_pages_outside_the_cache_and_bad_lengths(fresh):
    """Missing pages are not seen; max_q, max_kv and the table's width bound
    what is read."""
    torch, kv, _ = _mods()
    lens = [90, 70]
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "bf16", 64, 16, 1, 2, fresh, lens)
    k, v = _values64(cache, slots, "mxfp4_g32")
    for bad in (-1, cache.n_pages, 1 << 30, -(1 << 31)):
        t = table.clone()
        t[0, 1] = bad                                      # tokens 16..31 of request 0
        out, lse = kv.attention(q, cache, t, start, length, max(fresh), 90, return_lse=True)
        gone = torch.ones(160, dtype=torch.bool)
        gone[16:32] = False
        rows = [r for r in range(q.shape[0])]
        at = row = 0
        for n, ln in zip(fresh, lens):
            for i in range(n):
                see = gone[at:at + ln].clone()
                see[ln - n + i + 1:] = False
                for j in range(2):
                    x = torch.where(see, k[at:at + ln, 0] @ q[row + i, j].double().cpu() / 8, torch.tensor(-math.inf, dtype=torch.float64))
                    want = torch.softmax(x, 0) @ v[at:at + ln, 0]
                    assert float((out[row + i, j].double().cpu() - want).abs().max()) < 0.03
                    assert abs(float(lse[row + i, j]) - float(torch.logsumexp(x, 0))) < 1e-3
            row += n
            at += ln
        assert rows
    # a length past the table: the table's pages are all that is seen
    long = kv.attention(q, cache, table[:, :3].contiguous(), start, length, max(fresh), 1 << 30, causal=False)
    short = kv.attention(q, cache, table, start, torch.tensor([48, 48], dtype=torch.int32, device="cuda"), max(fresh), 90, causal=False)
    assert torch.equal(long, short)
    # max_kv below the length
    cut = kv.attention(q, cache, table, start, length, max(fresh), 48, causal=False)
    assert torch.equal(cut, short)
    # rows past max_q are left alone
    keep = torch.full_like(q, 3.0)
    kv.attention(q, cache, table, start, length, 1, 90, out=keep)
    row = 0
    for n in fresh:
        assert bool((keep[row + 1:row + n] == 3.0).all()) and not bool((keep[row] == 3.0).all())
        row += n
    # offsets that are no offsets
    keep.fill_(3.0)
    wild = torch.tensor([0, 1 << 30, -5], dtype=torch.int32, device="cuda")
    kv.attention(q, cache, table, wild, length, max(fresh), 90, out=keep)


def test_strided_rows_and_other_stream_and_graph():
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("int4_g64", "bf16", 128, 32, 2, 4, [1, 1, 1], [900, 33, 257])
    want, lse = kv.attention(q, cache, table, start, length, 1, 900, return_lse=True)
    row = torch.randn((3, 12, 128), device="cuda").bfloat16()
    row[:, 2:10] = q
    outs = torch.zeros((3, 8, 3, 128), device="cuda").bfloat16()
    got = kv.attention(row[:, 2:10], cache, table, start, length, 1, 900, out=outs[:, :, 1])
    assert torch.equal(got, want) and bool((outs[:, :, 0] == 0).all()) and bool((outs[:, :, 2] == 0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = kv.attention_workspace(3, 3, 8, cache, 1, 900)
    out = torch.empty_like(q)
    with torch.cuda.stream(side):
        kv.attention(q, cache, table, start, length, 1, 900, out=out, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    other = torch.empty_like(q)
    kv.attention(q, cache, table, start, length, 1, 900, out=other, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kv.attention(q, cache, table, start, length, 1, 900, out=out, ws=ws)
    for n in (900, 300, 900):                              # lengths may change between replays
        length[0] = n
        out.fill_(0)
        eager = kv.attention(q, cache, table, start, length, 1, 900)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_same_bits_every_time():
    torch, kv, _ = _mods()
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "f16", 128, 64, 2, 4, [1, 40], [5000, 777])
    first = kv.attention(q, cache, table, start, length, 40, 5000, return_lse=True)
    for _ in range(5):
        again = kv.attention(q, cache, table, start, length, 40, 5000, return_lse=True)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_cache_past_4_gib_of_codes():
    """Pages whose bytes lie past 2^32 in a code buffer."""
    torch, kv, S = _mods()
    pages, page, heads, dim = 1 << 17, 64, 9, 128          # 4.5 GiB of codes each
    cache = kv.KVCache(pages, page, heads, dim, S.FMT_MXFP4_G32)
    ids = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    n = 150
    slots = (ids[0].repeat_interleave(page)[:n] * page + torch.arange(n) % page).int().cuda()
    k, v = ((torch.randn((n, heads, dim)) + 0.3).bfloat16().cuda() for _ in range(2))
    q = torch.randn((1, heads, dim)).bfloat16().cuda()
    cache.append(k, v, slots)
    k64, v64 = _values64(cache, slots, "mxfp4_g32")
    rk, _ = cache.read(slots)
    assert torch.equal(rk.double().cpu(), k64)
    i32 = dict(dtype=torch.int32, device="cuda")
    out, lse = kv.attention(q, cache, ids.cuda(), torch.tensor([0, 1], **i32), torch.tensor([n], **i32), 1, n, return_lse=True)
    _check(out, lse, _reference(q, k64, v64, [1], [n], 1, True, 0, dim ** -0.5), "bf16", dim)
    q2 = torch.randn((100, heads, dim)).bfloat16().cuda()
    out, lse = kv.attention(q2, cache, ids.cuda(), torch.tensor([0, 100], **i32), torch.tensor([n], **i32), 100, n, return_lse=True)
    _check(out, lse, _reference(q2, k64, v64, [100], [n], 1, True, 0, dim ** -0.5), "bf16", dim)


def test_refusals_in_python():
    torch, kv, S = _mods()
    cache, table, slots, q, start, length = _setup("mxfp4_g32", "bf16", 64, 16, 2, 2, [1], [20])
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(block_table=table.long()), dict(q_start=start[:1]),
                dict(kv_len=length.float()), dict(out=q[:, :2].float())):
        args = dict(q=q, cache=cache, block_table=table, q_start=start, kv_len=length, max_q=1, max_kv=20) | bad
        with pytest.raises(ValueError):
            kv.attention(**args)
    with pytest.raises(kv.SvdqError):
        kv.attention(q[:, :3], cache, table, start, length, 1, 20)
    with pytest.raises(ValueError):
        kv.KVCache.wrap(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, "int4_g64")
    with pytest.raises(kv.SvdqError):
        kv.KVCache(2, 24, 1, 64, S.FMT_MXFP4_G32)
    with pytest.raises(ValueError):
        cache.append(q[:, :2], q[:, :2], slots[:3])
