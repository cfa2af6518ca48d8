"""Cases of the attention-side operators: what is measured, in plain torch and through the library.

The operators are those between a QKV projection and the attention output of a decoder that keeps its keys and values
in the library's 4-bit formats:

    norm_rope   RMS norm of every query and key head and the position rotation, one pass (forward, and its gradient)
    append      4-bit group quantization of new keys and values into a paged cache, and the read-back of the cache
    plan        block tables, slot map and positions of a step, from the requests' lengths
    attention   softmax attention over the 4-bit paged cache (single tokens, chunks of a prompt, whole prompts)

Cache layout (also the library's): codes uint8 [pages, heads, page_size, D / 2], element 2i in the low nibble of byte i;
mxfp4_g32: E2M1 codes and one e8m0 byte per 32 elements; int4_g64: sign (bit 3) and magnitude (bits 0-2), one fp16 scale
per 64 elements; scales [pages, heads, page_size, D / group].
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
GROUP = {"mxfp4_g32": 32, "int4_g64": 64}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # q and k of one image generation step of the 4608-token, 9216-wide QKV projection (24 heads of 128)
        {"name": "norm_rope 4608x24 bf16", "op": "norm_rope", "tokens": 4608, "q_heads": 24, "k_heads": 24, "dim": 128,
         "dtype": "bf16", "halves": False, "norm": True},
        # one decoding step of 64 requests with grouped heads: the latency of the call counts
        {"name": "norm_rope 64x32/8 f16", "op": "norm_rope", "tokens": 64, "q_heads": 32, "k_heads": 8, "dim": 128,
         "dtype": "f16", "halves": True, "norm": True},
        # training on the same 4608-token layer, an odd number of tokens
        {"name": "norm_rope_grad 4607x24 bf16", "op": "norm_rope_grad", "tokens": 4607, "q_heads": 24, "k_heads": 24,
         "dim": 128, "dtype": "bf16", "halves": False, "norm": True},
        # training of the 2048-token, 1280-wide layers: 20 heads of 64
        {"name": "norm_rope_grad 2048x20 f16", "op": "norm_rope_grad", "tokens": 2048, "q_heads": 20, "k_heads": 20,
         "dim": 64, "dtype": "f16", "halves": True, "norm": True},
        # one new token of 96 requests written into their pages, and the pages read back (swap-out)
        {"name": "append 96x8 int4 f16", "op": "append", "tokens": 96, "heads": 8, "dim": 128, "dtype": "f16",
         "fmt": "int4_g64", "page": 16},
        # a whole 4608-token prompt, all heads, written and read back
        {"name": "append 4608x24 mxfp4 bf16", "op": "append", "tokens": 4608, "heads": 24, "dim": 128, "dtype": "bf16",
         "fmt": "mxfp4_g32", "page": 64},
        # the scheduler's step for 512 decoding requests
        {"name": "plan 512 decode", "op": "plan", "requests": 512, "fresh": 1, "past": 8192, "page": 16},
        # the scheduler's step for 61 prompts of very different lengths
        {"name": "plan 61 prompts", "op": "plan", "requests": 61, "fresh": 2048, "past": 4096, "page": 64},
        # one token of one request, 20 heads of 64 with a cache of their own each: few rows, latency counts
        {"name": "attention 1x1 of 8192 int4 f16", "op": "attention", "requests": 1, "fresh": 1, "length": 8192,
         "q_heads": 20, "k_heads": 20, "dim": 64, "dtype": "f16", "fmt": "int4_g64", "page": 32, "causal": True,
         "window": 0},
        # a decoding batch with grouped heads and lengths up to 16384: the cache's bytes count
        {"name": "attention 48x1 of 16384 mxfp4", "op": "attention", "requests": 48, "fresh": 1, "length": 16384,
         "q_heads": 32, "k_heads": 8, "dim": 128, "dtype": "bf16", "fmt": "mxfp4_g32", "page": 64, "causal": True,
         "window": 0},
        # 4608 tokens that all see each other, 24 heads of 128: the matrix products count
        {"name": "attention 1x4608 full mxfp4", "op": "attention", "requests": 1, "fresh": 4608, "length": 4608,
         "q_heads": 24, "k_heads": 24, "dim": 128, "dtype": "bf16", "fmt": "mxfp4_g32", "page": 64, "causal": False,
         "window": 0},
        # chunks of five prompts behind what is cached of them already, odd lengths
        {"name": "attention 5x2047 of 8191 int4", "op": "attention", "requests": 5, "fresh": 2047, "length": 8191,
         "q_heads": 32, "k_heads": 8, "dim": 128, "dtype": "bf16", "fmt": "int4_g64", "page": 64, "causal": True,
         "window": 0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "plan", "attention", "attention", "attention"])
    dtype, fmt = rng.choice(["bf16", "f16"]), rng.choice(["mxfp4_g32", "int4_g64"])
    dim = rng.choice([64, 128])
    k_heads = rng.choice([1, 2, 4, 5, 8, 10, 20, 24])
    group = rng.choice([1, 2, 4, 5, 8]) if k_heads <= 8 else 1
    if op in ("norm_rope", "norm_rope_grad"):
        top = 4608 * 48 // (k_heads * (group + 1))
        return {"op": op, "tokens": _log(rng, 1, min(8192, top)), "q_heads": k_heads * group, "k_heads": k_heads,
                "dim": rng.choice([64, 80, 96, 128]), "dtype": dtype, "halves": rng.random() < 0.5, "norm": rng.random() < 0.8}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, min(8192, 4608 * 24 // k_heads)), "heads": k_heads, "dim": dim,
                "dtype": dtype, "fmt": fmt, "page": rng.choice([16, 32, 64, 128])}
    if op == "plan":
        requests = _log(rng, 1, 1024)
        return {"op": op, "requests": requests, "fresh": _log(rng, 1, min(4096, 65536 // requests)),
                "past": _log(rng, 1, 16384), "page": rng.choice([16, 32, 64, 128])}
    kind = rng.choice(["single", "few", "chunk"])
    if kind == "chunk":
        requests, fresh = rng.choice([1, 2, 3, 4]), _log(rng, 65, 2048)
        length = fresh + _log(rng, 1, 6144)
    else:
        requests, fresh = _log(rng, 1, 48), 1 if kind == "single" else rng.randint(2, 9)
        length = fresh + _log(rng, 1, 16384 - fresh)
    return {"op": op, "requests": requests, "fresh": fresh, "length": length, "q_heads": k_heads * group,
            "k_heads": k_heads, "dim": dim, "dtype": dtype, "fmt": fmt, "page": rng.choice([16, 32, 64, 128]),
            "causal": rng.random() < 0.8, "window": rng.choice([0, 0, 0, max(1, length // 3)])}


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each request: full length for the first, spread out for the rest."""
    b = np.arange(case["requests"])
    spread = (b * 0.6180339887498949 + 0.37) % 1.0
    fresh = np.maximum(1, np.round(case["fresh"] * (0.25 + 0.75 * spread))).astype(np.int64)
    fresh[0] = case["fresh"]
    if case["op"] == "plan":
        return fresh, np.round(case["past"] * spread).astype(np.int64) + fresh
    total = np.maximum(fresh, np.round(case["length"] * (0.25 + 0.75 * ((b * 0.7548776662466927 + 0.11) % 1.0)))).astype(np.int64)
    total[0] = case["length"]
    return fresh, total


def _pairs(case, fresh, total):
    """Pairs of a query and a key that it sees, and keys that are seen at all."""
    pairs = keys = 0
    for n, length in zip(fresh.tolist(), total.tolist()):
        pos = np.arange(length - n, length)
        last = pos if case["causal"] else np.full(n, length - 1)
        first = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros(n, np.int64)
        count = np.maximum(0, np.minimum(last, length - 1) - first + 1)
        pairs += int(count.sum())
        keys += int(last.max() - first.min() + 1)
    return pairs, keys


def work(case):
    op, d = case["op"], case.get("dim", 0)
    if op in ("norm_rope", "norm_rope_grad"):
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        table = case["tokens"] * d * 4
        if op == "norm_rope":
            return {"bytes": rows * d * 4 + table, "flops": rows * d * 7}
        return {"bytes": rows * d * 6 + table, "flops": rows * d * 18}
    if op == "append":
        n = case["tokens"] * case["heads"] * d * 2
        pool = -(-case["tokens"] // case["page"]) * case["page"] * case["heads"] * d * 2
        held = 0.5 + (1 if case["fmt"] == "mxfp4_g32" else 2) / GROUP[case["fmt"]]
        return {"bytes": n * (2 + held) + pool * (held + 2), "flops": n * 4 + pool}
    fresh, total = _lengths(case)
    if op == "plan":
        new_pages = int((-(-total // case["page"]) - -(-(total - fresh) // case["page"])).sum())
        return {"bytes": int(fresh.sum()) * 8 + case["requests"] * 16 + new_pages * 8, "flops": int(fresh.sum()) * 4}
    pairs, keys = _pairs(case, fresh, total)
    held = 0.5 + (1 if case["fmt"] == "mxfp4_g32" else 2) / GROUP[case["fmt"]]
    rows = int(fresh.sum()) * case["q_heads"]
    return {"bytes": keys * case["k_heads"] * d * 2 * held + rows * (d * 4 + 4), "flops": pairs * case["q_heads"] * d * 4}


# ------------------------------------------------------------------------------------------------------------ inputs
def _rows(g, dtype, *shape):
    """Activations: normal, with channels of different size and a few large ones."""
    size = torch.exp(0.4 * torch.randn(shape[-2:], generator=g, device="cuda"))
    size = size * torch.where(torch.rand(shape[-2:], generator=g, device="cuda") < 0.02, 6.0, 1.0)
    return (torch.randn(shape, generator=g, device="cuda") * size).to(dtype)


def _tables(count, dim):
    """cos and sin of the rotation for `count` positions, fp32 [count, dim / 2]."""
    freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    angle = torch.arange(count, device="cuda", dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _quantize(x, fmt):
    """Codes (one per element, uint8) and scales of x [..., D] in 32 bits."""
    g = x.float().reshape(*x.shape[:-1], -1, GROUP[fmt])
    top = g.abs().amax(-1)
    if fmt == "int4_g64":
        scale = torch.clamp(top / 7.0, max=65504.0).half()
        s = scale.float()[..., None]
        q = torch.where(s == 0, torch.zeros_like(g), torch.clamp(torch.round(g / torch.where(s == 0, torch.ones_like(s), s)), -7, 7))
        code = q.abs().to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    else:
        bits = (top / 6.0).view(torch.int32)
        e = torch.clamp(((bits >> 23) & 255) + ((bits & 0x7FFFFF) != 0), max=254)
        a = torch.ldexp(g, 127 - e[..., None]).abs()
        index = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
        code = index | (torch.signbit(g).to(torch.uint8) << 3)
        scale = e.to(torch.uint8)
    return code.reshape(x.shape), scale


def _values(codes, scales, fmt):
    """fp32 values [..., D] of packed codes [..., D / 2] and scales [..., D / group]."""
    n = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    mag = (n & 7).float()
    if fmt == "mxfp4_g32":
        table = torch.tensor(E2M1, device=codes.device)
        mag = table[(n & 7).int()]
        step = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        step = scales.float()
    v = torch.where(n >= 8, -mag, mag).reshape(*n.shape[:-1], -1, GROUP[fmt]) * step[..., None]
    return v.reshape(n.shape)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    op, dt = case["op"], DTYPES.get(case.get("dtype"))
    s = {"case": case}
    if op in ("norm_rope", "norm_rope_grad"):
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        qkv = _rows(g, dt, t, hq + 2 * hk, d)
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk]}
        s["cos"], s["sin"] = _tables(t + 5, d)
        s["positions"] = torch.randperm(t + 5, generator=g, device="cuda")[:t].int()
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2))
        if op == "norm_rope_grad":
            s["gq"] = torch.randn((t, hq, d), generator=g, device="cuda").to(dt)
            s["gk"] = torch.randn((t, hk, d), generator=g, device="cuda").to(dt)
        return s
    if op == "append":
        t, h, d, page, fmt = case["tokens"], case["heads"], case["dim"], case["page"], case["fmt"]
        kv = _rows(g, dt, t, 2 * h, d)
        pages = -(-t // page)
        s |= {"k": kv[:, :h], "v": kv[:, h:], "slots": torch.randperm(pages * page, generator=g, device="cuda")[:t].int()}
        s["every"] = torch.arange(pages * page, device="cuda", dtype=torch.int32)
        s |= _cache(pages, page, h, d, fmt)
        if own:
            s["cache"] = _handle(s, fmt)
        return s
    fresh, total = _lengths(case)
    b, page = case["requests"], case["page"]
    need = -(-total // page)
    if op == "plan":
        before, width, pool = -(-(total - fresh) // page), int(need.max()) + 3, int(need.sum()) + 17
        order = torch.randperm(pool, generator=g, device="cuda").int()
        start = np.concatenate(([0], np.cumsum(before)))
        col = torch.arange(width, device="cuda")
        at = torch.from_numpy(start[:-1]).cuda()[:, None] + col
        held = col < torch.from_numpy(before).cuda()[:, None]
        s["table"] = torch.where(held, order[torch.clamp(at, max=pool - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
        s["past"] = torch.from_numpy((total - fresh).astype(np.int32)).cuda()
        s["fresh"] = torch.from_numpy(fresh.astype(np.int32)).cuda()
        free = order[int(start[-1]):].contiguous()
        s["free"], s["count"], s["tokens"] = free, torch.tensor([free.numel()], device="cuda", dtype=torch.int32), int(fresh.sum())
        return s
    hq, hk, d, fmt = case["q_heads"], case["k_heads"], case["dim"], case["fmt"]
    pool = int(need.sum()) + 3
    order = torch.randperm(pool, generator=g, device="cuda").int()
    width = int(need.max())
    start = torch.from_numpy(np.concatenate(([0], np.cumsum(need)[:-1]))).cuda()
    col = torch.arange(width, device="cuda")
    s["table"] = torch.where(col < torch.from_numpy(need).cuda()[:, None], order[torch.clamp(start[:, None] + col, max=pool - 1)], torch.full((b, width), -1, device="cuda", dtype=torch.int32)).contiguous()
    s |= _cache(pool, page, hk, d, fmt)
    size = torch.exp(0.3 * torch.randn((2, hk, 1, d), generator=g, device="cuda"))
    for i, name in enumerate("kv"):
        for at in range(0, pool, max(1, (1 << 26) // (hk * page * d))):
            part = slice(at, min(pool, at + max(1, (1 << 26) // (hk * page * d))))
            x = torch.randn((part.stop - part.start, hk, page, d), generator=g, device="cuda") * size[i]
            code, scale = _quantize(x.to(dt), fmt)
            s[name + "_codes"][part], s[name + "_scales"][part] = _pack(code), scale
    s["q"] = (1.5 * torch.randn((int(fresh.sum()), hq, d), generator=g, device="cuda")).to(dt)
    s["start"] = torch.from_numpy(np.concatenate(([0], np.cumsum(fresh))).astype(np.int32)).cuda()
    s["length"] = torch.from_numpy(total.astype(np.int32)).cuda()
    if own:
        from diffusion_smooth_group_amd import kv
        s["cache"] = _handle(s, fmt)
        s["ws"] = kv.attention_workspace(b, int(fresh.sum()), hq, s["cache"], case["fresh"], case["length"], "cuda")
    return s


def _cache(pages, page, heads, dim, fmt):
    scale = torch.uint8 if fmt == "mxfp4_g32" else torch.float16
    return {n: torch.zeros((pages, heads, page, w), device="cuda", dtype=t)
            for n, w, t in (("k_codes", dim // 2, torch.uint8), ("k_scales", dim // GROUP[fmt], scale),
                            ("v_codes", dim // 2, torch.uint8), ("v_scales", dim // GROUP[fmt], scale))}


def _handle(s, fmt):
    from diffusion_smooth_group_amd import kv
    return kv.KVCache.wrap(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], fmt)


# ---------------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)(s, case, case["op"])


def _run_own(s, case, op):
    from diffusion_smooth_group_amd import kv
    if op == "norm_rope":
        return kv.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["wq"], s["wk"], eps=EPS, norm=case["norm"],
                               halves=case["halves"], positions=s["positions"])
    if op == "norm_rope_grad":
        return kv.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["cos"], s["sin"], s["wq"], s["wk"], eps=EPS,
                                        norm=case["norm"], halves=case["halves"], positions=s["positions"])
    if op == "append":
        s["cache"].append(s["k"], s["v"], s["slots"])
        return s["cache"].read(s["every"], dtype=DTYPES[case["dtype"]])
    if op == "plan":
        p = kv.plan(s["past"], s["fresh"], s["table"], s["free"], s["count"], page_size=case["page"], tokens=s["tokens"])
        return p.block_table, p.q_start, p.kv_len, p.slots, p.positions, p.free_count, p.missing
    return kv.attention(s["q"], s["cache"], s["table"], s["start"], s["length"], max_q=case["fresh"],
                        max_kv=case["length"], causal=case["causal"], window=case["window"], ws=s["ws"], return_lse=True)


def _turn(x, c, n, halves):
    """Rotates the pairs of x [T, H, D] by the angles of cos c and sin n [T, D / 2]."""
    c, n = c[:, None], n[:, None]
    if halves:
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * n, a * n + b * c), -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), -1).reshape(x.shape)


def _run_plain(s, case, op):
    if op in ("norm_rope", "norm_rope_grad"):
        at = s["positions"].long()
        c, n = s["cos"][at], s["sin"][at]
        if op == "norm_rope":
            return _norm_turn(s["q"], s["wq"], c, n, case), _norm_turn(s["k"], s["wk"], c, n, case)
        dq, dwq = _norm_turn_grad(s["gq"], s["q"], s["wq"], c, n, case)
        dk, dwk = _norm_turn_grad(s["gk"], s["k"], s["wk"], c, n, case)
        return dq, dk, dwq, dwk
    if op == "append":
        fmt, dt = case["fmt"], DTYPES[case["dtype"]]
        page, at = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        (kc, ks), (vc, vs) = _quantize(s["k"], fmt), _quantize(s["v"], fmt)
        s["k_codes"][page, :, at], s["k_scales"][page, :, at] = _pack(kc), ks
        s["v_codes"][page, :, at], s["v_scales"][page, :, at] = _pack(vc), vs
        k, v = (_values(s[n + "_codes"], s[n + "_scales"], fmt).transpose(1, 2).reshape(-1, case["heads"], case["dim"]) for n in "kv")
        page, at = s["every"].long(), None
        return k[page].to(dt), v[page].to(dt)
    if op == "plan":
        return _plan_plain(s, case["page"])
    return _attention_plain(s, case)


def _norm_turn(x, w, c, n, case):
    y = x.float()
    if case["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(y, c, n, case["halves"]).to(x.dtype)


def _norm_turn_grad(grad, x, w, c, n, case):
    back, x32 = _turn(grad.float(), c, -n, case["halves"]), x.float()
    if not case["norm"]:
        return back.to(x.dtype), torch.zeros(x.shape[-1], device=x.device)
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    up, unit = back * w.float(), x32 * r
    return (r * (up - unit * (up * unit).mean(-1, keepdim=True))).to(x.dtype), (back * unit).sum((0, 1))


def _plan_plain(s, page):
    past, fresh, table = s["past"].long(), s["fresh"].long(), s["table"]
    before, after = (past + page - 1) // page, (past + fresh + page - 1) // page
    need, count = after - before, s["count"].long()
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)
    index = first[:, None] + col - before[:, None]
    new = (col >= before[:, None]) & (col < after[:, None])
    page_of = torch.where(index < count, s["free"][torch.clamp(count - 1 - index, 0, s["free"].numel() - 1)], torch.full_like(table, -1))
    table.copy_(torch.where(new, page_of, table))
    ends = fresh.cumsum(0)
    q_start = torch.cat((torch.zeros_like(ends[:1]), ends))
    t = torch.arange(s["tokens"], device=table.device)
    r = torch.searchsorted(ends, t, right=True)
    pos = past[r] + t - q_start[r]
    held = table[r, pos // page].long()
    slots = torch.where(held < 0, held, held * page + pos % page)
    taken, wanted = torch.minimum(need.sum(), count), need.sum()
    return (table, q_start.int(), (past + fresh).int(), slots.int(), pos.int(), (count - taken).int(),
            torch.clamp(wanted - count, min=0).int())


def _attention_plain(s, case):
    fmt, page, hq, hk, d = case["fmt"], case["page"], case["q_heads"], case["k_heads"], case["dim"]
    length, start, table = s["length"].long(), s["start"].long(), s["table"].long()
    b, m = table.shape[0], case["fresh"]
    pages = torch.clamp(table, min=0)
    k, v = (_values(s[n + "_codes"][pages], s[n + "_scales"][pages], fmt).transpose(1, 2).reshape(b, hk, -1, d) for n in "kv")
    keys = k.shape[2]
    fresh = start[1:] - start[:-1]
    i = torch.arange(m, device="cuda")
    rows = torch.clamp(start[:-1, None] + i, max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(b, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(b, hk, hq // hk, m, keys)
    at, pos = torch.arange(keys, device="cuda"), (length - fresh)[:, None] + i
    see = (at < length[:, None])[:, None].expand(b, m, keys)
    if case["causal"]:
        see = see & (at <= pos[..., None])
    if case["window"]:
        see = see & (at > pos[..., None] - case["window"])
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = torch.clamp(x.amax(-1, keepdim=True), min=-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1)
    o = torch.matmul(p.view(b, hk, -1, keys), v).view(b, hk, hq // hk, m, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), top[..., 0] + total.log())
    real = i < fresh[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)[real]
    return out.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b, m, hq)[real]


# ------------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm_rope", "norm_rope_grad"):
        at = s["positions"].long()
        z = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]
        if op == "norm_rope":
            return tuple(_exact_turn(_exact_norm(s[n].double(), s["w" + n].double(), case), z, case) for n in "qk")
        got = [_exact_grad(s["g" + n].double(), s[n].double(), s["w" + n].double(), z, case) for n in "qk"]
        return got[0][0], got[1][0], got[0][1], got[1][1]
    if op == "append":
        out = []
        for x in (s["k"], s["v"]):
            pool = torch.zeros((s["every"].numel(), case["heads"], case["dim"]), device="cuda", dtype=torch.float64)
            pool[s["slots"].long()] = _exact_held(x.double(), case["fmt"])
            out.append(pool)
        return tuple(out)
    if op == "plan":
        return None
    fresh, total = _lengths(case)
    pairs, _ = _pairs(case, fresh, total)
    if pairs * case["q_heads"] * case["dim"] * 4 > 2e13:
        return None
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    for r, (n, length) in enumerate(zip(fresh.tolist(), total.tolist())):
        row = int(s["start"][r])
        held = s["table"][r, :-(-length // case["page"])].long()
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        hidden = torch.zeros((n, length), device="cuda", dtype=torch.bool)
        if case["causal"]:
            hidden |= key > pos
        if case["window"]:
            hidden |= key <= pos - case["window"]
        for h in range(hk):
            k, v = (_exact_read(s[c + "_codes"][held, h], s[c + "_scales"][held, h], case["fmt"])[:length] for c in "kv")
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                x = (s["q"][row:row + n, j].double() @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                lse[row:row + n, j] = torch.logsumexp(x, -1)
                out[row:row + n, j] = torch.nan_to_num(torch.softmax(x, -1)) @ v
    return out, lse


def _exact_norm(x, w, case):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w if case["norm"] else x


def _exact_turn(x, z, case):
    pair = x.unflatten(-1, (2, -1)).transpose(-1, -2) if case["halves"] else x.unflatten(-1, (-1, 2))
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    return (y.transpose(-1, -2) if case["halves"] else y).flatten(-2)


def _exact_grad(grad, x, w, z, case):
    """By the Jacobian of x / rms(x): identity over the rms less the outer product of x over D rms^3."""
    back = _exact_turn(grad, z.conj(), case)
    if not case["norm"]:
        return back, torch.zeros(x.shape[-1], device="cuda", dtype=torch.float64)
    rms = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    t = back * w
    dx = t / rms - x * (x * t).sum(-1, keepdim=True) / (x.shape[-1] * rms ** 3)
    return dx, (back * x / rms).flatten(0, 1).sum(0)


def _exact_held(x, fmt):
    """What the cache holds of x: the format's rule in 64 bits, the nearest code by search."""
    g = x.unflatten(-1, (-1, GROUP[fmt]))
    top = g.abs().amax(-1, keepdim=True)
    if fmt == "int4_g64":
        step = torch.clamp(top / 7, max=65504.0).half().double()
        code = torch.clamp(torch.round(g / torch.where(step > 0, step, torch.ones_like(step))), -7, 7)
        return (code * step).flatten(-2)
    step = torch.where(top > 0, 2.0 ** torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 6)), torch.zeros_like(top))
    u = (g / torch.where(step > 0, step, torch.ones_like(step)))
    best = torch.zeros_like(u)
    near = torch.full_like(u, math.inf)
    for index in (1, 3, 5, 7, 0, 2, 4, 6):   # even codes last, so that they win ties
        off = (u.abs() - E2M1[index]).abs()
        best = torch.where(off <= near, torch.full_like(u, E2M1[index]), best)
        near = torch.minimum(off, near)
    return (best * torch.sign(u) * step).flatten(-2)


def _exact_read(codes, scales, fmt):
    """fp64 rows [tokens, D] of one head's pages."""
    low, high = codes % 16, torch.div(codes, 16, rounding_mode="floor")
    n = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), device="cuda", dtype=torch.long)
    n[..., 0::2], n[..., 1::2] = low.long(), high.long()
    table = torch.tensor(E2M1 if fmt == "mxfp4_g32" else range(8), device="cuda", dtype=torch.float64)
    table = torch.cat((table, -table))
    step = 2.0 ** (scales.double() - 127) if fmt == "mxfp4_g32" else scales.double()
    return (table[n] * step.repeat_interleave(GROUP[fmt], -1)).flatten(0, 1)
