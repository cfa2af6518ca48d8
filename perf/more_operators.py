"""Cases of the operators of an image model's conditioned blocks: what is measured, in plain torch and through the library.

Where an encoder's states (a text's, an image's, a sound's) enter a model whose linears are 4-bit, these run between the
linears:

    group_norm        group norm over a channels-last map with an activation (forward, and its gradient)
    cross_attention   softmax attention of one sequence's queries to an encoder's 16-bit keys and values of another length,
                      with grouped heads and key masks (prompts, images and single tokens; forward, and its gradient)

Rows of heads are [tokens, heads, D], or [requests, tokens, heads, D] where all requests have the same number; a map is
[samples, height, width, channels].
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------------------- cases
def _cross(name, op, requests, rows, keys, q_heads, k_heads, dim, dtype, ragged=False, mask="none"):
    c = {"op": op, "requests": requests, "rows": rows, "keys": keys, "q_heads": q_heads, "k_heads": k_heads, "dim": dim,
         "dtype": dtype, "ragged": ragged, "mask": mask}
    return {"name": name} | c if name else c


def _norm(name, op, samples, height, width, channels, groups, act, dtype):
    c = {"op": op, "samples": samples, "height": height, "width": width, "channels": channels, "groups": groups,
         "act": act, "dtype": dtype}
    return {"name": name} | c if name else c


def listed():
    return [
        # a decoder's step: one token of 8 requests each looks at an encoder's 1500 states; latency counts
        _cross("cross 8x1 of 1500 f16", "cross", 8, 1, 1500, 20, 20, 64, "f16"),
        # a decoder's step of many requests with grouped heads over long documents of different lengths: bytes count
        _cross("cross 64x1 of 4096 32/8 bf16", "cross", 64, 1, 4096, 32, 8, 128, "bf16", ragged=True),
        # an image layer with a text's 77 states, both halves of a guided step
        _cross("cross 2x4096 of 77 bf16", "cross", 2, 4096, 77, 10, 10, 64, "bf16"),
        # images of different sizes with a padded text of up to 300 states and heads of 72
        _cross("cross 3x2047 of 300 masked f16", "cross", 3, 2047, 300, 16, 16, 72, "f16", ragged=True, mask="tail"),
        # 4608 tokens that look at the 4096 states of a reference image: the products count
        _cross("cross 1x4608 of 4096 bf16", "cross", 1, 4608, 4096, 24, 24, 128, "bf16"),
        # training of the image layer with a text's 77 states: the shared keys' gradients are sums over 4096 rows
        _cross("cross_grad 2x4096 of 77 bf16", "cross_grad", 2, 4096, 77, 10, 10, 64, "bf16"),
        # training of the 24-head layer with 512 states
        _cross("cross_grad 1x4608 of 512 f16", "cross_grad", 1, 4608, 512, 24, 24, 128, "f16"),
        # training with grouped heads, odd lengths and masked states
        _cross("cross_grad 5x1023 of 2049 masked bf16", "cross_grad", 5, 1023, 2049, 32, 8, 128, "bf16", ragged=True,
               mask="random"),
        # the deepest map of one image: latency counts
        _norm("group_norm 1x8x8x1280 f16", "norm", 1, 8, 8, 1280, 32, "silu", "f16"),
        # a map of a decoder to pixels: larger than the chip's caches hold
        _norm("group_norm 1x512x512x128 bf16", "norm", 1, 512, 512, 128, 32, "silu", "bf16"),
        # training of the largest latent map, both halves of a guided step
        _norm("group_norm_grad 2x128x128x320 bf16", "norm_grad", 2, 128, 128, 320, 32, "silu", "bf16"),
        # training with odd sides and no activation, as in front of an attention
        _norm("group_norm_grad 3x33x31x960 f16", "norm_grad", 3, 33, 31, 960, 32, "none", "f16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm_grad"):
        groups = rng.choice([1, 4, 8, 16, 32, 32, 32])
        channels = groups * rng.choice([8, 16, 24]) if groups < 32 else 32 * rng.choice([1, 2, 4, 5, 8, 10, 15, 20, 30, 40, 60, 80])
        samples = _log(rng, 1, 16)
        side = math.sqrt((1 << 25 if op == "norm" else 1 << 24) / (samples * channels))
        height = _log(rng, 1, max(1, min(512, side)))
        width = _log(rng, 1, max(1, min(512, side)))
        return _norm("", op, samples, height, width, channels, groups, rng.choice(["none", "silu", "silu", "gelu"]), dtype)
    k_heads = rng.choice([1, 2, 4, 5, 8, 10, 16, 20, 24])
    group = rng.choice([1, 2, 4, 5, 8]) if k_heads <= 8 else 1
    dim = rng.choice([40, 64, 72, 80, 96, 128])
    requests = _log(rng, 1, 32)
    top = 4608 * 4096 * 24 // (requests * k_heads * group)
    if op == "cross_grad":
        top //= 4
    keys = _log(rng, 1, max(1, min(8192, top)))
    rows = 1 if op == "cross" and rng.random() < 0.3 else _log(rng, 1, max(1, min(8192, top // keys, (1 << 24) // (requests * k_heads * group))))
    return _cross("", op, requests, rows, keys, k_heads * group, k_heads, dim, dtype, rng.random() < 0.5,
                  rng.choice(["none", "none", "tail", "random"]))


def _lengths(case):
    """Rows and encoder states of each request: full length for the first, spread out for the rest where they are ragged."""
    b, n = np.arange(case["requests"]), case["requests"]
    if not case["ragged"]:
        return np.full(n, case["rows"], np.int64), np.full(n, case["keys"], np.int64)
    rows = np.round(case["rows"] * (0.25 + 0.75 * ((b * 0.6180339887498949 + 0.37) % 1.0))).astype(np.int64)
    keys = np.round(case["keys"] * (0.25 + 0.75 * ((b * 0.7548776662466927 + 0.11) % 1.0))).astype(np.int64)
    rows, keys = np.maximum(rows, 1), np.maximum(keys, 1)
    rows[0], keys[0] = case["rows"], case["keys"]
    return rows, keys


def _mask(case, keys):
    """Which states are seen, one truth value for each, the same for every seed: None, a text's length, or scattered ones."""
    if case["mask"] == "none":
        return None
    kept = []
    for r, n in enumerate(keys.tolist()):
        at = np.arange(n)
        if case["mask"] == "tail":              # a text of any length from none to all (the first of all)
            kept.append(at < (n if r == 0 else round(n * ((r * 0.5698402909980532) % 1.0))))
        else:                                   # about three quarters, in no order
            kept.append((at * 0.6180339887498949 + r * 0.37) % 1.0 < 0.75)
    return np.concatenate(kept)


def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n = case["samples"] * case["height"] * case["width"] * case["channels"]
        c = case["channels"]
        if case["op"] == "norm":
            return {"bytes": 4 * n + 4 * c, "flops": 8 * n}
        return {"bytes": 6 * n + 12 * c + 8 * case["samples"] * case["groups"], "flops": 20 * n}
    rows, keys = _lengths(case)
    mask, hq, hk, d = _mask(case, keys), case["q_heads"], case["k_heads"], case["dim"]
    ends = np.cumsum(keys)
    seen = keys if mask is None else np.array([int(mask[e - n:e].sum()) for e, n in zip(ends, keys)])
    pairs = int((rows * seen).sum())
    q, k = int(rows.sum()) * hq * d * 2, int(seen.sum()) * hk * d * 2
    every = int(keys.sum()) * hk * d * 2
    if case["op"] == "cross":
        return {"bytes": 2 * q + 2 * k, "flops": 4 * pairs * hq * d}
    # q, the output, its gradient and the sums of exponentials are read, three gradients written
    return {"bytes": 4 * q + 2 * k + 2 * every + int(rows.sum()) * hq * 4, "flops": 10 * pairs * hq * d}


# ------------------------------------------------------------------------------------------------------------ inputs
def _randn(g, dtype, *shape, size=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * size).to(dtype)


def _heads(g, dtype, tokens, heads, dim, size):
    """Rows of heads, a part of a wider projection's rows: channels of different size and a mean of their own."""
    scale = torch.exp(0.3 * torch.randn((heads, dim), generator=g, device="cuda"))
    mean = 0.2 * torch.randn((heads, dim), generator=g, device="cuda")
    return ((torch.randn((tokens, heads, dim), generator=g, device="cuda") + mean) * scale * size).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        n, h, w, c = case["samples"], case["height"], case["width"], case["channels"]
        mean, scale = torch.randn(c, generator=g, device="cuda"), torch.exp(0.5 * torch.randn(c, generator=g, device="cuda"))
        s["x"] = (torch.randn((n, h, w, c), generator=g, device="cuda").mul_(scale).add_(mean)).to(dt)
        s["weight"] = (1 + 0.2 * torch.randn(c, generator=g, device="cuda")).to(dt)
        s["bias"] = (0.2 * torch.randn(c, generator=g, device="cuda")).to(dt)
        if case["op"] == "norm_grad":           # the forward pass leaves each group's mean and inverse deviation
            s["grad"] = _randn(g, dt, n, h, w, c)
            x = s["x"].double().view(n, h * w, case["groups"], -1)
            var, mu = torch.var_mean(x, dim=(1, 3), unbiased=False)
            s["stats"] = torch.stack((mu, torch.rsqrt(var + EPS)), -1).float()
        return s
    rows, keys = _lengths(case)
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    tokens, states = int(rows.sum()), int(keys.sum())
    s["q"] = _heads(g, dt, tokens, hq, d, 1.2)
    kv = _heads(g, dt, states, 2 * hk, d, 1.0)              # one projection gives an encoder's keys and values
    s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
    mask = _mask(case, keys)
    s["mask"] = None if mask is None else torch.from_numpy(mask).cuda()
    s["start"] = [torch.from_numpy(np.concatenate(([0], np.cumsum(n))).astype(np.int32)).cuda() for n in (rows, keys)]
    s["lengths"] = rows.tolist(), keys.tolist()
    if case["op"] == "cross_grad":              # the forward pass leaves its output and the sums of exponentials
        s["grad"] = _randn(g, dt, tokens, hq, d, size=0.5)
        out, lse = _cross_plain(s, case)
        s["out"], s["lse"] = out.to(dt), lse
    if not case["ragged"]:                      # requests of one length: [requests, tokens, heads, D]
        b = case["requests"]
        for n in ("q", "k", "v", "grad", "out", "lse", "mask"):
            if s.get(n) is not None:
                s[n] = s[n].unflatten(0, (b, -1))
    return s


# ---------------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "norm":
        return _norm_plain(s, case)
    if case["op"] == "norm_grad":
        return _norm_grad_plain(s, case)
    flat = s if case["ragged"] else s | {n: s[n].flatten(0, 1) for n in ("q", "k", "v", "grad", "mask") if s.get(n) is not None}
    if case["op"] == "cross":
        return _cross_plain(flat, case)[0].to(s["q"].dtype).view(s["q"].shape)
    return tuple(t.to(s["q"].dtype).view(s[n].shape) for n, t in zip("qkv", _cross_grad_plain(flat, case)))


def _run_own(s, case):
    from diffusion_smooth_group_amd import image
    if case["op"] == "norm":
        return image.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=EPS, act=None if case["act"] == "none" else case["act"])
    if case["op"] == "norm_grad":
        return image.group_norm_backward(s["grad"], s["x"], s["stats"], case["groups"], s["weight"], s["bias"],
                                         act=None if case["act"] == "none" else case["act"])
    where = {"mask": s["mask"]}
    if case["ragged"]:
        where |= {"q_start": s["start"][0], "k_start": s["start"][1], "max_q": case["rows"], "max_k": case["keys"]}
    if case["op"] == "cross":
        return image.cross_attention(s["q"], s["k"], s["v"], **where)
    return image.cross_attention_backward(s["grad"], s["q"], s["k"], s["v"], s["out"], s["lse"], **where)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _norm_plain(s, case):
    x = s["x"].float().flatten(1, 2).unflatten(2, (case["groups"], -1))
    y = x - x.mean((1, 3), keepdim=True)
    y = (y * torch.rsqrt(y.square().mean((1, 3), keepdim=True) + EPS)).flatten(2)
    return _act(y * s["weight"].float() + s["bias"].float(), case["act"]).to(s["x"].dtype).view(s["x"].shape)


def _norm_grad_plain(s, case):
    cut = (case["groups"], -1)
    x = s["x"].float().flatten(1, 2).unflatten(2, cut)
    mean, inv = s["stats"][:, None, :, :1], s["stats"][:, None, :, 1:]
    unit = (x - mean) * inv
    w = s["weight"].float()
    g = s["grad"].float().flatten(1, 2) * _act_slope(unit.flatten(2) * w + s["bias"].float(), case["act"])
    dw, db = (g * unit.flatten(2)).sum((0, 1)), g.sum((0, 1))
    u = (g * w).unflatten(2, cut)
    dx = inv * (u - u.mean((1, 3), keepdim=True) - unit * (u * unit).mean((1, 3), keepdim=True))
    return dx.to(s["x"].dtype).view(s["x"].shape), dw, db


def _padded(s, case):
    """Queries [B, Hk, G M, D], keys and values [B, Hk, N, D] in fp32, which keys are seen, and the rows' places."""
    b, hk, gr = case["requests"], case["k_heads"], case["q_heads"] // case["k_heads"]
    at = []
    for start, most in zip(s["start"], (case["rows"], case["keys"])):
        i = torch.arange(most, device="cuda")
        start = start.long()
        at.append((start[:-1, None] + i, i < (start[1:] - start[:-1])[:, None]))
    (qi, qok), (ki, kok) = at
    qi, ki = torch.where(qok, qi, 0), torch.where(kok, ki, 0)
    see = kok if s["mask"] is None else kok & s["mask"].view(-1)[ki]
    k, v = (torch.where(see[..., None, None], s[n][ki].float(), 0).transpose(1, 2).contiguous() for n in "kv")
    return _grouped(s["q"][qi], hk, gr), k, v, see[:, None, None], qi, qok, ki, kok


def _grouped(t, hk, gr):
    """[B, M, Hk G, D] as fp32 [B, Hk, G M, D]."""
    return t.float().unflatten(2, (hk, gr)).permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()


def _rows(t, ok):
    """[B, Hk, G M, ...] as [tokens, heads, ...], the requests' own rows only."""
    return t.unflatten(2, (-1, ok.shape[1])).movedim(3, 1).flatten(2, 3)[ok]


def _cross_plain(s, case):
    q, k, v, see, _, qok, _, _ = _padded(s, case)
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(1 / math.sqrt(case["dim"]))
    x.masked_fill_(~see, -math.inf)
    top = torch.clamp(x.amax(-1, keepdim=True), min=-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return _rows(out, qok), _rows((top + total.log())[..., 0], qok)


def _cross_grad_plain(s, case):
    q, k, v, see, qi, qok, ki, kok = _padded(s, case)
    hk, gr, scale = case["k_heads"], case["q_heads"] // case["k_heads"], 1 / math.sqrt(case["dim"])
    g = _grouped(torch.where(qok[..., None, None], s["grad"][qi], 0), hk, gr)
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale).masked_fill_(~see, -math.inf)
    p = x.sub_(torch.clamp(x.amax(-1, keepdim=True), min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), g)
    dp = torch.matmul(g, v.transpose(-1, -2).contiguous())
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
    return _rows(dq, qok), dk.transpose(1, 2)[kok], dv.transpose(1, 2)[kok]


# ------------------------------------------------------------------------------------------------- results in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _norm_exact(s, case)
    pieces = {"q": [], "k": [], "v": []}
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    rows, keys = s["lengths"]
    flat = {n: s[n] if case["ragged"] or s.get(n) is None else s[n].flatten(0, 1) for n in ("q", "k", "v", "grad", "mask") if n in s}
    r0 = k0 = 0
    for m, n in zip(rows, keys):
        kept = torch.arange(k0, k0 + n, device="cuda")
        if flat["mask"] is not None:
            kept = kept[flat["mask"][k0:k0 + n]]
        out = {"q": torch.zeros((m, hq, d), device="cuda", dtype=torch.float64),
               "k": torch.zeros((n, hk, d), device="cuda", dtype=torch.float64),
               "v": torch.zeros((n, hk, d), device="cuda", dtype=torch.float64)}
        for h in range(hq if kept.numel() else 0):
            c = h // (hq // hk)
            q, k, v = flat["q"][r0:r0 + m, h].double(), flat["k"][kept, c].double(), flat["v"][kept, c].double()
            w = torch.softmax(q @ k.T / math.sqrt(d), -1)
            if case["op"] == "cross":
                out["q"][:, h] = w @ v
                continue
            g = flat["grad"][r0:r0 + m, h].double()
            out["v"][kept - k0, c] += w.T @ g
            slope = g @ v.T
            slope = w * (slope - (w * slope).sum(-1, keepdim=True)) / math.sqrt(d)
            out["q"][:, h] = slope @ k
            out["k"][kept - k0, c] += slope.T @ q
        for name in pieces:
            pieces[name].append(out[name])
        r0, k0 = r0 + m, k0 + n
    whole = [torch.cat(pieces[n]).view(s[n].shape) for n in "qkv"]
    return whole[0] if case["op"] == "cross" else tuple(whole)


def _norm_exact(s, case):
    n, c, per = case["samples"], case["channels"], case["channels"] // case["groups"]
    x = s["x"].double().reshape(n, -1, c)
    w, b = s["weight"].double(), s["bias"].double()
    results = []
    dw, db = torch.zeros(c, device="cuda", dtype=torch.float64), torch.zeros(c, device="cuda", dtype=torch.float64)
    for i in range(case["groups"]):
        part = slice(i * per, (i + 1) * per)
        y, wi, bi = x[..., part], w[part], b[part]
        if case["op"] == "norm":
            var, mean = torch.var_mean(y, dim=(1, 2), unbiased=False, keepdim=True)
            z = (y - mean) / torch.sqrt(var + EPS) * wi + bi
            results.append({"silu": z * torch.sigmoid(z), "gelu": z * torch.special.ndtr(z), "none": z}[case["act"]])
            continue
        mean, inv = (s["stats"][:, i, j].double()[:, None, None] for j in (0, 1))
        unit = (y - mean) * inv
        z = unit * wi + bi
        p = torch.sigmoid(z)
        slope = {"silu": p + z * p * (1 - p), "none": torch.ones_like(z),
                 "gelu": torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[case["act"]]
        g = s["grad"].double().reshape(n, -1, c)[..., part] * slope
        dw[part], db[part] = (g * unit).sum((0, 1)), g.sum((0, 1))
        u = g * wi
        results.append(inv * (u - u.mean((1, 2), keepdim=True) - unit * (u * unit).mean((1, 2), keepdim=True)))
    y = torch.cat(results, -1).view(s["x"].shape)
    return y if case["op"] == "norm" else (y, dw, db)
