"""Serves one attention layer over a paged 4-bit cache: prompts of different
lengths, then single tokens, then a request that ends and gives its pages back.

    python examples/serve_attention.py [--requests 8] [--steps 16]

Random weights; prints the time of a step and how far the last step's output is
from the same rows computed as one long prompt (both read the same 4-bit cache,
so they differ by 16-bit rounding only).
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from diffusion_smooth_group_amd import kv  # noqa: E402
from diffusion_smooth_group_amd import svdq as S  # noqa: E402
from diffusion_smooth_group_amd.attention_layer import SVDQAttention  # noqa: E402


def linear(rng, k, n, fmt):
    w = torch.from_numpy(rng.standard_normal((k, n)).astype(np.float32) / np.sqrt(k)).bfloat16()
    return S.SVDQLinear.pack(w.view(torch.int16).numpy().view(np.uint16), S.BF16, None, 16, fmt)


def layer(seed, width, q_heads, k_heads, dim, pages, page, fmt, positions):
    rng = np.random.default_rng(seed)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    cache = kv.KVCache(pages, page, k_heads, dim, fmt)
    w = [torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).bfloat16().cuda() for _ in range(2)]
    return SVDQAttention(linear(rng, width, (q_heads + 2 * k_heads) * dim, fmt), linear(rng, q_heads * dim, width, fmt), q_heads, cache,
                         angle.cos().float().cuda(), angle.sin().float().cuda(), *w, halves=True)


class Pool:
    """The pages of a cache and the requests that hold them."""

    def __init__(self, requests, pages, page, width):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page = page
        self.free, self.count = torch.arange(pages, **i32), torch.tensor([pages], **i32)
        self.table, self.length = torch.full((requests, width), -1, **i32), torch.zeros(requests, **i32)

    def step(self, fresh):
        new = torch.tensor(fresh, dtype=torch.int32, device="cuda")
        p = kv.plan(self.length, new, self.table, self.free, self.count, self.page, int(sum(fresh)))
        self.length, self.count = p.kv_len, p.free_count
        return p

    def end(self, done):
        d = torch.tensor(done, dtype=torch.int32, device="cuda")
        self.length, self.count = self.length.clone(), self.count.clone()
        kv.release(d, self.table, self.length, self.free, self.count, self.page)


def serve(requests=8, steps=16, width=512, q_heads=8, k_heads=2, dim=64, page=16, fmt=S.FMT_MXFP4_G32, seed=0, report=print):
    prompts = [5 + 37 * (r % 5) for r in range(requests)]
    longest = max(prompts) + steps + 1
    pages = sum(-(-(n + steps + 1) // page) for n in prompts) + 4
    net = layer(seed, width, q_heads, k_heads, dim, pages, page, fmt, longest)
    pool = Pool(requests, pages, page, -(-longest // page))
    g = torch.Generator().manual_seed(seed + 1)
    x = [torch.randn((n + steps, width), generator=g).bfloat16().cuda() for n in prompts]
    net(torch.cat([v[:n] for v, n in zip(x, prompts)]), pool.step(prompts), max(prompts), longest)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for t in range(steps):
        y = net(torch.stack([v[n + t] for v, n in zip(x, prompts)]), pool.step([1] * requests), 1, longest)
    end.record()
    torch.cuda.synchronize()
    report(f"{requests} requests, {steps} single-token steps: {begin.elapsed_time(end) / steps * 1e3:.1f} us a step")
    # the same tokens as whole prompts, in the pages of an empty pool
    again = Pool(requests, pages, page, -(-longest // page))
    whole = net(torch.cat(x), again.step([n + steps for n in prompts]), longest, longest)
    last = whole[torch.tensor([n + steps for n in prompts]).cumsum(0) - 1]
    off = float((last.float() - y.float()).norm() / y.float().norm())
    left = int(pool.count)
    pool.end([1] + [0] * (requests - 1))
    back = int(pool.count) - left
    report(f"last step against whole prompts: {off:.2e}; request 0 gave {back} pages back")
    return off, back, -(-(prompts[0] + steps) // page)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    serve(a.requests, a.steps)
