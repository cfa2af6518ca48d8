"""GPU tests of the attention layer: captured calls, padded steps, masks."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _layer(fmt, pages=700, positions=6000, **kw):
    import serve_attention
    return serve_attention.layer(3, 256, 4, 2, 64, pages, 16, fmt, positions, **kw)


def _step(torch, kv, past, fresh, tokens=None, width=400, pages=700):
    i32 = dict(dtype=torch.int32, device="cuda")
    b = len(past)
    table, at = torch.full((b, width), -1, dtype=torch.int32), 0
    for r, n in enumerate(past):
        used = -(-n // 16)
        table[r, :used] = torch.arange(at, at + used)
        at += used
    free = torch.arange(pages - 1, at - 1, -1, **i32)
    return kv.plan(torch.tensor(past, **i32), torch.tensor(fresh, **i32), table.cuda(), free, torch.tensor([free.numel()], **i32), 16,
                   sum(fresh) if tokens is None else tokens)


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_captured_call_outlives_larger_ones(fmt):
    """A graph of a small step (with chunks that are joined) after calls that
    need more workspace: it writes to nobody else's memory and gives the eager
    result at every replay."""
    import torch

    from diffusion_smooth_group_amd import kv
    net = _layer(fmt)
    x = torch.randn((2, 256), device="cuda").bfloat16()
    big = torch.randn((900, 256), device="cuda").bfloat16()
    # fill the cache that the small step reads: 4000 and 1500 tokens
    net(torch.randn((5500, 256), device="cuda").bfloat16(), _step(torch, kv, [0, 0], [4000, 1500]), 4000, 4000)
    small, large = _step(torch, kv, [4000, 1500], [1, 1]), _step(torch, kv, [5600], [900], width=700)
    large = large._replace(slots=torch.full_like(large.slots, -1))          # nothing is written to the cache
    assert kv.attention_workspace_size(2, 2, 4, net.cache, 1, 4001) > 0
    want = net(x, small, 1, 4001)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = net(x, small, 1, 4001)
    for again in range(4):
        net(big, large, 900, 6500)                         # more of every workspace
        held = [torch.full((1 << s,), 0x5A, dtype=torch.uint8, device="cuda") for s in range(9, 24) for _ in range(4)]
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 0x5A).all()) for t in held)
        assert torch.equal(out, want) and torch.equal(net(x, small, 1, 4001), want)


def test_calls_on_two_streams_share_no_workspace(monkeypatch):
    import torch

    from diffusion_smooth_group_amd import kv
    from diffusion_smooth_group_amd import svdq as S
    net = _layer(1)
    net(torch.randn((4000, 256), device="cuda").bfloat16(), _step(torch, kv, [0], [4000]), 4000, 4000)
    step, x = _step(torch, kv, [4000], [1]), torch.randn((1, 256), device="cuda").bfloat16()
    used = []
    attention, linear = kv._call, S._call
    monkeypatch.setattr(kv, "_call", lambda name, *a: (used.append(a[5]) if name == "svdq_kv_attention" else None, attention(name, *a)))
    monkeypatch.setattr(S, "_call", lambda name, *a: (used.append(a[6].value) if name == "svdq_linear_forward" else None, linear(name, *a)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = net(x, step, 1, 4001)
    here, used[:] = list(used), []
    with torch.cuda.stream(side):
        second = net(x, step, 1, 4001)
    torch.cuda.synchronize()
    assert len(here) == len(used) == 3 and not set(here) & set(used)
    assert torch.equal(first, second)


def test_rows_of_no_request_are_the_projection_of_zeros():
    """A step padded to a fixed number of tokens, in memory that held NaN."""
    import torch

    from diffusion_smooth_group_amd import kv
    net = _layer(1)
    x = torch.randn((70, 256), device="cuda").bfloat16()
    padded = torch.cat((x, torch.zeros((58, 256), device="cuda").bfloat16()))
    want = net(x, _step(torch, kv, [0, 0], [40, 30]), 40, 40)
    zeros = net.out.forward(torch.zeros((58, net.out.K), device="cuda").bfloat16())
    for _ in range(3):
        held = [torch.full((128 * n,), float("nan"), device="cuda").bfloat16() for n in (64, 128, 256, 512, 1024)]
        del held
        got = net(padded, _step(torch, kv, [0, 0], [40, 30], tokens=128), 40, 40)
        assert torch.equal(got[:70], want) and torch.equal(got[70:], zeros)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 7), (False, 7)])
def test_masks_of_the_layer_are_those_of_the_attention(causal, window):
    """The layer against its operators, called one after the other."""
    import torch

    from diffusion_smooth_group_amd import kv
    from diffusion_smooth_group_amd.attention_layer import SVDQAttention
    net = _layer(1)
    net = SVDQAttention(net.qkv, net.out, 4, net.cache, net.how["cos"], net.how["sin"], net.how["wq"], net.how["wk"], halves=True,
                        window=window, causal=causal)
    x = torch.randn((100, 256), device="cuda").bfloat16()
    step = _step(torch, kv, [0, 0], [60, 40])
    got = net(x, step, 60, 60)
    rows = net.qkv.forward(x).view(100, 8, 64)
    q = net.cache.append(rows[:, 4:6], rows[:, 6:], step.slots, q=rows[:, :4], positions=step.positions, **net.how)
    o = kv.attention(q, net.cache, step.block_table, step.q_start, step.kv_len, 60, 60, causal=causal, window=window)
    assert torch.equal(got, net.out.forward(o.contiguous().view(100, 256)))
