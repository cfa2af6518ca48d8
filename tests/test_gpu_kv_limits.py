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
