"""CPU test of the attention's workspace through the C ABI: the size for a
server's largest batch is enough while its requests end."""
import ctypes as C

from tests.test_kv_host import OK, attn, cache, fn


def size(requests, max_q, max_kv, tokens=None):
    n = C.c_size_t()
    d = attn(requests=requests, tokens=requests * max_q if tokens is None else tokens, q_heads=32, max_q=max_q, max_kv=max_kv)
    assert fn("svdq_kv_attention_workspace")(d, cache(heads=8), n) == OK
    return n.value


def test_the_size_does_not_shrink_with_the_bounds():
    for max_kv in (100, 1024, 5000, 16384, 200000):
        for max_q in (1, 4, 64, 2048):
            sizes = [size(r, max_q, max_kv) for r in (1, 2, 4, 32, 64, 128, 200, 256, 300)]
            assert sizes == sorted(sizes)
        sizes = [size(4, q, max_kv) for q in (1, 2, 5, 20, 64, 100, 300, 2048)]
        assert sizes == sorted(sizes)
    sizes = [size(64, 1, n) for n in (1, 900, 1024, 1100, 2000, 5000, 16384, 1 << 20, (1 << 31) - 1)]
    assert sizes == sorted(sizes)
    assert size(256, 1, 16384) >= size(64, 1, 16384) > 0 and size(4, 2048, 16384) >= size(4, 64, 16384) > 0
