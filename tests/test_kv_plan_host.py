"""CPU test of the step tables' C ABI: outputs that overlap inputs are refused
before anything is launched (workgroups read what another would write)."""
import ctypes as C

import pytest

from tests.test_kv_host import INVALID, fn

NAMES = ("past", "fresh", "requests", "page_size", "tokens", "free_pages", "free_count", "free_capacity", "block_table", "table_stride",
         "q_start", "kv_len", "slots", "positions", "free_left", "missing", "stream")
IN = {"past": 40, "fresh": 40, "free_pages": 100, "free_count": 1}
OUT = {"block_table": 400, "q_start": 41, "kv_len": 40, "slots": 3000, "positions": 3000, "free_left": 1, "missing": 1}


def call(**change):
    at = {n: 1 << 20 | i << 16 for i, n in enumerate(NAMES)}       # buffers of their own, never dereferenced
    at |= dict(requests=40, page_size=16, tokens=3000, free_capacity=100, table_stride=10, stream=None)
    at |= change
    return fn("svdq_kv_plan")(*[C.c_void_p(at[n]) if n in IN or n in OUT else at[n] for n in NAMES])


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("into", list(IN))
def test_an_output_over_an_input_is_refused(out, into):
    base = 1 << 24
    assert call(**{into: base, out: base}) == INVALID
    assert call(**{into: base, out: base + 4 * (IN[into] - 1)}) == INVALID       # its last entry
    assert call(**{into: base + 4 * (OUT[out] - 1), out: base}) == INVALID
