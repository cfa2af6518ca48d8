"""CPU tests of the cache operators' C ABI: exported symbols, sizes and the
refusal of every wrong argument before anything is launched."""
import ctypes as C
import os
import re

import pytest

from diffusion_smooth_group_amd import kv
from diffusion_smooth_group_amd import svdq as S

HDR = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "svdq_kv.h")
OK, INVALID, SHAPE, UNSUPPORTED, CAPACITY = 0, 1, 2, 3, 4
P = C.c_void_p(4096)         # aligned, never dereferenced: every call here is refused first


def fn(name):
    f = getattr(S.lib_handle(), name)
    f.argtypes, f.restype = kv._SIGS[name], C.c_int
    return f


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"^svdq_status\s+(svdq_\w+)\s*\(", open(HDR).read(), re.M))
    assert names == set(kv._SIGS)
    for n in names:
        assert hasattr(S.lib_handle(), n)


@pytest.mark.parametrize("fmt,dim,code,scale", [(1, 128, 64, 4), (1, 64, 32, 2), (0, 128, 64, 4), (0, 64, 32, 2)])
def test_cache_size(fmt, dim, code, scale):
    c, s = C.c_size_t(), C.c_size_t()
    assert fn("svdq_kv_cache_size")(7, 32, 5, dim, fmt, c, s) == OK
    assert (c.value, s.value) == (7 * 32 * 5 * code, 7 * 32 * 5 * scale)


def test_cache_size_refusals():
    c, s = C.c_size_t(), C.c_size_t()
    f = fn("svdq_kv_cache_size")
    assert f(7, 32, 5, 128, 1, None, s) == INVALID
    assert f(-1, 32, 5, 128, 1, c, s) == INVALID
    assert f(7, 32, 0, 128, 1, c, s) == INVALID
    assert f(7, 32, 5, 128, 9, c, s) == INVALID
    assert f(7, 32, 5, 128, S.FMT_INT8_W8A8, c, s) == UNSUPPORTED
    for page in (0, 8, 24, 48, 512, -16):
        assert f(7, page, 5, 128, 1, c, s) == SHAPE
    for dim in (0, 32, 80, 96, 256):
        assert f(7, 32, 5, dim, 1, c, s) == SHAPE
    assert f(1 << 31, 16, 5, 128, 1, c, s) == UNSUPPORTED
    assert f(1 << 62, 256, 5, 128, 1, c, s) == UNSUPPORTED      # no product overflows on the way
    assert f((1 << 31) // 256, 256, 5, 128, 1, c, s) == UNSUPPORTED
    assert f((1 << 31) // 256 - 1, 256, 5, 128, 1, c, s) == OK


def heads(n=4, token=512, head=128, data=P):
    return kv.svdq_heads(data, token, head, n)


def qk(**kw):
    d = kv.svdq_qk_desc(10, 128, S.BF16, kv.QK_NORM | kv.QK_ROPE, 1e-6, P, P, P, P, 10, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def cache(**kw):
    c = kv.svdq_kv_cache(P, P, P, P, 8, 32, 4, 128, S.FMT_MXFP4_G32)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_DESC = [(dict(tokens=-1), INVALID), (dict(dtype=2), INVALID), (dict(flags=8), INVALID), (dict(head_dim=0), SHAPE),
            (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
            (dict(cos=None), INVALID), (dict(sin=None), INVALID), (dict(n_positions=-1), INVALID),
            (dict(flags=kv.QK_ROPE_HALVES), INVALID), (dict(cos=C.c_void_p(4100)), SHAPE), (dict(wq=C.c_void_p(4098)), SHAPE)]


@pytest.mark.parametrize("change,status", BAD_DESC)
def test_desc_refusals(change, status):
    h = heads()
    assert fn("svdq_qk_norm_rope")(qk(**change), h, h, h, h, None) == status
    assert fn("svdq_qk_norm_rope_backward")(qk(**change), h, h, h, h, h, h, P, P, P, 1 << 30, None) == status
    assert fn("svdq_kv_append")(qk(**change), h, h, h, h, cache(), P, None) == status


BAD_HEADS = [(dict(data=None), INVALID), (dict(data=C.c_void_p(4104)), SHAPE), (dict(token=516), SHAPE), (dict(head=132), SHAPE),
             (dict(head=120), SHAPE), (dict(token=-512), SHAPE), (dict(n=5), SHAPE)]


@pytest.mark.parametrize("change,status", BAD_HEADS)
def test_view_refusals(change, status):
    h, bad = heads(), heads(**change)
    for at in range(4):
        args = [h, h, h, h]
        args[at] = bad
        if change.get("n"):
            if at < 2:
                continue         # another number of heads is an error in the outputs
        assert fn("svdq_qk_norm_rope")(qk(), *args, None) == status, at
    for at in range(2, 6):
        args = [h] * 6
        args[at] = bad
        assert fn("svdq_qk_norm_rope_backward")(qk(), *args, P, P, P, 1 << 30, None) == status, at
    for at in (1, 2):
        args = [h] * 4
        args[at] = bad
        assert fn("svdq_kv_append")(qk(), *args, cache(), P, None) == status, at
    assert fn("svdq_kv_read")(cache(), P, 10, S.F16, bad, h, None) == status
    assert fn("svdq_kv_read")(cache(), P, 10, S.F16, h, bad, None) == status


def test_norm_rope_empty_calls_and_row_limit():
    h = heads()
    assert fn("svdq_qk_norm_rope")(qk(tokens=0), h, h, h, h, None) == OK
    assert fn("svdq_kv_append")(qk(tokens=0), None, h, h, None, cache(), None, None) == OK
    assert fn("svdq_kv_read")(cache(), None, 0, S.F16, None, None, None) == OK
    assert fn("svdq_qk_norm_rope")(qk(tokens=1 << 29), h, h, h, h, None) == UNSUPPORTED
    assert fn("svdq_qk_norm_rope")(qk(), heads(n=0), h, heads(n=0), h, None) == INVALID
    assert fn("svdq_qk_norm_rope")(None, h, h, h, h, None) == INVALID


@pytest.mark.parametrize("tokens", [(1 << 31) // 4, 1 << 40, (1 << 62) + 1, (1 << 63) - 1])
def test_sizes_past_what_a_launch_holds_are_refused_without_overflow(tokens):
    h, n = heads(), C.c_size_t()
    assert fn("svdq_qk_norm_rope")(qk(tokens=tokens), h, h, h, h, None) == UNSUPPORTED
    assert fn("svdq_qk_backward_workspace")(qk(tokens=tokens), 4, 4, n) == UNSUPPORTED
    assert fn("svdq_qk_norm_rope_backward")(qk(tokens=tokens), h, h, h, h, h, h, P, P, P, 1 << 30, None) == UNSUPPORTED
    assert fn("svdq_kv_append")(qk(tokens=tokens), None, h, h, None, cache(), P, None) == UNSUPPORTED
    assert fn("svdq_kv_read")(cache(), P, tokens, S.F16, h, h, None) == UNSUPPORTED
    q = heads(8, 1024, 128)
    for change in (dict(requests=tokens), dict(tokens=tokens, max_q=(1 << 31) - 1, requests=1 << 20)):
        assert fn("svdq_kv_attention")(attn(**change), q, cache(), q, None, P, 1 << 30, None) == UNSUPPORTED


def test_backward_workspace():
    n = C.c_size_t()
    assert fn("svdq_qk_backward_workspace")(qk(), 4, 4, n) == OK and n.value == 2 * 2 * 128 * 4    # 40 rows: two groups of 32
    assert fn("svdq_qk_backward_workspace")(qk(), 0, 4, n) == INVALID
    assert fn("svdq_qk_backward_workspace")(qk(), 4, 4, None) == INVALID
    h = heads()
    f = fn("svdq_qk_norm_rope_backward")
    assert f(qk(), h, h, h, h, h, h, P, P, None, 0, None) == INVALID
    assert f(qk(), h, h, h, h, h, h, P, P, P, n.value - 1, None) == CAPACITY
    assert f(qk(), h, h, h, h, h, h, P, P, C.c_void_p(4100), n.value, None) == INVALID


@pytest.mark.parametrize("change,status", [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(v_codes=4104), SHAPE),
                                           (dict(page_size=48), SHAPE), (dict(head_dim=96), SHAPE), (dict(fmt=2), UNSUPPORTED),
                                           (dict(heads=0), INVALID), (dict(n_pages=1 << 40), UNSUPPORTED)])
def test_cache_refusals(change, status):
    h = heads()
    assert fn("svdq_kv_append")(qk(), h, h, h, h, cache(**change), P, None) == status
    assert fn("svdq_kv_read")(cache(**change), P, 10, S.F16, h, h, None) == status
    assert fn("svdq_kv_attention")(attn(), h, cache(**change), h, None, P, 1 << 30, None) == status


def test_append_refusals():
    h = heads()
    f = fn("svdq_kv_append")
    assert f(qk(), h, h, h, None, cache(), P, None) == INVALID
    assert f(qk(), None, h, h, h, cache(), P, None) == INVALID
    assert f(qk(), None, h, h, None, cache(), None, None) == INVALID
    assert f(qk(head_dim=64), None, h, h, None, cache(), P, None) == SHAPE
    assert f(qk(), None, heads(3), h, None, cache(), P, None) == SHAPE
    assert f(qk(), heads(0), h, h, heads(0), cache(), P, None) == SHAPE


def attn(**kw):
    d = kv.svdq_attn_desc(3, 10, 8, S.BF16, 4, 100, 0, kv.ATTN_CAUSAL, 0.1, P, P, P, 16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(requests=-1), INVALID), (dict(tokens=-1), INVALID), (dict(dtype=3), INVALID), (dict(flags=2), INVALID),
    (dict(max_q=-1), INVALID), (dict(max_kv=-1), INVALID), (dict(window=-1), INVALID), (dict(table_stride=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(q_heads=10), SHAPE), (dict(scale=float("nan")), INVALID), (dict(q_start=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(block_table=None), INVALID), (dict(requests=1 << 40), UNSUPPORTED)])
def test_attention_refusals(change, status):
    q = heads(8, 1024, 128)
    if "q_heads" in change:
        q = heads(change["q_heads"], 2048, 128)
    assert fn("svdq_kv_attention")(attn(**change), q, cache(), q, None, P, 1 << 30, None) == status


def test_attention_views_and_workspace():
    q, n = heads(8, 1024, 128), C.c_size_t()
    f = fn("svdq_kv_attention")
    assert f(attn(), heads(4), cache(), q, None, P, 1 << 30, None) == SHAPE
    assert f(attn(), q, cache(), heads(8, 1028), None, P, 1 << 30, None) == SHAPE
    assert f(attn(), None, cache(), q, None, P, 1 << 30, None) == INVALID
    assert f(attn(requests=0), q, cache(), q, None, None, 0, None) == OK
    assert f(attn(tokens=0), q, cache(), q, None, None, 0, None) == OK
    big = dict(max_kv=100000, table_stride=4000)
    assert fn("svdq_kv_attention_workspace")(attn(**big), cache(), n) == OK and n.value > 0
    assert f(attn(**big), q, cache(), q, None, None, 0, None) == INVALID
    assert f(attn(**big), q, cache(), q, None, P, 256, None) == CAPACITY
    assert f(attn(**big), q, cache(), q, None, C.c_void_p(4112), 1 << 40, None) == INVALID


def test_one_workspace_serves_every_window():
    full, part = C.c_size_t(), C.c_size_t()
    for kv_len in (1, 127, 128, 129, 1300, 8191, 100000):
        for requests in (1, 3, 64):
            base = dict(max_kv=kv_len, requests=requests, tokens=4 * requests)
            assert fn("svdq_kv_attention_workspace")(attn(**base), cache(), full) == OK
            for window in (1, 31, 1269, 1280, 5000):
                for flags in (0, kv.ATTN_CAUSAL):
                    assert fn("svdq_kv_attention_workspace")(attn(window=window, flags=flags, **base), cache(), part) == OK
                    assert part.value == full.value


def test_plan_and_release_refusals():
    f = fn("svdq_kv_plan")
    good = [P, P, 4, 16, 8, P, P, 100, P, 10, P, P, P, P, C.c_void_p(8192), P, None]

    def with_(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    assert with_(_2=-1) == INVALID and with_(_4=-1) == INVALID and with_(_7=-1) == INVALID and with_(_9=-1) == INVALID
    assert with_(_3=24) == INVALID
    assert with_(_2=8193) == UNSUPPORTED and with_(_4=1 << 31) == UNSUPPORTED
    for at in (0, 1, 5, 6, 8, 10, 11, 12, 13, 14, 15):
        assert with_(**{f"_{at}": None}) == INVALID, at
    assert with_(_14=P) == INVALID          # free_left may not be free_count
    r = fn("svdq_kv_release")
    good_r = [P, 4, 16, P, 10, P, P, P, 100, None]
    for at in (0, 3, 5, 6, 7):
        a = list(good_r)
        a[at] = None
        assert r(*a) == INVALID, at
    for at, v, st in ((1, -1, INVALID), (1, 8193, UNSUPPORTED), (2, 24, INVALID), (4, -1, INVALID), (8, -1, INVALID)):
        a = list(good_r)
        a[at] = v
        assert r(*a) == st, (at, v)
    assert r(None, 0, 16, None, 0, None, None, P, 0, None) == OK
