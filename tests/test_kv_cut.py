"""CPU tests of how an attention call over the 4-bit cache is cut
(csrc/svdq_kv_cut.h, the same code as in the kernels and in their launch),
built with g++ and UndefinedBehaviorSanitizer: which keys a row sees, and that
the chunks of a row tile are its keys, up to the largest arguments."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "diffusion_smooth_group_amd", "csrc")
OUT = os.path.join(ROOT, "_build", "kv_cut")
MAX32 = (1 << 31) - 1
UNSUPPORTED = 3

SOURCE = r"""
#include <cstdio>
#include "svdq_kv_cut.h"
using namespace svdq_kv;
struct P {
  const int32_t *q_start, *kv_len;
  int32_t tokens, max_q, max_kv, window, causal, group, chunk;
};
int main() {
  long long requests, tokens, q_heads, max_q, max_kv, window, causal, stride, shift, heads, dim, cus, s, e, len;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &requests, &tokens, &q_heads, &max_q,
               &max_kv, &window, &causal, &stride, &shift, &heads, &dim, &cus, &s, &e, &len) == 15) {
    svdq_attn_desc d = {};
    d.requests = requests; d.tokens = tokens; d.q_heads = int32_t(q_heads); d.max_q = int32_t(max_q); d.max_kv = int32_t(max_kv);
    d.window = int32_t(window); d.flags = causal ? SVDQ_ATTN_CAUSAL : 0u; d.table_stride = stride;
    svdq_kv_cache c = {};
    c.n_pages = 1000; c.page_size = 1 << shift; c.heads = int32_t(heads); c.head_dim = int32_t(dim);
    Cut t = {};
    const int st = int(cut_of(&d, &c, int(cus), &t));
    printf("%d %d %d %d %lld %lld", st, t.rows, t.splits, t.chunk, (long long)(st ? 0 : part_rows(&d, &c, t)),
           (long long)(st ? 0 : most_part_rows(&d, &c, int(cus))));
    if (st == 0) {
      const int32_t start[2] = {int32_t(s), int32_t(e)}, length[1] = {int32_t(len)};
      const P p = {start, length, t.tokens, d.max_q, t.keys, d.window, int32_t(causal), int32_t(q_heads / heads), t.chunk};
      const Request r(p, 0);
      printf(" %d", r.rows);
      if (r.rows > 0) {
        const int rows = r.rows * p.group, tiles = (rows + t.rows - 1) / t.rows;
        for (int i : {0, r.rows - 1}) printf(" %d %d", r.low(p, i), r.high(p, i));
        for (int rt : {0, tiles - 1}) {
          const TileRange g(p, r, rt, t.rows);
          printf(" %d %d %d %d %d", g.first, g.last, g.from, g.to, g.n);
          for (int i : {0, g.n - 1}) printf(" %d %d", i < 0 ? 0 : g.chunk_from(p, i), i < 0 ? 0 : g.chunk_to(p, i));
        }
      }
    }
    printf("\n");
  }
}
"""
FIELDS = ("requests", "tokens", "q_heads", "max_q", "max_kv", "window", "causal", "stride", "shift", "heads", "dim", "cus", "start",
          "end", "length")


@pytest.fixture(scope="module")
def program():
    os.makedirs(OUT, exist_ok=True)
    src, exe = os.path.join(OUT, "cut.cpp"), os.path.join(OUT, "cut")
    with open(src, "w") as f:
        f.write(SOURCE)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run([shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(rocm, "include"), "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                    src, "-o", exe], check=True, capture_output=True)
    return exe


def run(exe, cases):
    text = "".join(" ".join(str(int(c[f])) for f in FIELDS) + "\n" for c in cases)
    r = subprocess.run([exe], input=text, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return [list(map(int, line.split())) for line in r.stdout.splitlines()]


def case(**kw):
    c = dict(requests=3, tokens=12, q_heads=8, max_q=4, max_kv=100, window=0, causal=1, stride=16, shift=5, heads=4, dim=128, cus=256,
             start=0, end=4, length=100)
    return c | kw


def check(c, got):
    """Against the definition in Python's integers."""
    status, tile_rows, splits, chunk, part, most = got[:6]
    assert part <= most, c
    if status:
        return
    n = min(c["end"], c["tokens"]) - c["start"]
    rows = max(0, min(n, c["max_q"]))
    assert got[6] == rows, c
    if rows == 0:
        return
    room = c["stride"] << c["shift"]
    length = max(0, min(c["length"], c["max_kv"], room))
    last_pos = c["length"] - (c["end"] - c["start"])

    def sees(i):
        pos = last_pos + i
        return (min(length, max(0, pos - c["window"] + 1)) if c["window"] else 0), (max(0, min(pos + 1, length)) if c["causal"] else length)
    assert got[7:11] == [*sees(0), *sees(rows - 1)], c
    group = c["q_heads"] // c["heads"]
    tiles = -(-rows * group // tile_rows)
    at = 11
    for rt in (0, tiles - 1):
        first, last, begin, end, chunks, f0, t0, f1, t1 = got[at:at + 9]
        at += 9
        assert (first, last) == (rt * tile_rows // group, min(rows - 1, (rt * tile_rows + tile_rows - 1) // group)), c
        assert (begin, end) == (sees(first)[0] // 32 * 32, sees(last)[1]), c
        if end <= begin:
            assert chunks == 0, c
            continue
        # the chunks are the tile's keys, and none is left out of the launch
        assert chunk > 0 and chunk % 128 == 0 and 1 <= chunks <= splits, c
        assert (f0, t0) == (begin, min(end, begin + chunk)) and t1 == end and f1 == begin + (chunks - 1) * chunk < end, c
        # indexes past the end that a kernel computes, before it bounds them, fit 32 bits
        assert end + (1 << 14) <= MAX32, c


def test_a_length_bound_of_int32_max(program):
    """The natural value of "no bound", with few and with many requests: the
    largest product of a table is what counts."""
    cases = [case(requests=r, tokens=r, max_q=1, end=1, heads=8, q_heads=32, max_kv=m, window=w, causal=k, length=n)
             for r in (1, 2, 64, 256, 1024, 5000) for m in (MAX32, MAX32 - 100, 1 << 30) for w in (0, 1, 700, MAX32) for k in (0, 1)
             for n in (1, 100, 511)]
    got = run(program, cases)
    for c, g in zip(cases, got):
        assert g[0] == 0, c
        check(c, g)


def test_lengths_near_the_end_of_int32_are_refused(program):
    """Tables that wide are allowed by the interface; the kernels' key indexes
    are 32-bit."""
    wide = [case(max_kv=m, stride=s, length=m, requests=r, tokens=4 * r) for m in (MAX32, (1 << 30) + 1) for s in (1 << 26, 1 << 40)
            for r in (1, 400)]
    for c, g in zip(wide, run(program, wide)):
        assert g[0] == UNSUPPORTED, c
    held = [case(max_kv=(1 << 30) - (1 << 14), stride=1 << 40, length=(1 << 30) - (1 << 14), window=w, requests=r, tokens=4 * r)
            for w in (0, 5, MAX32) for r in (1, 400, 5000)]
    for c, g in zip(held, run(program, held)):
        assert g[0] == 0, c
        check(c, g)


def test_windows_and_offsets_at_the_ends_of_int32(program):
    """Rows far before the first cached token, under the widest windows."""
    cases = [case(window=w, causal=k, length=n, start=s, end=e, tokens=t, max_q=q) for w in (1, MAX32 - 1, MAX32) for k in (0, 1)
             for n in (0, 1, 100, -1, -(1 << 31), MAX32) for s, e, t, q in ((0, 4, 12, 4), (0, MAX32, 12, 4), (8, 12, 12, 4), (3, 3, 12, 4), (5, 2, 12, 4))]
    for c, g in zip(cases, run(program, cases)):
        check(c, g)


def test_random_calls(program):
    rng = random.Random(7)
    cases = []
    for _ in range(4000):
        heads, group = rng.choice([1, 2, 5, 8, 24]), rng.choice([1, 2, 4, 5, 8])
        max_q = int(2 ** rng.uniform(0, 12))
        max_kv = int(2 ** rng.uniform(0, 31)) - 1
        rows = rng.randint(0, max_q + 3)
        start = rng.randint(0, 50)
        cases.append(case(requests=int(2 ** rng.uniform(0, 10)), tokens=start + max_q + rng.randint(0, 50), q_heads=heads * group, heads=heads,
                          max_q=max_q, max_kv=max_kv, window=rng.choice([0, 0, 1, 100, max_kv // 3]), causal=rng.randint(0, 1),
                          stride=rng.choice([1, 16, 300, 100000]), shift=rng.choice([4, 5, 6, 7, 8]), dim=rng.choice([64, 128]),
                          start=start, end=start + rows, length=rng.randint(0, min(max_kv, 1 << 20)) + rng.randint(0, 5)))
    for c, g in zip(cases, run(program, cases)):
        assert g[0] == 0, c
        check(c, g)


def test_a_workspace_serves_every_smaller_call(program):
    """Fewer requests, tokens, rows or keys are cut into more chunks."""
    rng = random.Random(11)

    def some(most):
        return rng.choice([most, rng.randint(1, most), int(2 ** rng.uniform(0, 31)) % most + 1])
    cases, of = [], []
    for _ in range(600):
        heads, group = rng.choice([1, 2, 5, 8, 24]), rng.choice([1, 2, 4, 5, 8])
        requests, max_q = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 12))
        full = case(requests=requests, tokens=rng.choice([requests, requests * max_q]), q_heads=heads * group, heads=heads, max_q=max_q,
                    max_kv=int(2 ** rng.uniform(0, 17)), stride=100000, cus=rng.choice([256, 256, 64, 304]))
        at = len(cases)
        cases.append(full)
        of.append(at)
        for _ in range(30):
            cases.append(full | dict(requests=some(requests), tokens=some(full["tokens"]), max_q=some(max_q), max_kv=some(full["max_kv"]),
                                     window=rng.choice([0, 0, 1, 300]), causal=rng.randint(0, 1), stride=rng.choice([100000, 3, 700])))
            of.append(at)
    got = run(program, cases)
    for c, g, i in zip(cases, got, of):
        assert g[0] in (0, UNSUPPORTED)
        if g[0] == 0 and got[i][0] == 0:
            assert g[4] <= got[i][5] and g[5] <= got[i][5], (c, cases[i])


def test_workspaces_stay_within_what_fills_the_chip(program):
    """A bound, not a multiple of the largest shape: at most 65536 partial rows
    with 256 compute units."""
    cases = [case(requests=r, tokens=r * q, max_q=q, max_kv=1 << 20, stride=1 << 20, q_heads=64, heads=h) for r in (1, 100, 500)
             for q in (1, 100, 5000) for h in (1, 8, 64)]
    for c, g in zip(cases, run(program, cases)):
        assert g[0] == UNSUPPORTED or g[5] <= 65536, c
