"""CPU tests of how the calls of the group norm and the cross attention are cut
(csrc/svdq_image_cut.h, the same code as in the kernels and in their launch),
built with g++ and UndefinedBehaviorSanitizer: every pixel, row, state and pair
belongs to one workgroup, what a launch and its workgroups hold fits, and a
request's rows and states lie inside the operands whatever its offsets say."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "diffusion_smooth_group_amd", "csrc")
OUT = os.path.join(ROOT, "_build", "image_cut")
MIN32, MAX32 = -(1 << 31), (1 << 31) - 1
OK, UNSUPPORTED = 0, 3
LDS, THREADS = 160 * 1024, 1 << 32

SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "svdq_image_cut.h"
using namespace svdq_image;
struct P {
  const int32_t *q_start, *k_start;
  int32_t tokens, states, max_q, max_k;
};
int main() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    if (!strcmp(what, "norm")) {
      long long samples, pixels, channels, groups, grad;
      if (scanf("%lld %lld %lld %lld %lld", &samples, &pixels, &channels, &groups, &grad) != 5) return 1;
      svdq_norm_desc d = {};
      d.samples = samples; d.pixels = pixels; d.channels = int32_t(channels); d.groups = int32_t(groups);
      NormCut t = {};
      const int st = int(norm_cut(&d, grad != 0, &t));
      printf("%d %d %d %d %d %d %d %lld %zu %zu %zu\n", st, t.threads, t.cv, t.rows, t.block, t.pieces, t.chunks, (long long)t.chunk,
             st ? 0 : norm_lds(t), st ? 0 : norm_join_lds(d.groups, t.threads), st ? 0 : norm_bytes(&d, t, grad != 0));
    } else if (!strcmp(what, "cross")) {
      long long requests, tokens, states, max_q, max_k, q_heads, k_heads, dim, cus, grad;
      if (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &requests, &tokens, &states, &max_q, &max_k, &q_heads, &k_heads, &dim, &cus, &grad) != 10) return 1;
      svdq_cross_desc d = {};
      d.requests = requests; d.tokens = tokens; d.states = states; d.max_q = int32_t(max_q); d.max_k = int32_t(max_k); d.head_dim = int32_t(dim);
      CrossCut t = {};
      const int st = int(cross_cut(&d, int(q_heads), int(k_heads), int(cus), grad != 0, &t));
      printf("%d %d %d %d %d %d %d %d %d %d %d %d %lld %lld %lld\n", st, t.group, t.pairs, t.row_slots, t.rows, t.row_tiles, t.splits, t.chunk, int(t.few_keys),
             t.key_tiles, t.row_splits, t.row_chunk, st ? 0LL : (long long)cross_part_floats(&d, t, grad != 0), st ? 0LL : (long long)cross_delta_floats(t, int(q_heads)),
             st ? 0LL : (long long)cross_key_floats(&d, t));
    } else if (!strcmp(what, "range")) {
      long long r, tokens, states, max_q, max_k, q0, q1, k0, k1, dense;
      if (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &r, &tokens, &states, &max_q, &max_k, &q0, &q1, &k0, &k1, &dense) != 10) return 1;
      const int32_t q[2] = {int32_t(q0), int32_t(q1)}, k[2] = {int32_t(k0), int32_t(k1)};
      const P p = {dense ? nullptr : q, dense ? nullptr : k, int32_t(tokens), int32_t(states), int32_t(max_q), int32_t(max_k)};
      const CrossRange c(p, int(r));
      printf("%d %d %d %d\n", c.q_first, c.rows, c.k_first, c.keys);
    } else {
      long long pairs, tiles;
      if (scanf("%lld %lld", &pairs, &tiles) != 2) return 1;
      for (long long i = 0; i < pairs * tiles; ++i) {
        const PairWork w{unsigned(i), int(pairs), int(tiles)};
        printf("%d %d ", w.pair, w.tile);
      }
      printf("\n");
    }
  }
}
"""


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


def run(exe, what, cases):
    r = subprocess.run([exe], input="".join(" ".join([what, *map(str, c)]) + "\n" for c in cases), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = [list(map(int, line.split())) for line in r.stdout.splitlines()]
    assert len(out) == len(cases)
    return out


def spread(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


# ------------------------------------------------------------------ group norm
def test_norm_cuts(program):
    rng = random.Random(1)
    cases = [(1, 64, 1280, 32, 0), (1, 512 * 512, 128, 32, 0), (256, 65536, 8, 1, 1), (1, 1, 8192, 8192, 1), (1, 1 << 36, 8, 1, 0), (1, 1 << 36, 8, 1, 1),
             (1 << 22, 9216, 32, 32, 0), ((1 << 31) - 1, 1, 8, 1, 1), (1, 1 << 57, 8, 1, 0), (64, 1 << 20, 1024, 32, 0), (300, 70000, 16, 4, 1)]
    for _ in range(4000):
        groups = rng.choice([1, 2, 3, 4, 5, 8, 16, 24, 32, 64, 512, 8192])
        per = spread(rng, 1, 8192 // groups)
        while groups * per % 8:
            per += 1
        if groups * per <= 8192:
            cases.append((spread(rng, 1, 1 << 24), spread(rng, 1, 1 << 22), groups * per, groups, rng.randrange(2)))
    took = {OK: 0, UNSUPPORTED: 0}
    for case, got in zip(cases, run(program, "norm", cases)):
        samples, pixels, channels, groups, grad = case
        status, threads, cv, rows, block, pieces, chunks, chunk, lds, join, size = got
        took[status] += 1
        if status != OK:
            continue
        assert threads % 64 == 0 and 64 <= threads <= 1024 and cv * rows <= threads and rows >= 1, case
        if block:
            assert groups % block == 0 and block <= 32 and cv * 8 == block * (channels // groups), case
            assert (pieces - 1) * rows < pixels <= pieces * rows and pieces <= (4 if grad else 8) and (not grad or threads <= 512), case
            assert samples * (groups // block) * threads < THREADS, case
            assert (2 * lds + cv * 64 if grad else lds) + 1024 <= LDS, case
            assert size == (samples * channels * 8 if grad and samples > 2 else 0), case
        else:
            assert cv * 8 == channels and chunk % rows == 0 and (chunks - 1) * chunk < pixels <= chunks * chunk and chunk <= 1 << 30, case
            assert (samples * chunks + (-(-channels // 32) if grad else 0)) * threads < THREADS, case
            # 256 pixels a thread, or a 256th of a sample's
            assert chunk <= max(256 * rows, -(-pixels // 256) + rows), case
            assert 2 * lds <= LDS and 512 * 4 <= join <= LDS, case
            assert size == samples * chunks * (groups + (channels if grad else 0)) * 8, case
    assert took[OK] > 2000 and took[UNSUPPORTED] > 20


# ------------------------------------------------------------- cross attention
def test_cross_cuts(program):
    rng = random.Random(2)
    cases = [(1, 1, 1, 1, 1, 1, 1, 8, 256, 0), (1, 1, 1 << 30, 1, 1 << 30, 1, 1, 128, 256, 0), (1, 1, 1 << 30, 1, 1 << 30, 1, 1, 128, 256, 1),
             (1, (1 << 30) - 1, 77, MAX32, MAX32, 1, 1, 64, 256, 1), (2, 10, 20, MAX32, MAX32, 8, 8, 64, 256, 1), (3, 0, 100, 0, 50, 4, 4, 64, 256, 1),
             (3, 100, 0, 50, 0, 4, 2, 64, 256, 1), ((1 << 30) - 1, 5, 5, 1, 1, 1, 1, 64, 256, 0)]
    for _ in range(4000):
        heads = spread(rng, 1, 64)
        requests, tokens, states = spread(rng, 1, 1 << 14), spread(rng, 1, 1 << 24), spread(rng, 1, 1 << 24)
        cases.append((requests, tokens, states, spread(rng, 1, tokens) if rng.random() < 0.9 else MAX32, spread(rng, 1, states) if rng.random() < 0.9 else MAX32,
                      heads * spread(rng, 1, 32), heads, 8 * rng.randrange(1, 17), rng.choice([256, 304, 32]), rng.randrange(2)))
    took = {OK: 0, UNSUPPORTED: 0}
    for case, got in zip(cases, run(program, "cross", cases)):
        requests, tokens, states, max_q, max_k, q_heads, k_heads, dim, cus, grad = case
        status, group, pairs, slots, rows, row_tiles, splits, chunk, few, key_tiles, row_splits, row_chunk, part, delta, key_part = got
        took[status] += 1
        if status != OK:
            continue
        most_q, most_k = min(max_q, tokens), min(max_k, states)
        assert group == q_heads // k_heads and pairs == requests * k_heads and slots == most_q * group and pairs * slots < 1 << 30, case
        assert rows in ((128,) if grad else (16, 128)) and (row_tiles - 1) * rows < slots <= row_tiles * rows or slots == row_tiles == 0, case
        assert splits >= 1 and chunk % 128 == 0 and (splits - 1) * chunk < max(most_k, 1) <= splits * chunk, case
        assert row_splits >= 1 and row_chunk % 64 == 0 and (row_splits - 1) * row_chunk < max(slots, 1) <= row_splits * row_chunk, case
        assert (key_tiles - 1) * 128 < most_k <= key_tiles * 128 or most_k == key_tiles == 0, case
        assert bool(few) == (most_k <= 128) and (not few or splits == 1), case
        # sums of two of these are 32-bit in the kernels
        assert most_k + chunk <= 1 << 31 and slots + row_chunk + 64 <= MAX32, case
        assert pairs * row_tiles * splits * 256 < THREADS and (splits == 1 or -(-pairs * slots // 4) * 256 < THREADS), case
        assert part == (pairs * slots * splits * (dim + (0 if grad else 2)) if splits > 1 else 0), case
        if grad:
            assert pairs * key_tiles * row_splits * 256 < THREADS and (row_splits == 1 or pairs * key_tiles * 32 * 256 < THREADS), case
            assert tokens * q_heads <= delta < tokens * q_heads + 64, case
            assert key_part == (pairs * key_tiles * 128 * row_splits * dim * 2 if row_splits > 1 else 0), case
    assert took[OK] > 2000 and took[UNSUPPORTED] > 20


@pytest.mark.parametrize("pairs", [1, 3, 8, 12, 16, 24, 40, 63])
def test_every_tile_of_every_pair_is_some_workgroups(program, pairs):
    cases = [(pairs, tiles) for tiles in (1, 2, 7, 8, 33)]
    for (_, tiles), got in zip(cases, run(program, "pairs", cases)):
        work = list(zip(got[::2], got[1::2]))
        assert sorted(work) == [(p, t) for p in range(pairs) for t in range(tiles)]
        if pairs % 8 == 0:              # a pair's workgroups go to one of eight dies
            assert all(len({i % 8 for i, (p, _) in enumerate(work) if p == q}) == 1 for q in range(pairs))


def test_ranges_lie_inside_the_operands(program):
    rng = random.Random(3)
    ends = (MIN32, MIN32 + 1, -1, 0, 1, 77, 4095, 4096, 4097, MAX32 - 1, MAX32)
    cases = [(0, 4096, 4096, most, most, a, b, b, a, 0) for a in ends for b in ends for most in (0, 1, 4096, MAX32)]
    for _ in range(2000):
        some = lambda: rng.choice([rng.randint(MIN32, MAX32), rng.randint(-10, 5000), rng.choice(ends)])
        cases.append((0, rng.choice([0, 1, 4096, MAX32 - 512]), rng.choice([0, 1, 4096, MAX32 - 512]), rng.choice([0, 3, 4096, MAX32]), rng.choice([0, 3, 4096, MAX32]),
                      some(), some(), some(), some(), 0))
    for case, (q_first, rows, k_first, keys) in zip(cases, run(program, "range", cases)):
        _, tokens, states, max_q, max_k, q0, q1, k0, k1, _ = case
        for first, n, most, all_, a, b in ((q_first, rows, max_q, tokens, q0, q1), (k_first, keys, max_k, states, k0, k1)):
            assert 0 <= n <= most and (n == 0 or 0 <= first and first + n <= all_), case
            inside = 0 <= a <= b <= all_
            assert not inside or (n == min(b - a, most) and (n == 0 or first == a)), case
    dense = [(r, 7 * 100, 7 * 33, 100, 33, 0, 0, 0, 0, 1) for r in range(7)] + [(3, 4 * ((1 << 29) - 200), 4 * 9, (1 << 29) - 200, 9, 0, 0, 0, 0, 1)]
    for (r, _, _, max_q, max_k, *_), got in zip(dense, run(program, "range", dense)):
        assert got == [r * max_q, max_q, r * max_k, max_k]
