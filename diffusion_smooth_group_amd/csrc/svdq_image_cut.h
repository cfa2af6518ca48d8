// svdq_image_cut.h -- how the calls of include/svdq_image.h are cut into
// workgroups.  Integer arithmetic only, shared by the host, the kernels and the
// CPU tests.
#pragma once
#include <cstddef>
#include <cstdint>

#include "svdq_image.h"
#include "svdq_kv_cut.h"

namespace svdq_image {

using svdq_kv::ceil_div;
using svdq_kv::larger;
using svdq_kv::product_below;
using svdq_kv::smaller;

// ------------------------------------------------------------------ group norm
constexpr int NORM_FEW_SAMPLES = 2;
constexpr int NORM_MAX_BLOCK = 32;      // groups of a workgroup of the one-launch form
constexpr int NORM_MOST_PIXELS = 256;   // pixels of a thread of the two-launch form, more in samples of 2^29 elements and up

struct NormCut {
  int threads;
  int cv, rows;             // 16-byte pieces of a pixel that a workgroup takes, pixels in flight in it
  int block, pieces;        // one launch: groups of a workgroup, pieces a thread; block = 0: two launches
  int chunks;               // two launches: chunks of a sample's pixels, of
  int64_t chunk;            // so many pixels (the last: the rest)
};

// One launch where a workgroup's share fits its registers: as many groups as make
// whole 16-byte pieces, up to 512 threads with four pieces each, forward also 1024
// with eight (1 x 32 x 32 x 640: 13.9 us on the GPU in one launch, 17.7 in two, and
// 9 instead of 14 on the host).  Its gradient's sums over samples: up to
// NORM_FEW_SAMPLES the same launch takes the samples in turn (2 x 8 x 8 x 1280: 14.0 us
// a call, 19.7 with a launch for the sums; four samples: 14.5 on the GPU against 7.3).
// Two launches: a workgroup of about 1024 threads a compute unit (1 x 512 x 512 x
// 128, when the kernels were slower: 42.5 us with 256, 44 with 512 of 512 threads, 47
// with 512 of 1024; the gradient of 2 x 128 x 128 x 320: 30, 34, 40): each joins all
// chunks of its sample.  More of them where a thread would have more than
// NORM_MOST_PIXELS, up to 256 a sample, so that sums of one after the other stay short.
inline svdq_status norm_cut(const svdq_norm_desc* d, bool grad, NormCut* out) {
  NormCut t = {};
  const int per = d->channels / d->groups;
  t.chunks = 1;
  t.chunk = d->pixels;
  int block = 1;
  while (block * per % 8 != 0) block *= 2;
  const int cv = block * per / 8;
  for (int most = 512; most <= (grad ? 512 : 1024) && cv <= 512; most *= 2) {
    const int64_t room = most / cv, rows = d->pixels < room ? (d->pixels < 1 ? 1 : d->pixels) : room;
    const int64_t pieces = ceil_div(d->pixels, rows);
    if (pieces <= (most == 512 ? 4 : 8)) {
      t.cv = cv; t.rows = int(rows); t.block = block; t.pieces = int(pieces);
      t.threads = int(ceil_div(int64_t(cv) * rows, 64)) * 64;
      if (product_below(d->samples, d->groups / block, t.threads, svdq_kv::MAX_THREADS) < 0) return SVDQ_ERR_UNSUPPORTED;
      *out = t;
      return SVDQ_OK;
    }
  }
  t.cv = d->channels / 8;
  // the thread count from 512 to 1024 that leaves the fewest idle
  int best = 0;
  for (int n = 512; n <= 1024; n += 64) {
    const int rows = n / t.cv;
    if (rows < 1) continue;
    const int used = rows * t.cv * 1024 / n;
    if (used >= best) { best = used; t.threads = n; t.rows = rows; }
  }
  const int64_t want = 256 / (d->samples < 1 ? 1 : d->samples);
  auto chunk_of = [&](int64_t n) { return ceil_div(ceil_div(d->pixels, n), t.rows) * t.rows; };
  t.chunk = chunk_of(want < 1 ? 1 : want);
  const int64_t most = int64_t(t.rows) * NORM_MOST_PIXELS, least = chunk_of(256);
  if (t.chunk > most) t.chunk = most > least ? most : least;
  const int64_t chunks = ceil_div(d->pixels, t.chunk);
  if (t.chunk > int64_t(1) << 30) return SVDQ_ERR_UNSUPPORTED;      // a chunk's pixels are a 32-bit number in the kernels
  // the gradient's second launch has workgroups of 32 channels behind the chunks'
  const int64_t work = product_below(d->samples, chunks, 1, svdq_kv::MAX_THREADS);
  if (work < 0 || product_below(work + (grad ? ceil_div(d->channels, 32) : 0), t.threads, 1, svdq_kv::MAX_THREADS) < 0) return SVDQ_ERR_UNSUPPORTED;
  t.chunks = int(chunks);
  *out = t;
  return SVDQ_OK;
}

// LDS of one sum a channel and row of pixels (rows of an odd length, so that the
// channels of neighbouring threads lie in banks of their own)
inline size_t norm_lds(const NormCut& t) { return size_t(t.cv) * 8 * size_t(t.rows | 1) * 4; }

// and of the join of chunks: three sums a group, three a thread where a group has several
inline size_t norm_join_lds(int groups, int threads) { return size_t(3) * size_t(groups + threads) * 4; }

inline size_t norm_bytes(const svdq_norm_desc* d, const NormCut& t, bool grad) {
  if (d->samples == 0) return 0;
  const size_t n = size_t(d->samples);
  if (t.block > 0) return grad && d->samples > NORM_FEW_SAMPLES ? n * size_t(d->channels) * 8 : 0;
  return n * size_t(t.chunks) * size_t(d->groups + (grad ? d->channels : 0)) * 8;
}

// ------------------------------------------------------------- cross attention
// A request's rows and states; offsets outside the operands give none.
struct CrossRange {
  int q_first, rows, k_first, keys;
  template <class P>
  SVDQ_HD CrossRange(const P& p, int r) {
    span(p.q_start, r, p.max_q, p.tokens, &q_first, &rows);
    span(p.k_start, r, p.max_k, p.states, &k_first, &keys);
  }
  SVDQ_HD static void span(const int32_t* start, int r, int most, int all, int* first, int* n) {
    const int s = start ? start[r] : r * most, e = start ? smaller(start[r + 1], all) : s + most;
    *first = s;
    *n = s < 0 || e <= s ? 0 : smaller(e - s, most);
  }
};

// Pairs (request, key head) with `tiles` workgroups each.  Workgroups go to the
// chip's eight dies in turn, each with a cache of its own: where the pairs
// divide by eight a pair's workgroups are eight apart, so that its keys and
// values are read into one of the caches only.
struct PairWork {
  int pair, tile;
  SVDQ_HD PairWork(unsigned id, int pairs, int tiles) {
    if (pairs % 8 == 0) {
      pair = int(id / 8u / unsigned(tiles) * 8u + id % 8u);
      tile = int(id / 8u % unsigned(tiles));
    } else {
      pair = int(id % unsigned(pairs));
      tile = int(id / unsigned(pairs));
    }
  }
};

struct CrossCut {
  int group, pairs;         // query heads a key head, requests x key heads
  int tokens, states;
  int row_slots;            // rows of a pair: query tokens x heads of the group, the heads fastest
  int rows;                 // rows of a tile: 16 or 128
  int row_tiles, splits, chunk;   // and chunks of a pair's keys
  bool few_keys;            // gradient: 128 at most, which lie in LDS at once
  int key_tiles, row_splits, row_chunk;   // gradient of keys: tiles of KEY_TILE keys, chunks of a pair's rows
};

constexpr int KEY_TILE = 128;

inline svdq_status cross_cut(const svdq_cross_desc* d, int q_heads, int k_heads, int cus, bool grad, CrossCut* out) {
  CrossCut t = {};
  t.group = q_heads / k_heads;
  const int64_t max_q = d->max_q < d->tokens ? d->max_q : d->tokens, max_k = d->max_k < d->states ? d->max_k : d->states;
  const int64_t slots = max_q * t.group;
  const int64_t pairs = product_below(d->requests, k_heads, 1, int64_t(1) << 30);
  // offsets into rows and keys are 32-bit, a chunk's and a stage's past the end as well
  if (pairs < 0 || product_below(pairs, slots, 1, int64_t(1) << 30) < 0 || max_k > int64_t(1) << 30 || product_below(pairs, max_k, 1, int64_t(1) << 40) < 0)
    return SVDQ_ERR_UNSUPPORTED;
  t.pairs = int(pairs);
  t.tokens = int(d->tokens);
  t.states = int(d->states);
  t.row_slots = int(slots);
  auto clamp = [](int64_t v, int64_t most) { v = v > most ? most : v; return v < 1 ? int64_t(1) : v; };
  const int64_t per = pairs > 0 ? pairs : 1;
  // Up to 16 rows a pair one tile of 16, whose waves share the keys; above it tiles
  // of 128, whose waves share the rows (8 x 32 rows, 20 heads of 64, 1500 states: 17.7
  // us against 18.1 in two tiles of 16; 40 rows, 8 heads of 128, 4096 states: 20.0
  // against 27.2; 64 x 32 rows over 77: 7.1 against 8.4).
  t.rows = !grad && slots <= 16 ? 16 : 128;
  t.row_tiles = int(ceil_div(slots, t.rows));
  // Chunks of keys where the tiles leave half the chip idle, two workgroups a compute
  // unit, of at least 256 keys (few rows) or 512 (64 x 1 row, 8 heads in groups of
  // four, up to 4096 states: 148 us without, 159 with two chunks, 150 with three; 8 x
  // 1, 20 heads of 64, 1500 states: 14.4 us and the join's 3.9 with three or six).
  const int64_t items = per * larger(t.row_tiles, 1);
  const int64_t n = clamp(int64_t(cus) * 2 / items, ceil_div(max_k, t.rows == 16 ? 256 : 512));
  t.chunk = int(ceil_div(ceil_div(max_k > 0 ? max_k : 1, n), 128) * 128);
  t.splits = int(ceil_div(max_k > 0 ? max_k : 1, t.chunk));
  t.few_keys = max_k <= 128;
  t.key_tiles = int(ceil_div(max_k, KEY_TILE));
  // Chunks of rows, the same (24 heads of 128, 4608 rows over 512 states: 87 us and the
  // join's 13 with five, 149 + 8 with two, 110 + 17 with eight; 2 x 4096 over 77, 10
  // heads of 64: 15.2 + 6 with 22, 18.4 + 4 with 11, 19.4 + 7 with 32).
  const int64_t kitems = per * larger(t.key_tiles, 1);
  const int64_t m = clamp(int64_t(cus) * 2 / kitems, ceil_div(slots, 128));
  t.row_chunk = int(ceil_div(ceil_div(slots > 0 ? slots : 1, m), 64) * 64);
  t.row_splits = int(ceil_div(slots > 0 ? slots : 1, t.row_chunk));
  // (a join's launch is smaller: only calls of few tiles are cut)
  if (product_below(pairs, t.row_tiles, t.splits, svdq_kv::MAX_THREADS / 256) < 0 ||
      (grad && product_below(pairs, t.key_tiles, t.row_splits, svdq_kv::MAX_THREADS / 256) < 0))
    return SVDQ_ERR_UNSUPPORTED;
  *out = t;
  return SVDQ_OK;
}

// bytes of the workspace: partial rows of the forward call or of dq
inline int64_t cross_part_floats(const svdq_cross_desc* d, const CrossCut& t, bool grad) {
  return t.splits > 1 ? int64_t(t.pairs) * t.row_slots * t.splits * (d->head_dim + (grad ? 0 : 2)) : 0;
}
inline int64_t cross_delta_floats(const CrossCut& t, int q_heads) { return ceil_div(int64_t(t.tokens) * q_heads, 64) * 64; }
inline int64_t cross_key_floats(const svdq_cross_desc* d, const CrossCut& t) {
  return t.row_splits > 1 ? int64_t(t.pairs) * t.key_tiles * KEY_TILE * t.row_splits * d->head_dim * 2 : 0;
}

}  // namespace svdq_image
