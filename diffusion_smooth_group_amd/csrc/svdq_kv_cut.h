// svdq_kv_cut.h -- how an attention call over the 4-bit cache is cut into row
// tiles and key chunks, and which keys a row sees.  Integer arithmetic only,
// shared by the host, the kernels of svdq_kv_attn.hip and the CPU tests.
#pragma once
#include <cstddef>
#include <cstdint>

#include "svdq_kv.h"

#ifdef __HIPCC__
#define SVDQ_HD __host__ __device__ __forceinline__
#else
#define SVDQ_HD inline
#endif

namespace svdq_kv {

SVDQ_HD int smaller(int a, int b) { return a < b ? a : b; }
SVDQ_HD int larger(int a, int b) { return a > b ? a : b; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// a * b * c where all are not negative and the product is below `limit`; -1 otherwise
inline int64_t product_below(int64_t a, int64_t b, int64_t c, int64_t limit) {
  const __int128 p = __int128(a) * b;
  if (p >= limit && c > 0) return -1;
  const __int128 q = c > 0 ? p * c : 0;
  return q >= limit ? -1 : int64_t(q);
}
// threads of a launch's x dimension
constexpr int64_t MAX_THREADS = int64_t(1) << 32;

// A request's rows and the keys they see.  All in 32 bits, of which the scalar
// unit has comparisons, and without overflow for any offsets and lengths.
struct Request {
  int rows, len, first;
  int before;               // position of row 0 (below 0: rows that stand before the first token)
  template <class P>
  SVDQ_HD Request(const P& p, int r) {
    const int s = p.q_start[r], e = smaller(p.q_start[r + 1], p.tokens), held = larger(p.kv_len[r], 0);
    first = s;
    rows = s < 0 || e <= s ? 0 : smaller(e - s, p.max_q);
    before = rows > 0 ? held - (p.q_start[r + 1] - s) : 0;
    len = smaller(held, p.max_kv);
  }
  // keys [low, high) that row i sees
  template <class P>
  SVDQ_HD int high(const P& p, int i) const {
    return p.causal ? larger(0, smaller(before + i + 1, len)) : len;
  }
  template <class P>
  SVDQ_HD int low(const P& p, int i) const {
    const int end = before + i + 1;
    return p.window > 0 && end > p.window ? smaller(end - p.window, len) : 0;
  }
};

// the 16 rows of row tile rt: rows are (query, head of the group), head fastest
struct TileRange {
  int first, last;          // queries of the first and last row
  int from, to;             // keys that any row sees, `from` rounded down to 32
  int all_low, all_high;    // keys that every row sees
  int n;                    // chunks in use
  template <class P>
  SVDQ_HD TileRange(const P& p, const Request& r, int rt, int rows_per_tile) {
    first = rt * rows_per_tile / p.group;
    last = smaller(r.rows - 1, (rt * rows_per_tile + rows_per_tile - 1) / p.group);
    from = r.low(p, first) & ~31;
    to = r.high(p, last);
    all_low = r.low(p, last);
    all_high = r.high(p, first);
    n = to > from ? (to - from + p.chunk - 1) / p.chunk : 0;
  }
  // keys [chunk_from, chunk_to) of chunk i
  template <class P>
  SVDQ_HD int chunk_from(const P& p, int i) const { return from + i * p.chunk; }
  template <class P>
  SVDQ_HD int chunk_to(const P& p, int i) const { return smaller(to, chunk_from(p, i) + p.chunk); }
};

// How a call is cut: row tiles per request and head, and key chunks.
struct Cut {
  int64_t items;            // requests x heads x row tiles
  int64_t row_slots;        // rows of a request and head
  int rows;                 // rows of a tile: 16 (k_attn16), 128 or 256 (k_attn_rows)
  int row_tiles, splits, chunk;
  int keys, tokens;         // most keys of a request, query rows: the arguments within what they can be
};

inline svdq_status cut_of(const svdq_attn_desc* d, const svdq_kv_cache* c, int cus, Cut* out) {
  Cut t;
  const int64_t group = d->q_heads / c->heads;
  const int64_t max_q = d->max_q < d->tokens ? d->max_q : d->tokens;
  t.row_slots = max_q * group;
  const int64_t slots = product_below(d->requests, c->heads, t.row_slots, (int64_t(1) << 31) - 512);   // a tile's last row, too, is an int
  if (slots < 0) return SVDQ_ERR_UNSUPPORTED;
  // Up to 80 rows a request and head, or 1024 in all, tiles of 16 that read the
  // cache once each (8 requests of 4000 tokens, 8 heads: 40 rows 25 us against 29
  // with a tile of 128, 72 rows 31 against 31; one request and head: 128 rows 15
  // against 23, 512 rows 19 against 23; one request, 8 heads: 128 rows 24 against
  // 24, 256 rows 29 against 26).  Above that the wide tiles, 256 rows where they
  // give half the compute units work: 4 requests of 2048 rows, 2 heads in pairs:
  // 103 us against 121 with 128 rows, but 2 requests of 300 rows, 24 heads: 54
  // against 47.
  t.rows = t.row_slots <= 80 || slots <= 1024 ? 16 : 128;
  if (t.rows == 128 && d->requests * c->heads * ceil_div(t.row_slots, 256) * 2 >= int64_t(cus)) t.rows = 256;
  const int64_t tiles = ceil_div(t.row_slots, t.rows);
  t.items = d->requests * c->heads * tiles;
  // No request has more keys than its row of the block table holds, so that a
  // max_kv of "no bound" is cut as the table's width is.
  const __int128 room = __int128(d->table_stride) * c->page_size;
  const int64_t keys = d->max_kv < room ? d->max_kv : int64_t(room);
  // Key indexes are 32-bit in the kernels: a chunk is no longer than this, and
  // look-ups run up to 8192 keys ahead.
  if (keys > SVDQ_KV_MAX_TOKENS) return SVDQ_ERR_UNSUPPORTED;
  int64_t span = keys;
  const bool causal = (d->flags & SVDQ_ATTN_CAUSAL) != 0u;   // else a row sees up to the end, whatever its window
  if (causal && d->window > 0 && int64_t(d->window) + max_q < span) span = int64_t(d->window) + max_q;
  if (d->window > 0) span += 31;        // the first tile is rounded down to 32
  // Chunks.  Wide tiles: of at least 512 keys, two workgroups a compute unit (one
  // of 256 rows), none where that many are there.  Tiles of 16: none up to 1024
  // keys, where the second launch costs more than it saves (a request, 8 heads,
  // 512 keys: 6.7 us on the GPU and 12 a call, against 7.6 and 15 in four; 1024
  // keys: 9.5 and 12, against 8.1 and 16); above that two workgroups a compute
  // unit over chunks of at least 256, four where those still have 1024 and eight
  // where they have 2048, so that what a chunk costs beside its keys stays small
  // and long ones end together (16 requests of up to 2048, 8 heads: 15 us with 4
  // chunks, 17 with 8, 20 with 16; of 8192: 33 with 8, 36 with 16; 48 of up to
  // 16384: 129 at eight workgroups a unit, 140 at four, 138 at twelve).
  const int64_t per = t.items > 0 ? t.items : 1;
  auto fit = [&](int64_t groups) { const int64_t f = int64_t(cus) * groups / per; return f < 1 ? int64_t(1) : f; };
  auto chunks = [&](int64_t keys) {
    auto least = [&](int64_t most, int64_t n) { return most < n ? most : n < 1 ? int64_t(1) : n; };
    if (t.rows != 16) return least(fit(t.rows == 128 ? 2 : 1), ceil_div(keys, 512));
    if (keys <= 1024) return int64_t(1);
    if (keys >= 2048 * fit(8)) return fit(8);
    if (keys >= 1024 * fit(4)) return fit(4);
    return least(fit(2), ceil_div(keys, 256));
  };
  const int64_t n = chunks(span);
  const int64_t chunk = ceil_div(ceil_div(span > 0 ? span : 1, n), 128) * 128;
  t.splits = int(ceil_div(span > 0 ? span : 1, chunk));
  t.chunk = int(chunk);
  t.keys = c->n_pages == 0 ? 0 : int(keys);
  t.tokens = int(d->tokens < 0x7FFFFFFF ? d->tokens : 0x7FFFFFFF);     // offsets are 32-bit
  t.row_tiles = int(tiles);
  if (t.items * t.splits >= MAX_THREADS / 512) return SVDQ_ERR_UNSUPPORTED;   // a join has fewer: only calls of few rows are cut
  *out = t;
  return SVDQ_OK;
}

inline size_t part_bytes(const svdq_kv_cache* c, int64_t rows) { return size_t(rows) * size_t(c->head_dim + 2) * 4; }

// partial rows that a call leaves for its join
inline int64_t part_rows(const svdq_attn_desc* d, const svdq_kv_cache* c, const Cut& t) {
  return t.splits > 1 ? d->requests * c->heads * t.row_slots * t.splits : 0;
}

// Partial rows of any call with at most these requests, tokens, max_q and
// max_kv: fewer of them are cut into more chunks.  Chunks of a tile x tiles are
// at most 8 workgroups a compute unit with tiles of 16, of which a tile has
// row_slots rows at most, 2 with 128 and 1 with 256; and each row has at most
// as many chunks as there are least ones in its keys.
inline int64_t most_part_rows(const svdq_attn_desc* d, const svdq_kv_cache* c, int cus) {
  const int64_t max_q = d->max_q < d->tokens ? d->max_q : d->tokens, row_slots = max_q * (d->q_heads / c->heads);
  const int64_t slots = d->requests * c->heads * row_slots, keys = int64_t(d->max_kv) + 31;
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  const int64_t few = keys <= 1024 ? 0 : least(8 * int64_t(cus) * least(16, row_slots), slots * ceil_div(keys, 256));
  const int64_t wide = keys <= 512 || row_slots <= 80 || slots <= 1024 ? 0 : least(256 * int64_t(cus), slots * ceil_div(keys, 512));
  return few > wide ? few : wide;
}

}  // namespace svdq_kv
