/*
 * svdq_kv.h -- C ABI of the operators around a 4-bit key/value cache for AMD
 * Instinct MI355X (gfx950): what runs between a QKV projection and the
 * attention output of a transformer whose keys and values are kept in the
 * 4-bit formats of svdq.h.
 *
 *   svdq_qk_norm_rope            RMS norm of every query / key head and the
 *                                position rotation, one pass over the rows
 *   svdq_qk_norm_rope_backward   its gradient, rows and norm weights
 *   svdq_kv_plan                 block tables, slot map, positions of a step
 *                                from the requests' lengths
 *   svdq_kv_release              returns finished requests' pages
 *   svdq_kv_append               4-bit quantization of new keys and values
 *                                into the paged cache (optionally with the
 *                                norm and rotation of the keys and queries)
 *   svdq_kv_read                 cache rows as 16-bit values
 *   svdq_kv_attention            softmax attention over the paged cache
 *
 * Conventions are those of svdq.h: every call returns an svdq_status, nothing
 * throws across the ABI, arguments are checked before anything is launched,
 * the caller owns all device memory, calls are asynchronous on `stream`, and
 * every pointer is device memory unless its name ends in _host.  Results do
 * not depend on the order in which workgroups run.
 */
#ifndef SVDQ_KV_H
#define SVDQ_KV_H

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of heads: element (t, h, d) of a T x heads x D operand is
 * data[t * token_stride + h * head_stride + d], in 16-bit elements.  Strides
 * are multiples of 8 and data is 16-byte aligned; head_stride >= D where
 * heads > 1.  A fused QKV row is three such views of one buffer. */
typedef struct {
  void* data;
  int64_t token_stride, head_stride;
  int32_t heads;
} svdq_heads;

enum {
  SVDQ_QK_NORM = 1u,        /* x <- x / sqrt(mean(x^2) + eps) * w for every head */
  SVDQ_QK_ROPE = 2u,        /* rotate the pairs of every head by the position's angles */
  SVDQ_QK_ROPE_HALVES = 4u  /* with SVDQ_QK_ROPE: pairs (i, i + D/2); without: (2i, 2i + 1) */
};

/* Norm and rotation of a call.  wq, wk: 16-bit [D] in `dtype`, or NULL for
 * ones.  cos, sin: fp32 [n_positions][D / 2], 16-byte aligned; needed with
 * SVDQ_QK_ROPE only.  positions: int32 [tokens], or NULL for 0, 1, 2, ...; a
 * position outside [0, n_positions) makes its token's result NaN (nothing
 * outside the table is read). */
typedef struct {
  int64_t tokens;
  int32_t head_dim;         /* multiple of 16, 16 to 256 */
  int32_t dtype;            /* svdq_dtype */
  unsigned flags;           /* SVDQ_QK_* */
  float eps;
  const void *wq, *wk;
  const float *cos, *sin;
  int64_t n_positions;
  const int32_t* positions;
} svdq_qk_desc;

/* q_out = rot(norm(q) wq), k_out = rot(norm(k) wk).  Sums and products are
 * fp32; one rounding to 16 bits at the end.  The rotation of a pair (a, b) by
 * (c, s) is (a c - b s, a s + b c).  q_out may be q and k_out k (the same
 * data and strides); other overlaps are not allowed.  k->heads may be 0. */
svdq_status svdq_qk_norm_rope(const svdq_qk_desc* desc, const svdq_heads* q, const svdq_heads* k,
                              const svdq_heads* q_out, const svdq_heads* k_out, hipStream_t stream);

/* Gradient: from gq, gk (with respect to q_out, k_out) and the inputs q, k:
 * dq, dk, and (SVDQ_QK_NORM; else they are filled with zero) dwq, dwk, fp32
 * [D] sums over tokens and heads; either may be NULL.  With g' the gradient
 * rotated back and r = 1 / rms: u = g' w, dx = r (u - x r mean(u x r)),
 * dw = sum g' x r.  The sums run in a fixed order.  ws: >=
 * svdq_qk_backward_workspace bytes, 16-byte aligned. */
svdq_status svdq_qk_backward_workspace(const svdq_qk_desc* desc, int32_t q_heads, int32_t k_heads, size_t* bytes);
svdq_status svdq_qk_norm_rope_backward(const svdq_qk_desc* desc, const svdq_heads* q, const svdq_heads* k,
                                       const svdq_heads* gq, const svdq_heads* gk, const svdq_heads* dq,
                                       const svdq_heads* dk, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                       hipStream_t stream);

/* A paged 4-bit cache of one layer (plain data; the buffers are the
 * caller's).  Token slot s of head h is row (s / page_size, h, s % page_size):
 *   codes   uint8 [n_pages][heads][page_size][D / 2], element 2i of a row in
 *           the low nibble of byte i
 *   scales  [n_pages][heads][page_size][D / G]
 * SVDQ_FMT_MXFP4_G32: E2M1 codes, G = 32, one e8m0 byte per group.
 * SVDQ_FMT_INT4_G64: sign (bit 3) and magnitude (bits 0-2), G = 64, one fp16
 * per group.  Codes and scales follow the quantizers of svdq.h, but the e8m0
 * byte is at most 252 (2^125), so that every held value is finite in bf16.
 * Codes are 16-byte aligned, scales 16-byte aligned. */
typedef struct {
  void *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t n_pages;
  int32_t page_size;        /* 16, 32, 64, 128 or 256 */
  int32_t heads;
  int32_t head_dim;         /* 64 or 128 */
  int32_t fmt;              /* SVDQ_FMT_INT4_G64 or SVDQ_FMT_MXFP4_G32 */
} svdq_kv_cache;

/* Bytes of one code buffer and one scale buffer (K and V have one each). */
svdq_status svdq_kv_cache_size(int64_t n_pages, int32_t page_size, int32_t heads, int32_t head_dim, svdq_format fmt,
                               size_t* code_bytes, size_t* scale_bytes);

/* Quantizes k and v (desc->tokens rows of cache->heads heads) into the slots
 * slots[t] (int32; a slot outside [0, n_pages * page_size) is skipped; two
 * tokens must not name one slot).  With SVDQ_QK_NORM / SVDQ_QK_ROPE in
 * desc->flags, k is normed and rotated first, as svdq_qk_norm_rope does,
 * rounded to 16 bits, and then quantized: the cache's bytes are those of
 * svdq_qk_norm_rope followed by a plain append.  q and q_out may be NULL;
 * where they are given, the queries are normed and rotated in the same
 * launch.  A NaN is held as zero and an infinity as the largest code of the
 * largest scale. */
svdq_status svdq_kv_append(const svdq_qk_desc* desc, const svdq_heads* q, const svdq_heads* k, const svdq_heads* v,
                           const svdq_heads* q_out, const svdq_kv_cache* cache, const int32_t* slots,
                           hipStream_t stream);

/* k_out, v_out (n rows of cache->heads heads, `dtype`) = the values of slots
 * slots[0 .. n), rounded once to 16 bits; a slot outside the cache gives
 * zeros.  Either output may be NULL. */
svdq_status svdq_kv_read(const svdq_kv_cache* cache, const int32_t* slots, int64_t n, svdq_dtype dtype,
                         const svdq_heads* k_out, const svdq_heads* v_out, hipStream_t stream);

/* A step of `requests` requests: request r holds past[r] tokens and gets
 * fresh[r] more (int32 [requests], not negative).  In request order, each
 * page that the new tokens open is taken from the end of the free list: the
 * i-th page of the step is free_pages[free_count[0] - 1 - i].  Written:
 *   block_table [requests][table_stride]  entries of the opened pages (the
 *               others are kept); -1 where the free list has run out
 *   q_start [requests + 1]   prefix sums of fresh
 *   kv_len [requests]        past + fresh
 *   slots, positions [tokens] of the new tokens, request after request;
 *               slot -1 where there is no page, the table has no column or
 *               the page's slots would pass 2^31;
 *               past the sum of fresh: slot -1, position 0
 *   free_left [1]            pages left in the free list
 *   missing [1]              pages that were wanted and not there
 * No output may overlap past, fresh, free_pages or free_count (refused).
 * requests <= SVDQ_KV_MAX_REQUESTS.
 * Entries of past or fresh below zero count as zero; past[r] + fresh[r] and
 * the sum of fresh stay below 2^31. */
#define SVDQ_KV_MAX_REQUESTS 8192
svdq_status svdq_kv_plan(const int32_t* past, const int32_t* fresh, int64_t requests, int32_t page_size,
                         int64_t tokens, const int32_t* free_pages, const int32_t* free_count, int64_t free_capacity,
                         int32_t* block_table, int64_t table_stride, int32_t* q_start, int32_t* kv_len, int32_t* slots,
                         int32_t* positions, int32_t* free_left, int32_t* missing, hipStream_t stream);

#define SVDQ_KV_MAX_TOKENS ((1 << 30) - 16384)

enum {
  SVDQ_ATTN_CAUSAL = 1u     /* a query sees keys up to its own position */
};

typedef struct {
  int64_t requests;         /* >= 0 */
  int64_t tokens;           /* query rows in all */
  int32_t q_heads;          /* multiple of cache->heads: query head h reads cache head h / (q_heads / heads) */
  int32_t dtype;            /* svdq_dtype of q and out */
  int32_t max_q, max_kv;    /* bounds on a request's query rows and cached tokens; rows or
                               tokens past them are not computed or seen.  max_kv may be
                               INT32_MAX: the table's width bounds the tokens as well, and
                               the smaller of both is at most SVDQ_KV_MAX_TOKENS */
  int32_t window;           /* > 0: a query at position p sees keys above p - window; 0: all */
  unsigned flags;           /* SVDQ_ATTN_* */
  float scale;              /* of the logits, commonly 1 / sqrt(D) */
  const int32_t* q_start;   /* [requests + 1], rising */
  const int32_t* kv_len;    /* [requests], the queries' own tokens included */
  const int32_t* block_table; /* [requests][table_stride] */
  int64_t table_stride;
} svdq_attn_desc;

/* out = softmax(scale q k^T over the keys a query sees) v, request by
 * request.  Query i of request r has position kv_len[r] - (its rows) + i.
 * A row that sees no key gives zeros (and lse -infinity); a row of no request
 * is left as it was.  Keys on a page outside the cache are not seen.  lse: NULL
 * or fp32 [tokens][q_heads], the natural logarithm of the sum of exponentials.
 * Products are on the 16-bit matrix cores with fp32 accumulation, softmax
 * statistics are fp32, the probabilities (INT4: times the value scale, or, with
 * bf16 and many rows, they and the values to f16's 11 bits) are rounded to 16
 * bits for the second product.  The cached values enter the products exactly but for
 * that, MXFP4 under every scale with f16, too (prompts with scales outside 2^-20 ..
 * 2^15 take three times as long there).  Where the operands of the second product
 * are f16 (f16 over INT4; many rows: f16, and bf16 over INT4), values up to 2^16 below
 * others of the request and head, by their scales, are as precise as those; further
 * below they lose bits.
 * ws: >= svdq_kv_attention_workspace
 * bytes, 256-byte aligned (may be NULL where that is 0); its content need
 * not be kept between calls.  The size goes by requests, tokens, q_heads,
 * max_q, max_kv and the cache's shape alone, and is enough for every call with
 * as many of them or fewer (same q_heads, same shape). */
svdq_status svdq_kv_attention_workspace(const svdq_attn_desc* desc, const svdq_kv_cache* cache, size_t* bytes);
svdq_status svdq_kv_attention(const svdq_attn_desc* desc, const svdq_heads* q, const svdq_kv_cache* cache,
                              const svdq_heads* out, float* lse, void* ws, size_t ws_bytes, hipStream_t stream);

/* Gives the pages of the requests with done[r] != 0 back: the first
 * ceil(kv_len[r] / page_size) entries of their block-table rows that are not
 * -1 are appended to free_pages (request order, page order) from
 * free_count[0] on, the entries are set to -1, kv_len[r] to 0, and
 * free_count[0] is raised.  Pages that would pass free_capacity are
 * dropped. */
svdq_status svdq_kv_release(const int32_t* done, int64_t requests, int32_t page_size, int32_t* block_table,
                            int64_t table_stride, int32_t* kv_len, int32_t* free_pages, int32_t* free_count,
                            int64_t free_capacity, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SVDQ_KV_H */
