/*
 * svdq_image.h -- C ABI of the operators that run between the 4-bit linears of
 * an image model's conditioned blocks on AMD Instinct MI355X (gfx950):
 *
 *   svdq_group_norm                 group norm of a channels-last map with an
 *                                   activation
 *   svdq_group_norm_backward        its gradient: map, weight and bias
 *   svdq_cross_attention            softmax attention of one sequence's queries
 *                                   to an encoder's 16-bit keys and values
 *   svdq_cross_attention_backward   its gradient: queries, keys and values
 *
 * Conventions are those of svdq.h and svdq_kv.h: every call returns an
 * svdq_status, nothing throws across the ABI, arguments are checked before
 * anything is launched, the caller owns all device memory, calls are
 * asynchronous on `stream`, every pointer of a call is device memory.  Results
 * do not depend on the order in which workgroups run.  Unless stated, no output
 * may overlap an input or another output.  A workspace's content need not be
 * kept between calls; two calls that may run at once need two.
 */
#ifndef SVDQ_IMAGE_H
#define SVDQ_IMAGE_H

#include "svdq_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A channels-last map: element (n, p, c) is data[n * sample_stride + p *
 * pixel_stride + c], in 16-bit elements.  Strides are multiples of 8, data is
 * 16-byte aligned, pixel_stride >= channels where pixels > 1. */
typedef struct {
  void* data;
  int64_t sample_stride, pixel_stride;
} svdq_map;

enum {
  SVDQ_ACT_NONE = 0,
  SVDQ_ACT_SILU = 1,        /* z / (1 + exp(-z)) */
  SVDQ_ACT_GELU = 2         /* z Phi(z), the erf form */
};

typedef struct {
  int64_t samples, pixels;  /* pixels: height x width, at least 1 where samples > 0.  A launch has
                               fewer than 2^32 threads: more samples than that takes, 2^22 /
                               groups at least, are SVDQ_ERR_UNSUPPORTED */
  int32_t channels;         /* multiple of 8 and of groups, at most SVDQ_NORM_MAX_CHANNELS */
  int32_t groups;
  int32_t dtype;            /* svdq_dtype of maps, weight and bias */
  int32_t act;              /* SVDQ_ACT_* */
  float eps;
  const void *weight, *bias;  /* [channels], 16-byte aligned, or NULL for ones and zeros */
} svdq_norm_desc;
#define SVDQ_NORM_MAX_CHANNELS 8192

/* y = act((x - mean) rstd w + b), mean and rstd = 1 / sqrt(var + eps) over the
 * pixels and the channels / groups channels of a group, sample by sample (var
 * is the mean square deviation).  Statistics are fp32, of deviations
 * from the mean or from a mean of a part of the data, so that neither a mean far
 * from zero nor values far from the rest cost digits; one rounding to 16 bits at
 * the end.  y may be x (the same data and strides).
 * stats: NULL or fp32 [samples][groups][2], mean and rstd.
 * ws: >= svdq_group_norm_workspace bytes, 16-byte aligned (may be NULL where
 * that is 0). */
svdq_status svdq_group_norm_workspace(const svdq_norm_desc* desc, size_t* bytes);
svdq_status svdq_group_norm(const svdq_norm_desc* desc, const svdq_map* x, const svdq_map* y, float* stats, void* ws,
                            size_t ws_bytes, hipStream_t stream);

/* Gradient from g (with respect to y), x and the forward call's stats.  With
 * xh = (x - mean) rstd, z = xh w + b, dz = g act'(z), u = dz w:
 *   dx = rstd (u - mean(u) - xh mean(u xh)), dw = sum dz xh, db = sum dz
 * dx may be g or x (the same data and strides).  dw, db: fp32 [channels];
 * either may be NULL.  Sums run in a fixed order.  samples = 0: dw, db are
 * filled with zero. */
svdq_status svdq_group_norm_backward_workspace(const svdq_norm_desc* desc, size_t* bytes);
svdq_status svdq_group_norm_backward(const svdq_norm_desc* desc, const svdq_map* x, const svdq_map* g,
                                     const float* stats, const svdq_map* dx, float* dw, float* db, void* ws,
                                     size_t ws_bytes, hipStream_t stream);

/* Which rows and encoder states belong together.  Rows of heads are svdq_heads
 * (svdq_kv.h); k and v have as many heads, which divides the number of q's:
 * query head h reads head h / (q_heads / k_heads).  Token strides are below
 * 2^23 elements, and the heads of a group lie within 2^28. */
typedef struct {
  int64_t requests;
  int64_t tokens, states;   /* query rows and encoder states in all, below 2^31 */
  int32_t head_dim;         /* multiple of 8, 8 to 128 */
  int32_t dtype;            /* svdq_dtype of all operands */
  int32_t max_q, max_k;     /* bounds on a request's rows and states; what is past them is
                               not computed or seen.  requests x q_heads x max_q is below 2^30,
                               max_k at most 2^30 (both no more than tokens and states) */
  float scale;              /* of the logits, commonly 1 / sqrt(D); finite */
  const int32_t *q_start;   /* [requests + 1], rising: request r has rows q_start[r] .. q_start[r + 1];
                               NULL: max_q rows each, tokens = requests max_q */
  const int32_t *k_start;   /* the same of its states; NULL: max_k each, states = requests max_k */
  const uint8_t *mask;      /* [states], 0: the state is not seen; or NULL */
} svdq_cross_desc;

/* out = softmax(scale q k^T over the states that are seen) v, request by
 * request.  A row that sees nothing gives zeros (and lse -infinity); what keys
 * and values hold where the mask is 0 does not matter, NaN included.  A row of
 * no request is left as it was.  lse: NULL or fp32 [tokens][q_heads], the
 * natural logarithm of the sum of exponentials.  Products are on the 16-bit
 * matrix cores with fp32 accumulation, statistics are fp32, the probabilities
 * are rounded to 16 bits for the second product.
 * ws: >= svdq_cross_attention_workspace bytes for the same sizes, 256-byte
 * aligned (may be NULL where that is 0). */
svdq_status svdq_cross_attention_workspace(const svdq_cross_desc* desc, int32_t q_heads, int32_t k_heads, size_t* bytes);
svdq_status svdq_cross_attention(const svdq_cross_desc* desc, const svdq_heads* q, const svdq_heads* k, const svdq_heads* v,
                                 const svdq_heads* out, float* lse, void* ws, size_t ws_bytes, hipStream_t stream);

/* Gradient from g (with respect to out), the inputs, and out and lse of the
 * forward call.  With p = exp(scale q k^T - lse), delta = g . out:
 *   dv = sum p g, ds = p (g . v - delta), dq = scale sum ds k, dk = scale sum ds q
 * (dk, dv: over rows and the query heads of a key head).  Where min(max_k, states)
 * is 128 or less, delta = sum p (g . v) instead, which is the same for the forward
 * call's out, and out is not read; above that the rounding of out enters delta,
 * which counts against dq the more the more states share a row's weight (bf16,
 * relative to 64 bits: 2.4e-3 up to some thousand states, 2.9e-3 over 7346 of
 * random logits, where the result's own rounding is 1.7e-3).  States that the mask
 * hides get zeros, rows and states of no request or past the bounds are left
 * as they were.  The probabilities and ds are rounded to 16 bits for their
 * products (f16: ds under a power of two of its row's or state's own, so that
 * small and large gradients keep their digits).  Sums run in a fixed order. */
svdq_status svdq_cross_attention_backward_workspace(const svdq_cross_desc* desc, int32_t q_heads, int32_t k_heads,
                                                    size_t* bytes);
svdq_status svdq_cross_attention_backward(const svdq_cross_desc* desc, const svdq_heads* q, const svdq_heads* k,
                                          const svdq_heads* v, const svdq_heads* out, const float* lse,
                                          const svdq_heads* g, const svdq_heads* dq, const svdq_heads* dk,
                                          const svdq_heads* dv, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SVDQ_IMAGE_H */
