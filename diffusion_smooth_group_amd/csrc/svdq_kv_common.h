// svdq_kv_common.h -- what the two kernel files of the 4-bit cache share:
// 16-bit conversions, vector types and the argument checks of include/svdq_kv.h.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "svdq_kv.h"
#include "svdq_kv_cut.h"

namespace svdq_kv {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int DT>
__device__ __forceinline__ float h2f(unsigned v) {
  if constexpr (DT == SVDQ_BF16) return __uint_as_float(v << 16);
  else return float(__builtin_bit_cast(_Float16, (unsigned short)v));
}

// two floats -> two 16-bit values (round to nearest even), low half first
template <int DT>
__device__ __forceinline__ unsigned pack2(float a, float b) {
  if constexpr (DT == SVDQ_BF16) return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(unsigned, f16x2{(_Float16)a, (_Float16)b});
}

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool dtype_ok(int dt) { return dt == SVDQ_F16 || dt == SVDQ_BF16; }
inline svdq_status launch_ok() { return hipGetLastError() == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP; }

// log2 of a page size the cache takes, -1 otherwise
inline int page_shift(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    case 256: return 8;
    default: return -1;
  }
}

inline svdq_status check_heads(const svdq_heads* v, int D) {
  if (!v || !v->data || v->heads < 1) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(v->data, 16) || v->token_stride % 8 != 0 || v->head_stride % 8 != 0 || v->token_stride < 0) return SVDQ_ERR_SHAPE;
  if (v->heads > 1 && v->head_stride < D) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

inline svdq_status check_cache_shape(const svdq_kv_cache* c) {
  if (!c || c->n_pages < 0 || c->heads < 1) return SVDQ_ERR_INVALID_ARG;
  if (c->fmt != SVDQ_FMT_INT4_G64 && c->fmt != SVDQ_FMT_MXFP4_G32)
    return c->fmt == SVDQ_FMT_INT8_W8A8 ? SVDQ_ERR_UNSUPPORTED : SVDQ_ERR_INVALID_ARG;
  if (page_shift(c->page_size) < 0 || (c->head_dim != 64 && c->head_dim != 128)) return SVDQ_ERR_SHAPE;
  // slots are int32
  if (c->n_pages >= (int64_t(1) << 31) || c->n_pages * c->page_size >= (int64_t(1) << 31)) return SVDQ_ERR_UNSUPPORTED;
  return SVDQ_OK;
}

inline svdq_status check_cache(const svdq_kv_cache* c) {
  const svdq_status st = check_cache_shape(c);
  if (st != SVDQ_OK) return st;
  if (c->n_pages == 0) return SVDQ_OK;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return SVDQ_ERR_INVALID_ARG;
  for (const void* p : {(const void*)c->k_codes, (const void*)c->k_scales, (const void*)c->v_codes, (const void*)c->v_scales})
    if (!aligned(p, 16)) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

}  // namespace svdq_kv
