// svdq_kv_attn.hip -- gfx950 (MI355X) attention over the paged 4-bit cache
// (include/svdq_kv.h).
//
//   out_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t - m_i)
//
// over the keys t that row i sees.  One pass over the keys with a running
// reference m and sum; the cached codes are turned into matrix-core operands
// in registers, and no 16-bit copy of the cache is ever written.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "svdq_kv_common.h"

namespace {

using namespace svdq_kv;

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part;              // [row slot][split][D] partial sums, then [row slot][split][2] reference and sum
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t *q_start, *kv_len, *table;
  int64_t qt, qh, ot, oh, table_stride, n_pages;
  int32_t tokens, requests, q_heads, heads, group;      // group = q_heads / heads
  int32_t max_q, max_kv, window, causal, page_shift;
  int32_t row_tiles, row_slots, splits, chunk;  // row tiles and rows a request and head has at most; key chunks
  float c;                  // scale log2(e)
};

constexpr float LOWEST = -3.0e38f;   // reference of a row that has seen no key

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two E2M1 codes of byte B of w, times 2^(e - 127) with e in bits 23-30 of
// `scale`, as two 16-bit values (both products are exact).
template <int DT, int B>
__device__ __forceinline__ unsigned cvt_mx(unsigned w, float scale) {
  if constexpr (DT == SVDQ_BF16) return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
  else return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, B));
}

// INT4 codes are sign and magnitude: moved to the sign and the low mantissa
// bits of an fp8 (e4m3) byte they are its subnormals, magnitude x 2^-9, so the
// fp8 converters under the scale 2^9 turn them into exact small integers.
// even: nibbles 0, 2, 4, 6 in bytes 0 .. 3; odd: nibbles 1, 3, 5, 7.
__device__ __forceinline__ unsigned int4_even(unsigned w) { return (w & 0x07070707u) | ((w << 4) & 0x80808080u); }
__device__ __forceinline__ unsigned int4_odd(unsigned w) { return ((w >> 4) & 0x07070707u) | (w & 0x80808080u); }
template <int DT, bool HI>
__device__ __forceinline__ unsigned cvt_int4(unsigned fp8) {   // bytes 0, 1 (or 2, 3) as 16-bit integers
  if constexpr (DT == SVDQ_BF16) return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(fp8, 512.0f, HI));
  else return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(fp8, 512.0f, HI));
}

// e8m0 byte in bits 23-30, ready as the converters' scale.  f16 has 40 binades,
// the cache's scales 254.  Few rows: Rows16 has bf16 operands for f16, too.  Many
// rows: values are held at 2^-3 of their size, which is exact for the scales
// 2^-20 .. 2^15, and the missing 2^3 is put back on the fp32 sums; a workgroup
// that meets other scales (`off_scale`; a group of zeros has any) does its rows
// again as Rows16 does.
__device__ __forceinline__ unsigned f16_scale(unsigned e) { return min(max(e, 107u), 142u); }
__device__ __forceinline__ unsigned off_scale(unsigned e) { return e ^ f16_scale(e); }   // 0: one that f16 takes
template <int DT>
__device__ __forceinline__ float mx_scale(unsigned e) {
  if constexpr (DT == SVDQ_F16) e = f16_scale(e) - 3u;
  return __uint_as_float(e << 23);
}
template <int DT, int FMT>
constexpr bool checks_scales() { return DT == SVDQ_F16 && FMT == SVDQ_FMT_MXFP4_G32; }
template <int DT, int FMT>
constexpr float value_gain() { return DT == SVDQ_F16 && FMT == SVDQ_FMT_MXFP4_G32 ? 8.0f : 1.0f; }

// A row's reference is raised only when its maximum has passed it by 2^SLACK;
// between that no accumulator is touched.  f16: probabilities are held at 2^6
// of their size, so that f16's subnormals start far below any that counts, and
// 2^(6 + 8) still fits.  INT4 with f16: what is rounded is p times a value
// scale, so the reference is raised to the maximum of logit + exponent of the
// tile's largest value scale.  All of this is part of the reference and drops
// out of the quotient.
template <int DT>
constexpr float p_shift() { return DT == SVDQ_F16 ? 6.0f : 0.0f; }
constexpr float SLACK = 8.0f;
template <int DT, int FMT>
constexpr bool scaled_reference() { return DT == SVDQ_F16 && FMT == SVDQ_FMT_INT4_G64; }
// exponent of a value scale as f16 has it (2^e <= s), -24 for zero
__device__ __forceinline__ float scale_exponent(float s) {
  return s == 0.0f ? -24.0f : float(int(__float_as_uint(s) >> 23) - 127);
}

// NaN if either is one: one instruction for three, where fmaxf has to quiet its
// operands first.  A row with a NaN gives NaN by its probabilities.
__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// max / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 of a column
__device__ __forceinline__ float quad_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = maximum(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const unsigned v = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return maximum(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const unsigned v = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// natural logarithm of a row's sum of exponentials
__device__ __forceinline__ float row_lse(float base, float sum) {
  return sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0.69314718055994531f;
}

// ----------------------------------------------------- 16 rows and one wave
// S^T = K Q^T on 16x16x32: keys are rows of the result, query rows its
// columns, so that a lane holds the probabilities of one query row for the
// keys [8b, 8b + 8) of a 32-key tile (b = lane / 16) -- which is the operand of
// O^T = V^T P^T as it stands; the keys of the two K tiles are dealt out for
// that (tile a, row r: key 8 (r / 4) + 4 a + r % 4).  V^T needs 8 keys of one
// column in a lane: a lane loads 8 keys' codes of its own columns and pairs
// neighbouring keys, MXFP4 after the conversion (each key has its own scale),
// INT4 before it.  The cache's bytes bound it (136 a key and head of 128): the
// codes go from memory to registers and are turned there, with two tiles in
// flight a wave and three waves a SIMD (four with D = 64).  Times are those of
// the call, the join of its chunks (5 us) included.  48 requests of up to 16384
// tokens, 8 heads of 128, 4 query heads each: MXFP4 117 us, 4.6 TB/s (f16 130:
// Rows16), INT4 133 us (f16 139), where the vector unit is the bound: bits to fp8,
// conversion, and scales on both sums.  20 heads of 64 with a query head each:
// MXFP4 197 us (f16 223), INT4 207, 3.4 and 3.3 TB/s, the vector unit again (as
// many instructions for half the bytes a key).  Measured while it was built, each
// against the form before it: INT4 with the converted values paired instead of
// their codes, 190 registers and two waves, 180 us against 133; two row tiles a
// wave on the same operands, MXFP4, 40 rows, two waves, 309 against 199 with three
// tiles of 16.
template <int FMT, int D>
struct Tile32 {
  static constexpr int NJ = D / 32;
  static constexpr int NS = D / 64;         // 8 keys' scales are 16 bytes a 64 elements in either format
  unsigned k[2][NJ];        // codes of the lane's key row in each K tile
  unsigned ke[2];           // MXFP4: e8m0 of the lane's key rows and group
  u32x4 ksc[NS];            // INT4: fp16 scales of the keys [8b, 8b + 8)
  unsigned v[8];            // codes of the lane's columns, keys [8b, 8b + 8)
  u32x4 vsc[NS];            // scales of these keys
  bool ok0, ok1;            // the pages of the tile's halves are there

  // page0, page1: the pages of the tile's two halves, the same for all lanes.
  // Where a page holds the whole tile every address is a scalar base plus the
  // lane's fixed offset; pages of 16 give the lanes of either half their own.
  __device__ __forceinline__ void load(const AttnParams& p, int token, int page0, int page1, int h, int lane) {
    ok0 = page0 >= 0 && page0 < p.n_pages;
    ok1 = page1 >= 0 && page1 < p.n_pages;
    const int64_t row0 = ((int64_t(ok0 ? page0 : 0) * p.heads + h) << p.page_shift) + (token & ((1 << p.page_shift) - 1));
    if (p.page_shift > 4) {
      load_rows(p, row0, 0, lane);
    } else {
      const int64_t row1 = (int64_t(ok1 ? page1 : 0) * p.heads + h) << 4;
      load_rows(p, row0, row1 - 16 - row0, lane);
    }
  }
  // shift: distance of the second half's rows from where they would follow
  __device__ __forceinline__ void load_rows(const AttnParams& p, int64_t row0, int64_t shift, int lane) {
    const int m = lane & 15, b = lane >> 4;
    constexpr int SB = D / 32;                  // scale bytes of a row
    const uint8_t *kc = p.kc + row0 * (D / 2), *ks = p.ks + row0 * SB, *vc = p.vc + row0 * (D / 2), *vs = p.vs + row0 * SB;
    const int64_t kshift = m >= 8 ? shift : 0, vshift = b >= 2 ? shift : 0;
    const uint8_t *kc1 = kc + kshift * (D / 2), *ks1 = ks + kshift * SB, *vc1 = vc + vshift * (D / 2), *vs1 = vs + vshift * SB;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const unsigned lt = unsigned(8 * (m >> 2) + 4 * a + (m & 3));
      if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
        if constexpr (D == 128) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(kc1 + (lt * 64u + 16u * b));
          k[a][0] = w[0]; k[a][1] = w[1]; k[a][2] = w[2]; k[a][3] = w[3];
          ke[a] = ks1[lt * 4u + b];
        } else {
          const u32x2 w = *reinterpret_cast<const u32x2*>(kc1 + (lt * 32u + 8u * b));
          k[a][0] = w[0]; k[a][1] = w[1];
          ke[a] = ks1[lt * 2u + (b >> 1)];
        }
      } else {
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(kc1 + (lt * unsigned(D / 2) + 32u * g + 8u * b));
          k[a][2 * g] = w[0];
          k[a][2 * g + 1] = w[1];
        }
      }
    }
    const unsigned vo = unsigned(8 * b * (D / 2) + D / 32 * m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (D == 128) v[i] = *reinterpret_cast<const unsigned*>(vc1 + (vo + unsigned(i * (D / 2))));
      else v[i] = *reinterpret_cast<const uint16_t*>(vc1 + (vo + unsigned(i * (D / 2))));
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) vsc[i] = *reinterpret_cast<const u32x4*>(vs1 + (8u * b * SB + 16u * i));
    if constexpr (FMT == SVDQ_FMT_INT4_G64) {
      // the lane's rows of S^T are the keys of its V block
      const uint8_t* kss = ks + vshift * SB;
#pragma unroll
      for (int i = 0; i < NS; ++i) ksc[i] = *reinterpret_cast<const u32x4*>(kss + (8u * b * SB + 16u * i));
    }
  }
};

// element offset of the 8 elements that fragment j of a key row covers in lane block b
template <int FMT, int D>
__device__ __forceinline__ int frag_dim(int j, int b) {
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) return (D / 4) * b + 8 * j;
  else return 64 * (j >> 1) + 16 * b + 8 * (j & 1);
}

template <int DT, int FMT>
__device__ __forceinline__ u32x4 key_frag(unsigned w, float scale) {
  u32x4 f;
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
    f[0] = cvt_mx<DT, 0>(w, scale);
    f[1] = cvt_mx<DT, 1>(w, scale);
    f[2] = cvt_mx<DT, 2>(w, scale);
    f[3] = cvt_mx<DT, 3>(w, scale);
  } else {
    const unsigned e = int4_even(w), o = int4_odd(w);   // elements 0 2, 4 6, 1 3, 5 7: the query fragments follow
    f[0] = cvt_int4<DT, false>(e);
    f[1] = cvt_int4<DT, true>(e);
    f[2] = cvt_int4<DT, false>(o);
    f[3] = cvt_int4<DT, true>(o);
  }
  return f;
}

__device__ __forceinline__ unsigned low_halves(unsigned x0, unsigned x1) { return __builtin_amdgcn_perm(x1, x0, 0x05040100u); }
__device__ __forceinline__ unsigned high_halves(unsigned x0, unsigned x1) { return __builtin_amdgcn_perm(x1, x0, 0x07060302u); }

// (by value: a bit cast of a vector's element in place reads element 0)
__device__ __forceinline__ f16x2 two_halves(unsigned u) { return __builtin_bit_cast(f16x2, u); }

// a * (half H of h) + c in one mixed-precision instruction.  With c a zero that
// the compiler does not know for one, the plain product takes one too (a
// constant zero is folded into a conversion and a product).
template <int H>
__device__ __forceinline__ float fma_half(float a, unsigned h, float c) { return __builtin_fmaf(a, float(two_halves(h)[H]), c); }
__device__ __forceinline__ float hidden_zero() {
  float z = 0.0f;
  asm("" : "+v"(z));
  return z;
}

template <int FMT>
__device__ __forceinline__ u32x4 query_order(u32x4 q) {
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) return q;
  return u32x4{low_halves(q[0], q[1]), low_halves(q[2], q[3]), high_halves(q[0], q[1]), high_halves(q[2], q[3])};
}

// MXFP4: exponent and converter scale of key i and group g
template <int D>
__device__ __forceinline__ unsigned value_exponent(const u32x4* sc, int i, int g) {
  const unsigned w = D == 128 ? sc[i / 4][i % 4] : sc[0][i / 2];
  return (w >> (D == 128 ? 8 * g : 16 * (i % 2) + 8 * g)) & 255u;
}
template <int DT, int D>
__device__ __forceinline__ float value_scale(const u32x4* sc, int i, int g) {
  const unsigned w = D == 128 ? sc[i / 4][i % 4] : sc[0][i / 2];
  const unsigned b = D == 128 ? 8 * g : 16 * (i % 2) + 8 * g;         // bit of the byte
  if constexpr (DT == SVDQ_F16) return mx_scale<DT>(value_exponent<D>(sc, i, g));
  return __uint_as_float(__builtin_amdgcn_alignbit(w, w, b + 9u) & 0x7F800000u);   // rotated to bits 23-30
}

// two value fragments (columns x and x + 1 of the pair) of 8 keys, MXFP4
template <int DT, int B>
__device__ __forceinline__ void value_pair_mx(const unsigned* v, const float* s, u32x4* f0, u32x4* f1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned x0 = cvt_mx<DT, B>(v[2 * i], s[2 * i]), x1 = cvt_mx<DT, B>(v[2 * i + 1], s[2 * i + 1]);
    (*f0)[i] = low_halves(x0, x1);
    (*f1)[i] = high_halves(x0, x1);
  }
}

// INT4: the codes of four keys are dealt out by columns before they are
// converted, half as many byte moves as for the converted values.  y[j]: bytes
// first + j of v[0] .. v[3] (j = 0, 1); `pick` has the bytes of two words.
__device__ __forceinline__ unsigned byte_pick(int first) { return first == 0 ? 0x05010400u : 0x07030602u; }
__device__ __forceinline__ void deal(const unsigned* v, unsigned pick, unsigned* y) {
  const unsigned a = __builtin_amdgcn_perm(v[1], v[0], pick), b = __builtin_amdgcn_perm(v[3], v[2], pick);
  y[0] = low_halves(a, b);
  y[1] = high_halves(a, b);
}
// one column's value fragment from its fp8 words of the keys 0 .. 3 and 4 .. 7
template <int DT>
__device__ __forceinline__ u32x4 value_int4(unsigned keys0, unsigned keys4) {
  return u32x4{cvt_int4<DT, false>(keys0), cvt_int4<DT, true>(keys0), cvt_int4<DT, false>(keys4), cvt_int4<DT, true>(keys4)};
}
// The same times the keys' scales (pairs), as f16 rounded once; `gain` is 512
// for the values themselves.
__device__ __forceinline__ u32x4 value_int4_scaled(unsigned keys0, unsigned keys4, const unsigned* scale, float gain) {
  const u32x4 f = {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(keys0, gain, false)),
                   __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(keys0, gain, true)),
                   __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(keys4, gain, false)),
                   __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(keys4, gain, true))};
  u32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __builtin_bit_cast(unsigned, two_halves(f[i]) * two_halves(scale[i]));
  return y;
}
// scale of key i and group g in the words of 8 keys, and a times it (see fma_half)
template <int D>
__device__ __forceinline__ float fma_scale(float a, const u32x4* sc, int i, int g, float c) {
  const unsigned w = D == 128 ? sc[i / 4][i % 4] : sc[0][i / 2];
  return __builtin_fmaf(a, float(two_halves(w)[D == 128 ? g : i % 2]), c);
}
// largest of 8 keys' scales
template <int D>
__device__ __forceinline__ float most_scale(const u32x4* sc) {
  f16x2 most = two_halves(sc[0][0]);
#pragma unroll
  for (int i = 1; i < D / 16; ++i) most = __builtin_elementwise_max(most, two_halves(sc[i / 4][i % 4]));
  return fmaxf(float(most[0]), float(most[1]));
}

// column of the result that lane row n of value tile x stands for.  MXFP4:
// the lane's elements in order.  INT4: tile x holds one scale group's columns
// only (D = 128: tiles 0-3 the first, 4-7 the second), the nibbles of the 16
// bits of the group that Rows16::step gives the lane in order.
template <int FMT, int D>
__device__ __forceinline__ constexpr int value_col(int n, int x) {
  constexpr int PER = D / 16;
  if (FMT == SVDQ_FMT_MXFP4_G32) return PER * n + x;
  if (D == 64) return 4 * n + x;
  return 64 * (x / 4) + 8 * (n & 7) + 4 * (n >> 3) + x % 4;
}

// 16-bit values as two bf16 ones whose sum they are: 8 bits, and the other three
// of an f16's eleven.
__device__ __forceinline__ void split_f16(u32x4 x, u32x4* hi, u32x4* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = h2f<SVDQ_F16>(x[i] & 0xFFFFu), b = h2f<SVDQ_F16>(x[i] >> 16);
    const unsigned w = pack2<SVDQ_BF16>(a, b);
    (*hi)[i] = w;
    (*lo)[i] = pack2<SVDQ_BF16>(a - h2f<SVDQ_BF16>(w & 0xFFFFu), b - __uint_as_float(w & 0xFFFF0000u));
  }
}

template <int DT, int FMT, int D>
struct Rows16 {
  static constexpr int NJ = D / 32, NX = D / 16;
  // f16 over MXFP4: f16 does not hold all scales of the cache, bf16 does.  The
  // operands are bf16, of q (exactly) and of the probabilities (to 16 bits) two
  // each.  48 requests of up to 16384 tokens, 8 heads of 128: 130 us, where f16
  // operands and scales outside 2^-20 .. 2^15 wrong took 118, and a look at every
  // scale with a second way for such tiles 131; 20 heads of 64: 223, 201, 266.
  static constexpr bool TWO = DT == SVDQ_F16 && FMT == SVDQ_FMT_MXFP4_G32;
  static constexpr int OT = TWO ? SVDQ_BF16 : DT;   // type of the operands
  static constexpr int LOW = TWO ? NJ * 64 : 1;     // a wave's second terms of q, in LDS
  u32x4 q[NJ];
  const u32x4* low_q;
  f32x4 o[NX];
  float base, sum;          // reference and this lane's part of the sum
  int low, high;            // keys that this lane's row sees

  // row: this lane's query row.  negate: the sign of the scale goes to the query,
  // so that the largest product is the largest logit.
  // wave_low: LOW pieces of LDS of the wave's own.
  __device__ __forceinline__ void start(const uint16_t* row, bool negate, int lane, u32x4* wave_low) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) q[j] = query_order<FMT>(*reinterpret_cast<const u32x4*>(row + frag_dim<FMT, D>(j, lane >> 4)));
    if (negate) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) q[j] ^= 0x80008000u;
    }
    if constexpr (TWO) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        u32x4 lo;
        split_f16(q[j], &q[j], &lo);
        wave_low[64 * j + lane] = lo;
      }
    }
    low_q = wave_low;
#pragma unroll
    for (int x = 0; x < NX; ++x) o[x] = f32x4{0, 0, 0, 0};
    base = LOWEST;
    sum = 0.0f;
  }

  // all: every row sees every key of the tile and both pages are there; c > 0
  __device__ __forceinline__ void step(const Tile32<FMT, D>& t, int token, int len, bool all, float c, int lane) {
    const int b = lane >> 4;
    const float zero = hidden_zero();
    int low_at = lane;
    if constexpr (TWO) asm volatile("" : "+v"(low_at));     // read here, not kept in registers from tile to tile
    f32x4 s[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      f32x4 acc = {0, 0, 0, 0};
      if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
        const float e = mx_scale<OT>(t.ke[a]);
        f32x4 more = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const u32x4 f = key_frag<OT, FMT>(t.k[a][j], e);
          acc = mfma16<OT>(f, q[j], acc);
          if constexpr (TWO) more = mfma16<OT>(f, low_q[64 * j + low_at], more);
        }
        s[a] = TWO ? acc + more : acc;
      } else {
        acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][0], 0.0f), q[0], acc);
        acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][1], 0.0f), q[1], acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[a][i] = fma_scale<D>(acc[i], t.ksc, 4 * a + i, 0, zero);
        if constexpr (D == 128) {
          acc = f32x4{0, 0, 0, 0};
          acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][2], 0.0f), q[2], acc);
          acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][3], 0.0f), q[3], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[a][i] = fma_scale<D>(acc[i], t.ksc, 4 * a + i, 1, s[a][i]);
        }
      }
    }
    const bool there = b >= 2 ? t.ok1 : t.ok0;
    const int last = there ? len - (token + 8 * b) : 0;       // keys from here on are not there: they may hold a NaN
    u32x4 vsc[Tile32<FMT, D>::NS];
#pragma unroll
    for (int i = 0; i < Tile32<FMT, D>::NS; ++i) vsc[i] = t.vsc[i];
    if (!all) {
      const unsigned first = unsigned(token + 8 * b - low), wide = there ? unsigned(max(high - low, 0)) : 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i / 4][i % 4] = first + unsigned(i) < wide ? s[i / 4][i % 4] : -__builtin_inff();
      if constexpr (FMT == SVDQ_FMT_INT4_G64) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (D == 128) vsc[i / 4][i % 4] = i < last ? vsc[i / 4][i % 4] : 0u;
          else vsc[0][i / 2] = i < last ? vsc[0][i / 2] : vsc[0][i / 2] & (i % 2 ? 0x0000FFFFu : 0xFFFF0000u);
        }
      }
    }
    const int m = lane & 15;
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = maximum(top, s[i / 4][i % 4]);
    top *= c;
    if constexpr (scaled_reference<DT, FMT>()) top += scale_exponent(most_scale<D>(vsc));
    top = quad_max(top) - p_shift<OT>();
    if (__any(top > base + SLACK)) {
      const float next = fmaxf(base, top), alpha = exp2_hw(base - next);
      base = next;
      sum *= alpha;
#pragma unroll
      for (int x = 0; x < NX; ++x) o[x] *= alpha;
    }
    if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
      // bf16: the probabilities are rounded to 8 bits, as usual for attention in
      // bf16: relative error 2.1e-3, of which the result's own rounding is 1.7e-3.
      // A second term for the rest leaves 1.7e-3 and costs 123 us instead of 118
      // (heads of 64: 211, 197).
      u32x4 pf, pl = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = exp2_hw(__builtin_fmaf(s[i / 2][2 * i % 4], c, -base)), p1 = exp2_hw(__builtin_fmaf(s[i / 2][2 * i % 4 + 1], c, -base));
        sum += p0 + p1;
        pf[i] = pack2<OT>(p0, p1);
        if constexpr (TWO) pl[i] = pack2<OT>(p0 - h2f<OT>(pf[i] & 0xFFFFu), p1 - __uint_as_float(pf[i] & 0xFFFF0000u));
      }
      // keys past the end or on a missing page hold anything, a NaN included:
      // their values must be zero, not only weighted with zero
      float sc[8];
      const int g = D == 128 ? m >> 2 : m >> 3;
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] = value_scale<OT, D>(t.vsc, i, g);
      if (!all) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = i < last ? sc[i] : 0.0f;
      }
      auto add = [&](int x, u32x4 f0, u32x4 f1) {
        o[x] = mfma16<OT>(f0, pf, o[x]);
        o[x + 1] = mfma16<OT>(f1, pf, o[x + 1]);
        if constexpr (TWO) {
          o[x] = mfma16<OT>(f0, pl, o[x]);
          o[x + 1] = mfma16<OT>(f1, pl, o[x + 1]);
        }
      };
      u32x4 f0, f1;
      value_pair_mx<OT, 0>(t.v, sc, &f0, &f1);
      add(0, f0, f1);
      value_pair_mx<OT, 1>(t.v, sc, &f0, &f1);
      add(2, f0, f1);
      if constexpr (D == 128) {
        value_pair_mx<OT, 2>(t.v, sc, &f0, &f1);
        add(4, f0, f1);
        value_pair_mx<OT, 3>(t.v, sc, &f0, &f1);
        add(6, f0, f1);
      }
    } else {
      // The value scales are on the probabilities, one operand per scale
      // group: the integers are exact, and p s is rounded where p was.
      float pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = exp2_hw(__builtin_fmaf(s[i / 4][i % 4], c, -base));
#pragma unroll
      for (int i = 0; i < 8; i += 2) sum += pr[i] + pr[i + 1];
      u32x4 pf[D / 64];
#pragma unroll
      for (int g = 0; g < D / 64; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pf[g][i] = pack2<DT>(fma_scale<D>(pr[2 * i], vsc, 2 * i, g, zero), fma_scale<D>(pr[2 * i + 1], vsc, 2 * i + 1, g, zero));
      // D = 128: lanes n and n + 8 hold eight columns of either group: each
      // takes four of both.  `own` are a lane's own columns of its group,
      // `other` the four that go to the lane across.
      constexpr int NG = D / 64;
      unsigned cols[NG][2][2];            // [group][keys 0 .. 3, 4 .. 7][byte]
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (D == 128) {
          unsigned own[2], other[2];
          deal(t.v + 4 * k, m < 8 ? byte_pick(0) : byte_pick(2), own);
          deal(t.v + 4 * k, m < 8 ? byte_pick(2) : byte_pick(0), other);
#pragma unroll
          for (int j = 0; j < 2; ++j) {   // row_ror:8 into the upper eight lanes, and into the lower ones
            cols[0][k][j] = unsigned(__builtin_amdgcn_update_dpp(int(own[j]), int(other[j]), 0x128, 0xF, 0xC, false));
            cols[NG - 1][k][j] = unsigned(__builtin_amdgcn_update_dpp(int(own[j]), int(other[j]), 0x128, 0xF, 0x3, false));
          }
        } else {
          deal(t.v + 4 * k, byte_pick(0), cols[0][k]);
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const unsigned w0 = cols[g][0][j], w4 = cols[g][1][j];
          o[4 * g + 2 * j] = mfma16<DT>(value_int4<DT>(int4_even(w0), int4_even(w4)), pf[g], o[4 * g + 2 * j]);
          o[4 * g + 2 * j + 1] = mfma16<DT>(value_int4<DT>(int4_odd(w0), int4_odd(w4)), pf[g], o[4 * g + 2 * j + 1]);
        }
    }
  }
};

template <int DT, int D>
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t token, int head, int d, const float* f) {
  uint16_t* y = p.out + token * p.ot + head * p.oh + d;
  if constexpr (D == 128) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<u32x4*>(y) = w;
  } else {
    *reinterpret_cast<u32x2*>(y) = u32x2{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])};
  }
}

// One workgroup: 16 query rows that share a cache head, one chunk of keys, four
// waves that take its 32-key tiles in turn and meet in LDS at the end.
template <int DT, int FMT, int D>
__global__ __launch_bounds__(256, D == 64 ? 4 : 3) void k_attn16(AttnParams p) {
  constexpr int NX = D / 16, PER = D / 16, LD = D + 4;
  __shared__ float so[4][16][LD];
  __shared__ float sb[4][16], ss[4][16];
  __shared__ u32x4 sq[4 * Rows16<DT, FMT, D>::LOW];
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  // workgroup -> (request, head, row tile, chunk), chunk fastest
  unsigned id = blockIdx.x;
  const int split = int(id % unsigned(p.splits));
  id /= unsigned(p.splits);
  const int rt = int(id % unsigned(p.row_tiles));
  id /= unsigned(p.row_tiles);
  const int h = int(id % unsigned(p.heads)), req = int(id / unsigned(p.heads));
  const Request r(p, req);
  const int rows = r.rows * p.group;
  if (rt * 16 >= rows) return;
  const TileRange range(p, r, rt, 16);
  if (split >= max(range.n, 1)) return;
  const int m = lane & 15, b = lane >> 4;
  const int row = rt * 16 + m;
  const int qi = min(row / p.group, r.rows - 1), qh = h * p.group + row % p.group;
  Rows16<DT, FMT, D> w;
  w.start(p.q + int64_t(r.first + qi) * p.qt + int64_t(qh) * p.qh, p.c < 0.0f, lane, sq + wave * Rows16<DT, FMT, D>::LOW);
  w.low = r.low(p, qi);
  w.high = row < rows ? r.high(p, qi) : 0;
  const int from = range.chunk_from(p, split), to = range.chunk_to(p, split);
  const int32_t* table = p.table + int64_t(req) * p.table_stride;
  const int last_col = (r.len - 1) >> p.page_shift;
  // This wave's tiles: from + 32 (wave + 4 i).  Their pages are fetched 64
  // tiles at a time, one a lane, so that no tile waits for a table entry.
  const int first = from + 32 * __builtin_amdgcn_readfirstlane(wave), tiles = first < to ? (to - first + 127) / 128 : 0;
  int pages0 = 0, pages1 = 0;
  auto fetch = [&](Tile32<FMT, D>& t, int i) {
    if ((i & 63) == 0) {
      const int at = first + 128 * (i + lane);
      pages0 = table[min(at >> p.page_shift, last_col)];
      pages1 = p.page_shift > 4 ? pages0 : table[min((at + 16) >> p.page_shift, last_col)];
    }
    t.load(p, first + 128 * i, __builtin_amdgcn_readlane(pages0, i & 63), __builtin_amdgcn_readlane(pages1, i & 63), h, lane);
  };
  auto multiply = [&](const Tile32<FMT, D>& t, int i) {
    const int token = first + 128 * i;
    w.step(t, token, r.len, token >= range.all_low && token + 32 <= range.all_high && t.ok0 && t.ok1, fabsf(p.c), lane);
  };
  if (tiles > 0) {
    Tile32<FMT, D> t0, t1;
    fetch(t0, 0);
    for (int i = 0;;) {
      if (i + 1 < tiles) fetch(t1, i + 1);
      multiply(t0, i);
      if (++i >= tiles) break;
      if (i + 1 < tiles) fetch(t0, i + 1);
      multiply(t1, i);
      if (++i >= tiles) break;
    }
  }
  // rows of lane (m, b), tile x, register i: column value_col(4 b + i, x)
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) so[wave][m][value_col<FMT, D>(4 * b + i, x)] = w.o[x][i];
  const float total = quad_sum(w.sum);
  if (b == 0) { sb[wave][m] = w.base; ss[wave][m] = total; }
  __syncthreads();
  const int orow = int(threadIdx.x) >> 4, d = (int(threadIdx.x) & 15) * PER;
  float base = sb[0][orow];
#pragma unroll
  for (int i = 1; i < 4; ++i) base = fmaxf(base, sb[i][orow]);
  float sum = 0.0f, f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = exp2_hw(sb[i][orow] - base);
    sum += a * ss[i][orow];
#pragma unroll
    for (int e = 0; e < PER; ++e) f[e] += a * so[i][orow][d + e];
  }
  const int row_o = rt * 16 + orow;
  if (row_o >= rows) return;
  if (range.n > 1) {
    const int64_t at = ((int64_t(req) * p.heads + h) * p.row_slots + row_o) * p.splits + split;
    float* y = p.part + at * D + d;
#pragma unroll
    for (int i = 0; i < PER; i += 4) *reinterpret_cast<f32x4*>(y + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
    if ((int(threadIdx.x) & 15) == 0) {
      float* bs = p.part + int64_t(p.requests) * p.heads * p.row_slots * p.splits * D + at * 2;
      bs[0] = base;
      bs[1] = sum;
    }
    return;
  }
  const int64_t tok = int64_t(r.first) + row_o / p.group;
  const int head = h * p.group + row_o % p.group;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] *= inv;
  store_row<DT, D>(p, tok, head, d, f);
  if (p.lse && (int(threadIdx.x) & 15) == 0)
    p.lse[tok * p.q_heads + head] = row_lse(base, sum);
}

// --------------------------------------------------- wide row tiles (prompts)
// 32 query rows a wave on 32x32x16, NW waves that share each stage of KT keys:
// the workgroup turns a stage's codes into 16-bit operands once, in LDS, in the
// order in which the matrix core reads them (16 bytes a lane, no conflicts):
//   K  [chunk of 8 elements][key]   key rows dealt out so that a lane's S^T
//      registers are 8 neighbouring keys at a time, the operand of O^T = V^T P^T
//   V  [8 keys][column]             column slots dealt out so that a tile of 32
//      holds one INT4 scale group and a lane's results are 4 neighbours
// Stages are double-buffered: stage i + 1 is written and stage i + 2 requested
// while stage i is multiplied, with one barrier a stage.
// INT4: the integers of K go in exactly, the scales of a key come in with the
// multiply-add that takes the reference off.  V, for bf16, goes in times its
// scales as f16, beside f16 probabilities: two roundings to 11 bits instead of
// one of the probabilities to 8 (relative error 1.7e-3 against 2.3e-3), and 5 x
// 2047 rows take 852 us where the scales on the probabilities take 931.
// For f16 that second rounding costs precision (3.4e-4 against 2.8e-4): there
// the integers go in and the scales stay on the probabilities.  MXFP4: the
// probabilities are rounded to the type's bits, as usual for attention; a second
// term for the rest would be half as many matrix instructions again.
// The matrix products bound it, and the vector work beside them: a matrix
// instruction keeps the SIMD from issuing vector ones for half its time.  4608
// tokens, 24 heads of 128, no mask, MXFP4: 261 us, 1000 TFLOP/s (a large bf16
// matrix product: 1250), of which 16% is the second round of 432 workgroups on
// 256 compute units (f16: 274).  5 x 2047 rows behind up to 8191 tokens, 32 heads
// over 8: INT4 830 .. 850 us, 815 TFLOP/s (f16: 955); MXFP4 695, 985 (f16: 726).
// These are calls back to back; one at a time they run 5 to 15% longer, and cards
// differ by 3%.  Slower when they were tried, against 262 us: the next products
// under this softmax (281 us), the two waves of a SIMD one phase apart (306), 64
// rows a wave (434), no running maximum (282).
template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float half_max(float x) {      // over lanes l, l ^ 32
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// N matrix instructions that take an operand from LDS each: four reads go ahead
// of the first, then one behind each (left alone, the compiler waits for nearly
// every read right where it is used).
template <int N>
__device__ __forceinline__ void reads_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
  for (int i = 0; i < N - 4; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
}

template <int FMT, int D, int NW>
struct Stage {
  static constexpr int KT = 64 * NW * 32 / D;     // keys a stage: one 32-element piece of K a thread
  static constexpr int PAGES = KT / 16;           // page lookups a stage
  u32x4 k;                  // 32 codes of one key
  unsigned ke;              // MXFP4: its e8m0; INT4: a key's fp16 scales (lanes < WH * 16)
  unsigned v[8];            // 4 codes of 8 keys
  u32x4 vsc[D == 128 ? 2 : 1];   // the 8 keys' scales (of a key: D / 32 bytes)
};

// A wave's 32 rows over the keys [from, to) where f16 does not take every
// MXFP4 scale of the chunk: 16 at a time, as k_attn16 does them (4608 tokens, 24
// heads of 128, all workgroups: three times the time).
template <int D>
__device__ __forceinline__ void exact_32(const AttnParams& p, const Request& r, int req, int h, int wrow, int rows, int split,
                                         int from, int to, bool whole, int lane, u32x4* wave_low) {
  constexpr int DT = SVDQ_F16, FMT = SVDQ_FMT_MXFP4_G32, PER = D / 16;
  const int m = lane & 15, b = lane >> 4, last_col = (r.len - 1) >> p.page_shift;
  const int32_t* table = p.table + int64_t(req) * p.table_stride;
  for (int row0 = wrow; row0 < smaller(rows, wrow + 32); row0 += 16) {
    const int row = row0 + m, q0 = row0 / p.group, q1 = smaller((row0 + 15) / p.group, r.rows - 1);
    const int qi = smaller(row / p.group, r.rows - 1), qh = h * p.group + row % p.group;
    Rows16<DT, FMT, D> w;
    w.low = r.low(p, qi);
    w.high = row < rows ? r.high(p, qi) : 0;
    w.start(p.q + int64_t(r.first + qi) * p.qt + int64_t(qh) * p.qh, p.c < 0.0f, lane, wave_low);
    const int end = smaller(to, r.high(p, q1)), all_low = r.low(p, q1), all_high = r.high(p, q0);
    for (int token = larger(from, r.low(p, q0) & ~31); token < end; token += 32) {
      Tile32<FMT, D> t;
      const int page = table[smaller(token >> p.page_shift, last_col)];
      t.load(p, token, page, p.page_shift > 4 ? page : table[smaller((token + 16) >> p.page_shift, last_col)], h, lane);
      w.step(t, token, r.len, token >= all_low && token + 32 <= all_high && t.ok0 && t.ok1, fabsf(p.c), lane);
    }
    const float sum = quad_sum(w.sum);
    if (row >= rows) continue;
    const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t tok = int64_t(r.first) + qi, slot = ((int64_t(req) * p.heads + h) * p.row_slots + row) * p.splits + split;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[PER];
#pragma unroll
      for (int x = 0; x < PER; ++x) f[x] = w.o[x][i] * inv;
      const int d = PER * (4 * b + i);             // value_col
      if (whole) {
        store_row<DT, D>(p, tok, qh, d, f);
      } else {
#pragma unroll
        for (int x = 0; x < PER; x += 4) *reinterpret_cast<f32x4*>(p.part + slot * D + d + x) = f32x4{f[x], f[x + 1], f[x + 2], f[x + 3]};
      }
    }
    if (b != 0) continue;
    if (!whole) {
      float* bs = p.part + int64_t(p.requests) * p.heads * p.row_slots * p.splits * D + slot * 2;
      bs[0] = w.base;
      bs[1] = sum;
    } else if (p.lse) {
      p.lse[tok * p.q_heads + qh] = row_lse(w.base, sum);
    }
  }
}

template <int DT, int FMT, int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_rows(AttnParams p) {
  using St = Stage<FMT, D, NW>;
  constexpr int KT = St::KT, NC = D / 8, NB = D / 32, NS = D / 16, NX = D / 32, NG = D / 64, PAGES = St::PAGES;
  constexpr bool MX = FMT == SVDQ_FMT_MXFP4_G32;
  constexpr int NA = MX ? 1 : NG;       // accumulators of a logit (INT4: one a scale group)
  constexpr int VT = MX ? DT : SVDQ_F16;  // type of the second product's operands
  constexpr bool PS = scaled_reference<DT, FMT>();   // value scales on the probabilities, not on the values
  constexpr int NP = PS ? NG : 1;       // probabilities of a logit
  __shared__ u32x4 sk[2][NC * KT];
  __shared__ u32x4 sv[2][KT / 8 * D];
  __shared__ __attribute__((aligned(16))) float sks[2][MX ? 1 : KT * NG];   // INT4: key scales x c
  __shared__ __attribute__((aligned(16))) unsigned svs[2][PS ? KT : 1];  // value scales
  __shared__ float svx[2][MX ? 1 : NW]; // exponents: PS: of the largest value scale of a wave's keys; else what its values were divided by
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  // workgroup -> (row tile, request, head, chunk), chunk fastest; the last row
  // tiles, which see most keys, first; one head's tiles keep to one XCD where
  // the number of heads allows it
  unsigned id = blockIdx.x;
  const int split = int(id % unsigned(p.splits));
  id /= unsigned(p.splits);
  const int h = int(id % unsigned(p.heads));
  id /= unsigned(p.heads);
  const int req = int(id % unsigned(p.requests));
  const int rt = p.row_tiles - 1 - int(id / unsigned(p.requests));
  constexpr int ROWS = 32 * NW;
  const Request r(p, req);
  const int rows = r.rows * p.group;
  if (rt * ROWS >= rows) return;
  const TileRange range(p, r, rt, ROWS);
  if (split >= max(range.n, 1)) return;
  const int m = lane & 31, hb = lane >> 5;
  // this wave's rows
  const int wv = __builtin_amdgcn_readfirstlane(wave);
  const int wrow = rt * ROWS + 32 * wv, wq0 = min(wrow / p.group, r.rows - 1), wq1 = min((wrow + 32 - 1) / p.group, r.rows - 1);
  const int wfrom = r.low(p, wq0), wto = wrow < rows ? r.high(p, wq1) : 0, wall_low = r.low(p, wq1), wall_high = r.high(p, wq0);
  const int row = wrow + m;
  const int qi = min(row / p.group, r.rows - 1), qh = h * p.group + row % p.group;
  const int low = r.low(p, qi), high = row < rows ? r.high(p, qi) : 0;
  u32x4 q[NS];
  {
    const uint16_t* src = p.q + int64_t(r.first + qi) * p.qt + int64_t(qh) * p.qh + 8 * hb;
#pragma unroll
    for (int e = 0; e < NS; ++e) q[e] = query_order<FMT>(*reinterpret_cast<const u32x4*>(src + 16 * e));
    if (p.c < 0.0f) {       // the sign of the scale goes to the query: the largest product is the largest logit
#pragma unroll
      for (int e = 0; e < NS; ++e) q[e] ^= 0x80008000u;
    }
  }
  const float c = fabsf(p.c) * value_gain<DT, FMT>();
  f32x16 o[NX];
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[x][i] = 0.0f;
  // A row's reference, and how far above it a logit may be before it is raised
  // (-infinity until the row has seen a key).
  float base = 0.0f, limit = -__builtin_inff(), sum = 0.0f;
  const float zero = hidden_zero();
  bool off = false;                     // a scale that f16 does not take has been met

  const int from = range.chunk_from(p, split), to = range.chunk_to(p, split);
  const int32_t* table = p.table + int64_t(req) * p.table_stride;
  const int last_col = (r.len - 1) >> p.page_shift, in_page = (1 << p.page_shift) - 1;
  // A wave brings the WH x 16 keys [16 WH wave, ..) of a stage, whose pages are
  // the same for all its lanes: addresses are scalar bases plus lane offsets.
  constexpr int WH = KT / 16 / NW;
  const int kkey = tid / NB, kb = tid % NB;                   // K piece: key of the stage, 32-element block
  const int vkeys = tid / (D / 4) * 8, vn = tid % (D / 4);    // V block: first of 8 keys, columns 4 vn ..
  // a lane's page of the stage at `token` (lane l: keys 16 (l % PAGES) ..)
  auto look_up = [&](int token) {
    const int t = token + 16 * (lane % PAGES);
    return table[min(t >> p.page_shift, last_col)];
  };
  auto bad_pages = [&](int page) { return unsigned(__ballot(page < 0 || page >= p.n_pages)); };   // bit i: keys 16 i ..
  auto request = [&](St& st, int token, int page) {
    const int good = page < 0 || page >= p.n_pages ? 0 : page;
    int64_t row[WH];        // cache row of the first key of each 16
#pragma unroll
    for (int i = 0; i < WH; ++i)
      row[i] = ((int64_t(__builtin_amdgcn_readlane(good, wv * WH + i)) * p.heads + h) << p.page_shift) +
               ((token + 16 * (wv * WH + i)) & in_page);
    auto at = [&](const void* base, int key, int row_bytes) {  // key of the wave's
      const uint8_t* b0 = static_cast<const uint8_t*>(base) + row[0] * row_bytes;
      if constexpr (WH == 1) return b0 + unsigned(key * row_bytes);
      const uint8_t* b1 = static_cast<const uint8_t*>(base) + row[WH - 1] * row_bytes;
      return (key >= 16 ? b1 : b0) + unsigned((key & 15) * row_bytes);
    };
    st.k = *reinterpret_cast<const u32x4*>(at(p.kc, lane / NB, D / 2) + 16 * kb);
    const int vk = lane / (D / 4) * 8;
    const uint8_t* vc = at(p.vc, vk, D / 2) + 2 * vn;
#pragma unroll
    for (int i = 0; i < 8; ++i) st.v[i] = *reinterpret_cast<const uint16_t*>(vc + i * (D / 2));
    const u32x4* vs = reinterpret_cast<const u32x4*>(at(p.vs, vk, NB));
    st.vsc[0] = vs[0];
    if constexpr (D == 128) st.vsc[1] = vs[1];
    if constexpr (MX) {
      st.ke = *(at(p.ks, lane / NB, NB) + kb);
    } else if (lane < 16 * WH) {
      if constexpr (D == 128) st.ke = *reinterpret_cast<const unsigned*>(at(p.ks, lane, 4));
      else st.ke = *reinterpret_cast<const uint16_t*>(at(p.ks, lane, 2));
    }
  };
  // Keys past the end or on a missing page may hold a NaN: their value scales
  // become zero (MXFP4: the smallest; f16: one, and the key's), before the stage is
  // turned into operands.
  auto mend = [&](St& st, int token, unsigned bad) {
    if (bad == 0u && token + KT <= r.len) return;       // the same for all threads
    const bool gone = (bad >> (vkeys / 16)) & 1u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool zero = gone || token + vkeys + i >= r.len;
      constexpr unsigned none = checks_scales<DT, FMT>() ? 0x7F7F7F7Fu : 0u;
      if constexpr (D == 128) {
        st.vsc[i / 4][i % 4] = zero ? none : st.vsc[i / 4][i % 4];
      } else {
        const unsigned other = i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        st.vsc[0][i / 2] = zero ? (st.vsc[0][i / 2] & other) | (none & ~other) : st.vsc[0][i / 2];
      }
    }
    if constexpr (checks_scales<DT, FMT>()) st.ke = ((bad >> (kkey / 16)) & 1u) != 0u || token + kkey >= r.len ? 127u : st.ke;
  };
  auto write = [&](const St& st, int buf) {
    // K: key row with bits 2 and 3 exchanged, and an exchange of neighbours by
    // block that spreads the writes over the banks
    const int krow = ((kkey & ~12) | ((kkey & 4) << 1) | ((kkey & 8) >> 1)) ^ (kb << 1);
    const float ks = MX ? mx_scale<DT>(st.ke) : 0.0f;
    if constexpr (checks_scales<DT, FMT>()) {
      unsigned any = off_scale(st.ke);
#pragma unroll
      for (int i = 0; i < 8; ++i) any += off_scale(value_exponent<D>(st.vsc, i, vn >> 3));
      if (any != 0u) {                  // of values other than zeros?
        off |= off_scale(st.ke) != 0u && ((st.k[0] | st.k[1] | st.k[2] | st.k[3]) & 0x77777777u) != 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) off |= off_scale(value_exponent<D>(st.vsc, i, vn >> 3)) != 0u && (st.v[i] & 0x7777u) != 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sk[buf][(4 * kb + j) * KT + krow] = key_frag<DT, FMT>(st.k[j], ks);
    const int slot = 64 * (vn / 16) + vn % 16;                 // column 4 vn + j: slot + 16 j
    u32x4* v = &sv[buf][vkeys / 8 * D + slot];
    if constexpr (MX) {
      u32x4 f0, f1;
      float sc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] = value_scale<DT, D>(st.vsc, i, vn >> 3);
      value_pair_mx<DT, 0>(st.v, sc, &f0, &f1);
      v[0] = f0;
      v[16] = f1;
      value_pair_mx<DT, 1>(st.v, sc, &f0, &f1);
      v[32] = f0;
      v[48] = f1;
    } else {
      unsigned cols[2][2], sc[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 2; ++k) deal(st.v + 4 * k, byte_pick(0), cols[k]);
      float gain = 512.0f;
      if constexpr (PS) {
        float x = most_scale<D>(st.vsc);
        x = D == 128 ? half_max(x) : quad_max(x);
        if (lane == 0) svx[buf][wave] = scale_exponent(x);
        if (vn == 0) {
          u32x4* y = reinterpret_cast<u32x4*>(&svs[buf][vkeys]);
          if constexpr (D == 128) {
            y[0] = st.vsc[0];
            y[1] = st.vsc[1];
          } else {
            y[0] = u32x4{st.vsc[0][0], st.vsc[0][0] >> 16, st.vsc[0][1], st.vsc[0][1] >> 16};
            y[1] = u32x4{st.vsc[0][2], st.vsc[0][2] >> 16, st.vsc[0][3], st.vsc[0][3] >> 16};
          }
        }
      } else {
        const unsigned pick = vn >= 16 ? 0x07060302u : 0x05040100u;      // D = 128: the half of the columns' group
        // 7 times a scale from 2^13 on would pass f16: then the wave's values go
        // in at an eighth, and their probabilities at eight times
        bool big = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) sc[i] = __builtin_amdgcn_perm(st.vsc[i / 2][2 * i % 4 + 1], st.vsc[i / 2][2 * i % 4], pick);
          else sc[i] = st.vsc[0][i];
          big |= (sc[i] & 0x7000u) == 0x7000u || (sc[i] & 0x70000000u) == 0x70000000u;
        }
        const bool any = __any(big);
        if (any) gain = 64.0f;
        if (lane == 0) svx[buf][wave] = any ? 3.0f : 0.0f;
      }
      if (lane < 16 * WH) {
        const f16x2 ks = two_halves(st.ke);
        if constexpr (NG == 2) *reinterpret_cast<f32x2*>(&sks[buf][2 * (16 * WH * wave + lane)]) = f32x2{float(ks[0]) * c, float(ks[1]) * c};
        else sks[buf][16 * WH * wave + lane] = float(ks[0]) * c;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned w0 = cols[0][j], w4 = cols[1][j];
        if constexpr (PS) {
          v[32 * j] = value_int4<VT>(int4_even(w0), int4_even(w4));
          v[32 * j + 16] = value_int4<VT>(int4_odd(w0), int4_odd(w4));
        } else {
          v[32 * j] = value_int4_scaled(int4_even(w0), int4_even(w4), sc, gain);
          v[32 * j + 16] = value_int4_scaled(int4_odd(w0), int4_odd(w4), sc, gain);
        }
      }
    }
  };

  // Logits of 64 keys of stage `buf` from key `at` of it on.  INT4: in powers of
  // two and less the reference so far, one multiply-add a logit and scale group
  // (5 x 2047 rows 4% faster than with one of its own for the reference).  MXFP4:
  // as they come from the product (taken here, before the maximum, the
  // multiply-add that it needs all the same costs 270 us instead of 262).
  auto logits = [&](int buf, int at, f32x16* s) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      f32x16 acc[NA];
#pragma unroll
      for (int g = 0; g < NA; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[g][i] = 0.0f;
#pragma unroll
      for (int e = 0; e < NS; ++e) {
        const u32x4 a = sk[buf][(2 * e + hb) * KT + ((at + 32 * kt + m) ^ ((e / 2) << 1))];
        acc[MX ? 0 : e / 4] = mfma32<DT>(a, q[e], acc[MX ? 0 : e / 4]);
      }
      reads_ahead<NS>();
      if constexpr (MX) {
        s[kt] = acc[0];
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {     // keys 16 (x / 2) + 8 hb + 4 (x % 2) ..
          f32x4 w[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g)
            w[g] = *reinterpret_cast<const f32x4*>(&sks[buf][(at + 32 * kt + 16 * (x / 2) + 8 * hb + 4 * (x % 2)) * NG + 4 * g]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (NG == 2)
              s[kt][4 * x + i] = __builtin_fmaf(acc[NA - 1][4 * x + i], w[i / 2][2 * i % 4 + 1],
                                                __builtin_fmaf(acc[0][4 * x + i], w[i / 2][2 * i % 4], -base));
            else
              s[kt][4 * x + i] = __builtin_fmaf(acc[0][4 * x + i], w[0][i], -base);
          }
        }
        asm volatile("" : "+v"(s[kt]));    // here, not after the next tile's products: 66 registers of spills
      }
    }
  };
  // Masks them and raises the rows' references where they need it.
  auto refer = [&](int token, int at, unsigned bad, float most, f32x16* s) {
    const int t0 = token + at;
    const unsigned gone = (bad >> (at / 16)) & 15u;
    if (!(t0 >= wall_low && t0 + 64 <= wall_high && gone == 0u)) {
      // (in place, as vectors: element by element the compiler copies the
      // logits on the way round this, too)
      const unsigned first = unsigned(t0 + 8 * hb - low), wide = unsigned(max(high - low, 0));
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const unsigned k = 32 * (i / 16) + 16 * ((i % 16) / 8) + i % 8;
        s[i / 16][i % 16] = first + k < wide ? s[i / 16][i % 16] : -__builtin_inff();
      }
      if (gone != 0u) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          s[i / 16][i % 16] = ((gone >> (i / 8)) & 1u) == 0u ? s[i / 16][i % 16] : -__builtin_inff();
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i / 16][i % 16]);     // `maximum` is no faster here (INT4 856 us, 852)
    top = half_max(top);
    if constexpr (MX) top = __builtin_fmaf(top, c, -base);
    else top += most;
    if (__any(top > limit)) {
      const bool first_keys = limit < 0.0f, seen = top > -__builtin_inff();
      const float up = first_keys ? (seen ? top - p_shift<VT>() : 0.0f) : fmaxf(top - p_shift<VT>(), 0.0f);
      const float alpha = first_keys ? 1.0f : exp2_hw(-up);
      base += up;
      limit = first_keys && !seen ? limit : p_shift<VT>() + SLACK;
      if constexpr (!MX) {
        s[0] -= up;
        s[1] -= up;
      }
      sum *= alpha;
#pragma unroll
      for (int x = 0; x < NX; ++x) o[x] *= alpha;
    }
  };
  // Probabilities of these keys as operands.
  auto weigh = [&](int buf, int at, float most, f32x16* s, u32x4 (*pf)[4]) {
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      s[i / 16][i % 16] = exp2_hw(MX ? __builtin_fmaf(s[i / 16][i % 16], c, -base) : s[i / 16][i % 16]);
      part += s[i / 16][i % 16];
    }
    sum += part;
    if constexpr (!PS) {
#pragma unroll
      for (int i = 0; i < 16; ++i) pf[0][i / 4][i % 4] = pack2<VT>(s[i / 8][2 * i % 16], s[i / 8][2 * i % 16 + 1]);
      if (!MX && most > 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {       // keys 16 i ..
          const _Float16 g = svx[buf][(at + 16 * i) / (16 * WH)] > 0.0f ? 8 : 1;
#pragma unroll
          for (int e = 0; e < 4; ++e) pf[0][i][e] = __builtin_bit_cast(unsigned, two_halves(pf[0][i][e]) * f16x2{g, g});
        }
      }
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) {       // keys 16 (x / 2) + 8 hb + 4 (x % 2) ..
        const u32x4 w = *reinterpret_cast<const u32x4*>(&svs[buf][at + 16 * (x / 2) + 8 * hb + 4 * (x % 2)]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float p0 = s[x / 4][4 * x % 16 + i], p1 = s[x / 4][4 * x % 16 + i + 1];
          pf[0][x / 2][2 * (x % 2) + i / 2] = pack2<VT>(fma_half<0>(p0, w[i], zero), fma_half<0>(p1, w[i + 1], zero));
          if constexpr (NP == 2)
            pf[NP - 1][x / 2][2 * (x % 2) + i / 2] = pack2<VT>(fma_half<1>(p0, w[i], zero), fma_half<1>(p1, w[i + 1], zero));
        }
      }
    }
  };
  // the largest exponent of these keys' values
  auto exponent = [&](int buf, int at) {
    if constexpr (MX) return 0.0f;
    float most = svx[buf][at / (16 * WH)];
#pragma unroll
    for (int i = 1; i < 4 / WH; ++i) most = fmaxf(most, svx[buf][at / (16 * WH) + i]);
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(most)));
  };
  auto add_values = [&](int buf, int at, const u32x4 (*pf)[4]) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 a = sv[buf][(at / 8 + 2 * j + hb) * D + 32 * x + m];
        o[x] = mfma32<VT>(a, pf[NP == 2 ? x / 2 : 0][j], o[x]);
      }
    }
    reads_ahead<4 * NX>();
  };

  if (from < to) {
    St st;
    int page = look_up(from);
    unsigned bad = bad_pages(page), bad1 = 0;
    request(st, from, page);
    page = look_up(from + KT);
    mend(st, from, bad);
    write(st, 0);
    if (from + KT < to) {
      bad1 = bad_pages(page);
      request(st, from + KT, page);
      page = look_up(from + 2 * KT);
    }
    __syncthreads();
    auto used = [&](int t) { return t < wto && t + 64 > wfrom && t < to; };
    int buf = 0;
    // Where the loop stands in memory, by what its instructions' fetches make of
    // it (4608 full, MXFP4, by its offset in 32 bytes: 265 .. 279 us, f16 268 .. 284;
    // 5 x 2047 rows: MXFP4 705 .. 727, INT4 846 .. 857).
    constexpr int OFFSET = !MX ? 6 : DT == SVDQ_F16 ? 0 : 2;       // words
    asm volatile(".p2align 6\n\t.rept %0\n\ts_nop 0\n\t.endr" ::"i"(OFFSET));
    for (int token = from; token < to; token += KT) {
      const unsigned here = bad;
      if (token + KT < to) {
        mend(st, token + KT, bad1);
        write(st, buf ^ 1);
        bad = bad1;
        if (token + 2 * KT < to) {
          bad1 = bad_pages(page);
          request(st, token + 2 * KT, page);
          page = look_up(token + 3 * KT);
        }
      }
#pragma unroll 2
      for (int at = 0; at < KT; at += 64) {
        if (!used(token + at)) continue;
        f32x16 s[2];
        u32x4 pf[NP][4];
        // the wave that multiplies issues before the one beside it that does
        // not, which keeps the two apart
        __builtin_amdgcn_s_setprio(1);
        logits(buf, at, s);
        __builtin_amdgcn_s_setprio(0);
        const float most = exponent(buf, at);
        refer(token, at, here, most, s);
        weigh(buf, at, most, s, pf);
        __builtin_amdgcn_s_setprio(1);
        add_values(buf, at, pf);
        __builtin_amdgcn_s_setprio(0);
      }
      __syncthreads();
      buf ^= 1;
    }
  }
  const bool whole = range.n <= 1;
  if constexpr (checks_scales<DT, FMT>()) {
    if (__syncthreads_or(off)) {
      static_assert(NW * Rows16<DT, FMT, D>::LOW <= NC * KT, "the queries' second terms lie where the keys were");
      exact_32<D>(p, r, req, h, wrow, rows, split, from, to, whole, lane, sk[0] + wave * Rows16<DT, FMT, D>::LOW);
      return;
    }
  }
  sum = half_sum(sum);
  if (limit < 0.0f) base = LOWEST;
  if (row >= rows) return;
  const float inv = !whole ? value_gain<DT, FMT>() : sum == 0.0f ? 0.0f : value_gain<DT, FMT>() / sum;
  const int64_t tok = int64_t(r.first) + row / p.group;
  const int head = h * p.group + row % p.group;
  const int64_t slot = ((int64_t(req) * p.heads + h) * p.row_slots + row) * p.splits + split;
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = 64 * g + 4 * (8 * (i / 4) + 4 * hb + i % 4);
      const f32x4 f = {o[2 * g][i] * inv, o[2 * g][i + 8] * inv, o[2 * g + 1][i] * inv, o[2 * g + 1][i + 8] * inv};
      if (whole) *reinterpret_cast<u32x2*>(p.out + tok * p.ot + head * p.oh + d) = u32x2{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])};
      else *reinterpret_cast<f32x4*>(p.part + slot * D + d) = f;
    }
  if (hb != 0) return;
  if (!whole) {
    float* bs = p.part + int64_t(p.requests) * p.heads * p.row_slots * p.splits * D + slot * 2;
    bs[0] = base;
    bs[1] = sum;
  } else if (p.lse) {
    p.lse[tok * p.q_heads + head] = row_lse(base, sum);
  }
}

// Joins the chunks of a row.  Few chunks: D / 4 lanes a row, several rows a
// workgroup.
template <int DT, int D, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join_few(AttnParams p) {
  constexpr int L = D / 4, G = 256 / L;
  const int64_t slot = int64_t(blockIdx.x) * G + int(threadIdx.x) / L, slots = int64_t(p.requests) * p.heads * p.row_slots;
  if (slot >= slots) return;
  unsigned id = unsigned(slot);
  const int row = int(id % unsigned(p.row_slots));
  id /= unsigned(p.row_slots);
  const int h = int(id % unsigned(p.heads)), req = int(id / unsigned(p.heads));
  const Request r(p, req);
  if (row >= r.rows * p.group) return;
  const TileRange range(p, r, row / ROWS, ROWS);
  if (range.n <= 1) return;
  const int d = int(threadIdx.x) % L * 4;
  const int64_t at = slot * p.splits;
  const f32x2* bs = reinterpret_cast<const f32x2*>(p.part + slots * p.splits * D) + at;
  const float* y = p.part + at * D + d;
  float base = LOWEST, sum = 0.0f;
  f32x4 f = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < range.n; ++s) base = fmaxf(base, bs[s][0]);
#pragma unroll 4
  for (int s = 0; s < range.n; ++s) {
    const f32x2 v = bs[s];
    const f32x4 u = *reinterpret_cast<const f32x4*>(y + int64_t(s) * D);
    const float a = exp2_hw(v[0] - base);
    sum += a * v[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] += a * u[e];
  }
  const int64_t tok = int64_t(r.first) + row / p.group;
  const int head = h * p.group + row % p.group;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2*>(p.out + tok * p.ot + head * p.oh + d) = u32x2{pack2<DT>(f[0] * inv, f[1] * inv), pack2<DT>(f[2] * inv, f[3] * inv)};
  if (p.lse && d == 0) p.lse[tok * p.q_heads + head] = row_lse(base, sum);
}

// Many chunks: a workgroup a row.  Its threads fetch all references at once,
// then 1024 / D groups of D / 4 threads walk the chunks and meet in LDS in a
// fixed order.
template <int DT, int D, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(AttnParams p) {
  constexpr int L = D / 4, G = 256 / L;
  __shared__ float sw[256];             // weights of 256 chunks
  __shared__ float red[G][D];
  __shared__ float wave_v[4], wave_s[4];
  const int tid = int(threadIdx.x);
  unsigned id = blockIdx.x;
  const int row = int(id % unsigned(p.row_slots));
  id /= unsigned(p.row_slots);
  const int h = int(id % unsigned(p.heads)), req = int(id / unsigned(p.heads));
  const Request r(p, req);
  if (row >= r.rows * p.group) return;
  const TileRange range(p, r, row / ROWS, ROWS);
  if (range.n <= 1) return;
  const int64_t at = int64_t(blockIdx.x) * p.splits;
  const f32x2* bs = reinterpret_cast<const f32x2*>(p.part + int64_t(gridDim.x) * p.splits * D) + at;
  float base = LOWEST;
  for (int s = tid; s < range.n; s += 256) base = fmaxf(base, bs[s][0]);
#pragma unroll
  for (int m = 1; m < 64; m *= 2) base = fmaxf(base, __shfl_xor(base, m));
  if ((tid & 63) == 0) wave_v[tid / 64] = base;
  __syncthreads();
  base = fmaxf(fmaxf(wave_v[0], wave_v[1]), fmaxf(wave_v[2], wave_v[3]));
  float sum = 0.0f;
  f32x4 f = {0, 0, 0, 0};
  const int grp = tid / L, d = (tid % L) * 4;
  for (int s0 = 0; s0 < range.n; s0 += 256) {
    const int n = min(256, range.n - s0);
    if (tid < n) {
      const f32x2 v = bs[s0 + tid];
      const float a = exp2_hw(v[0] - base);
      sw[tid] = a;
      sum += a * v[1];
    }
    __syncthreads();
    const float* y = p.part + (at + s0) * D + d;
#pragma unroll 4
    for (int s = grp; s < n; s += G) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(y + int64_t(s) * D);
      const float a = sw[s];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += a * v[e];
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
  if ((tid & 63) == 0) wave_s[tid / 64] = sum;
  *reinterpret_cast<f32x4*>(&red[grp][d]) = f;
  __syncthreads();
  sum = (wave_s[0] + wave_s[1]) + (wave_s[2] + wave_s[3]);
  if (tid >= D / 2) return;
  float f0 = 0.0f, f1 = 0.0f;
#pragma unroll
  for (int i = 0; i < G; ++i) { f0 += red[i][2 * tid]; f1 += red[i][2 * tid + 1]; }
  const int64_t tok = int64_t(r.first) + row / p.group;
  const int head = h * p.group + row % p.group;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<unsigned*>(p.out + tok * p.ot + head * p.oh + 2 * tid) = pack2<DT>(f0 * inv, f1 * inv);
  if (p.lse && tid == 0) p.lse[tok * p.q_heads + head] = row_lse(base, sum);
}

// ---------------------------------------------------------------- host side
int device_cus() {
  static std::atomic<int> cus[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int v = cus[dev].load(std::memory_order_relaxed);
  if (v <= 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cus[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

svdq_status check_attn(const svdq_attn_desc* d, const svdq_kv_cache* c) {
  if (!d || d->requests < 0 || d->tokens < 0 || !dtype_ok(d->dtype) || (d->flags & ~unsigned(SVDQ_ATTN_CAUSAL)) != 0u ||
      d->max_q < 0 || d->max_kv < 0 || d->window < 0 || d->table_stride < 0 || d->q_heads < 1)
    return SVDQ_ERR_INVALID_ARG;
  if (!(d->scale == d->scale)) return SVDQ_ERR_INVALID_ARG;
  const svdq_status st = check_cache(c);
  if (st != SVDQ_OK) return st;
  return d->q_heads % c->heads != 0 ? SVDQ_ERR_SHAPE : SVDQ_OK;
}

template <int DT, int D, int ROWS>
void launch_join(const AttnParams& p, const Cut& t, hipStream_t st) {
  const int64_t slots = int64_t(p.requests) * p.heads * t.row_slots;
  if (t.splits <= 16) k_attn_join_few<DT, D, ROWS><<<dim3(unsigned(ceil_div(slots, 1024 / D))), 256, 0, st>>>(p);
  else k_attn_join<DT, D, ROWS><<<dim3(unsigned(slots)), 256, 0, st>>>(p);
}

template <int DT, int FMT, int D>
void launch_attn(const AttnParams& p, const Cut& t, hipStream_t st) {
  const dim3 grid(unsigned(t.items * t.splits));
  if (t.rows == 16) {
    k_attn16<DT, FMT, D><<<grid, 256, 0, st>>>(p);
    if (t.splits > 1) launch_join<DT, D, 16>(p, t, st);
  } else if (t.rows == 128) {
    k_attn_rows<DT, FMT, D, 4><<<grid, 256, 0, st>>>(p);
    if (t.splits > 1) launch_join<DT, D, 128>(p, t, st);
  } else {
    k_attn_rows<DT, FMT, D, 8><<<grid, 512, 0, st>>>(p);
    if (t.splits > 1) launch_join<DT, D, 256>(p, t, st);
  }
}

template <int DT, int FMT>
void launch_attn(const AttnParams& p, const Cut& t, int D, hipStream_t st) {
  if (D == 64) launch_attn<DT, FMT, 64>(p, t, st);
  else launch_attn<DT, FMT, 128>(p, t, st);
}

}  // namespace

extern "C" svdq_status svdq_kv_attention_workspace(const svdq_attn_desc* d, const svdq_kv_cache* c, size_t* bytes) {
  svdq_status st = check_attn(d, c);
  if (st != SVDQ_OK) return st;
  if (!bytes) return SVDQ_ERR_INVALID_ARG;
  *bytes = 0;
  if (d->requests == 0 || d->tokens == 0 || d->max_q == 0) return SVDQ_OK;
  Cut t;
  if ((st = cut_of(d, c, device_cus(), &t)) != SVDQ_OK) return st;
  *bytes = part_bytes(c, most_part_rows(d, c, device_cus()));
  return SVDQ_OK;
}

extern "C" svdq_status svdq_kv_attention(const svdq_attn_desc* d, const svdq_heads* q, const svdq_kv_cache* c,
                                         const svdq_heads* out, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  svdq_status st = check_attn(d, c);
  if (st != SVDQ_OK) return st;
  if (!q || !out) return SVDQ_ERR_INVALID_ARG;
  if (q->heads != d->q_heads || out->heads != d->q_heads) return SVDQ_ERR_SHAPE;
  if (d->requests == 0 || d->tokens == 0 || d->max_q == 0) return SVDQ_OK;
  if ((st = check_heads(q, c->head_dim)) != SVDQ_OK || (st = check_heads(out, c->head_dim)) != SVDQ_OK) return st;
  if (!d->q_start || !d->kv_len || (d->table_stride > 0 && !d->block_table)) return SVDQ_ERR_INVALID_ARG;
  Cut t;
  if ((st = cut_of(d, c, device_cus(), &t)) != SVDQ_OK) return st;
  const size_t need = part_bytes(c, part_rows(d, c, t));
  if (need > 0) {
    if (!ws) return SVDQ_ERR_INVALID_ARG;
    if (ws_bytes < need) return SVDQ_ERR_CAPACITY;
    if (!aligned(ws, 256)) return SVDQ_ERR_INVALID_ARG;
  }
  AttnParams p = {};
  p.q = static_cast<const uint16_t*>(q->data);
  p.out = static_cast<uint16_t*>(out->data);
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  p.kc = static_cast<const uint8_t*>(c->k_codes);
  p.ks = static_cast<const uint8_t*>(c->k_scales);
  p.vc = static_cast<const uint8_t*>(c->v_codes);
  p.vs = static_cast<const uint8_t*>(c->v_scales);
  p.q_start = d->q_start; p.kv_len = d->kv_len; p.table = d->block_table;
  p.qt = q->token_stride; p.qh = q->head_stride;
  p.ot = out->token_stride; p.oh = out->head_stride;
  p.tokens = t.tokens; p.table_stride = d->table_stride; p.n_pages = c->n_pages;
  p.requests = int32_t(d->requests); p.q_heads = d->q_heads; p.heads = c->heads; p.group = d->q_heads / c->heads;
  p.max_q = d->max_q; p.max_kv = t.keys; p.window = d->window;
  p.causal = (d->flags & SVDQ_ATTN_CAUSAL) != 0u;
  p.page_shift = page_shift(c->page_size);
  p.row_tiles = t.row_tiles; p.row_slots = int32_t(t.row_slots); p.splits = t.splits; p.chunk = t.chunk;
  const bool mx = c->fmt == SVDQ_FMT_MXFP4_G32, bf = d->dtype == SVDQ_BF16;
  p.c = d->scale * 1.44269504088896341f;
  if (p.c == 0.0f) p.c = 1.2e-38f;      // every logit is zero to fp32, and a masked -infinity stays one
  if (bf) {
    if (mx) launch_attn<SVDQ_BF16, SVDQ_FMT_MXFP4_G32>(p, t, c->head_dim, stream);
    else launch_attn<SVDQ_BF16, SVDQ_FMT_INT4_G64>(p, t, c->head_dim, stream);
  } else {
    if (mx) launch_attn<SVDQ_F16, SVDQ_FMT_MXFP4_G32>(p, t, c->head_dim, stream);
    else launch_attn<SVDQ_F16, SVDQ_FMT_INT4_G64>(p, t, c->head_dim, stream);
  }
  return launch_ok();
}
