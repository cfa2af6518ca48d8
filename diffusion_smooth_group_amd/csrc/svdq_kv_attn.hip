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
  float* part;              // [item][split][16][D] partial sums, then [item][split][16][2] reference and sum
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t *q_start, *kv_len, *table;
  int64_t qt, qh, ot, oh, tokens, table_stride, n_pages;
  int32_t requests, q_heads, heads, group;      // group = q_heads / heads
  int32_t max_q, max_kv, window, causal, page_shift;
  int32_t row_tiles, splits, chunk;             // row tiles a request has at most; key chunks
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

// e8m0 byte in bits 23-30, ready as the converters' scale.  f16: values are
// held at 2^-3 of their size (so that 6 x 2^15 still fits and 2^-20 x 0.5 is
// still exact), exponents limited to what f16 can then hold; the missing 2^3
// is put back on the fp32 sums.
template <int DT>
__device__ __forceinline__ float mx_scale(unsigned e) {
  if constexpr (DT == SVDQ_F16) e = min(max(e, 3u), 142u) - 3u;
  return __uint_as_float(e << 23);
}
template <int DT, int FMT>
constexpr float value_gain() { return DT == SVDQ_F16 && FMT == SVDQ_FMT_MXFP4_G32 ? 8.0f : 1.0f; }

// f16 probabilities are held at 2^6 of their size: the f16 subnormals start
// far lower than any probability that counts, and 2^(6 + 8) still fits.  The
// factor is in the row's reference, so it drops out of the quotient.
template <int DT>
constexpr float p_shift() { return DT == SVDQ_F16 ? 6.0f : 0.0f; }
// The reference is raised only when a row's maximum has passed it by 2^8;
// between that the sums stay in range and no accumulator is touched.
constexpr float SLACK = 8.0f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// max / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 of a column
__device__ __forceinline__ float quad_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const unsigned v = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const unsigned v = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A request's rows and the keys they see.
struct Request {
  int rows, all_rows, len, true_len;
  int64_t first;
  __device__ __forceinline__ Request(const AttnParams& p, int r) {
    const int64_t s = p.q_start[r], e = p.q_start[r + 1];
    all_rows = int(e - s);
    first = s < 0 ? 0 : s;
    int64_t n = e < p.tokens ? e : p.tokens;
    n -= first;
    rows = n < 0 || s < 0 ? 0 : int(n < p.max_q ? n : p.max_q);
    true_len = p.kv_len[r];
    const int64_t room = p.table_stride << p.page_shift;
    int64_t l = true_len < p.max_kv ? true_len : p.max_kv;
    l = l < room ? l : room;
    len = p.n_pages == 0 || l < 0 ? 0 : int(l);
  }
  // keys [low, high) that row i sees
  __device__ __forceinline__ int high(const AttnParams& p, int i) const {
    const int pos = true_len - all_rows + i;
    return p.causal ? max(0, min(pos + 1, len)) : len;
  }
  __device__ __forceinline__ int low(const AttnParams& p, int i) const {
    const int pos = true_len - all_rows + i;
    return p.window > 0 ? max(0, pos - p.window + 1) : 0;
  }
};

// Cache rows of 16 neighbouring tokens of one head, and whether their page is there.
struct HalfTile {
  int64_t row;
  bool ok;
};
__device__ __forceinline__ HalfTile half_tile(const AttnParams& p, const int32_t* table, int token, int last_col, int h) {
  const int col = min(token >> p.page_shift, last_col);
  const int page = __builtin_amdgcn_readfirstlane(table[col]);
  HalfTile t;
  t.ok = page >= 0 && page < p.n_pages;
  t.row = ((int64_t(t.ok ? page : 0) * p.heads + h) << p.page_shift) + (token & ((1 << p.page_shift) - 1));
  return t;
}

// ----------------------------------------------------- 16 rows and one wave
// S^T = K Q^T on 16x16x32: keys are rows of the result, query rows its
// columns, so that a lane holds the probabilities of one query row for the
// keys [8b, 8b + 8) of a 32-key tile (b = lane / 16) -- which is the operand of
// O^T = V^T P^T as it stands; the keys of the two K tiles are dealt out for
// that (tile a, row r: key 8 (r / 4) + 4 a + r % 4).  V^T needs 8 keys of one
// column in a lane: a lane loads 8 keys' codes of its own columns and pairs
// neighbouring keys after the conversion.
template <int FMT, int D>
struct Tile32 {
  static constexpr int NJ = D / 32;
  static constexpr int NS = FMT == SVDQ_FMT_MXFP4_G32 ? (D == 128 ? 2 : 1) : (D == 128 ? 2 : 1);
  unsigned k[2][NJ];        // codes of the lane's key row in each K tile
  unsigned ke[2];           // MXFP4: e8m0 of the lane's key rows and group
  u32x4 ksc[NS];            // INT4: fp16 scales of the keys [8b, 8b + 8)
  unsigned v[8];            // codes of the lane's columns, keys [8b, 8b + 8)
  u32x4 vsc[NS];            // scales of these keys
  bool ok0, ok1;            // the pages of the tile's halves are there

  __device__ __forceinline__ void load(const AttnParams& p, const HalfTile& h0, const HalfTile& h1, int lane) {
    const int m = lane & 15, b = lane >> 4;
    ok0 = h0.ok;
    ok1 = h1.ok;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int lt = 8 * (m >> 2) + 4 * a + (m & 3);
      const int64_t row = (m >= 8 ? h1.row - 16 : h0.row) + lt;
      const uint8_t* c = p.kc + row * (D / 2);
      if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
        if constexpr (D == 128) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(c + 16 * b);
          k[a][0] = w[0]; k[a][1] = w[1]; k[a][2] = w[2]; k[a][3] = w[3];
          ke[a] = p.ks[row * 4 + b];
        } else {
          const u32x2 w = *reinterpret_cast<const u32x2*>(c + 8 * b);
          k[a][0] = w[0]; k[a][1] = w[1];
          ke[a] = p.ks[row * 2 + (b >> 1)];
        }
      } else {
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(c + 32 * g + 8 * b);
          k[a][2 * g] = w[0];
          k[a][2 * g + 1] = w[1];
        }
      }
    }
    const int64_t row = (b >= 2 ? h1.row - 16 : h0.row) + 8 * b;
    const uint8_t* c = p.vc + row * (D / 2) + (D == 128 ? 4 * m : 4 * (m >> 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const unsigned*>(c + i * (D / 2));
    constexpr int SB = FMT == SVDQ_FMT_MXFP4_G32 ? D / 32 : D / 32;   // scale bytes of a row
    const u32x4* sv = reinterpret_cast<const u32x4*>(p.vs + row * SB);
#pragma unroll
    for (int i = 0; i < NS; ++i) vsc[i] = sv[i];
    if constexpr (FMT == SVDQ_FMT_INT4_G64) {
      const u32x4* sk = reinterpret_cast<const u32x4*>(p.ks + row * SB);
#pragma unroll
      for (int i = 0; i < NS; ++i) ksc[i] = sk[i];
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

template <int FMT>
__device__ __forceinline__ u32x4 query_order(u32x4 q) {
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) return q;
  return u32x4{low_halves(q[0], q[1]), low_halves(q[2], q[3]), high_halves(q[0], q[1]), high_halves(q[2], q[3])};
}

// 8 keys' scales of one head row group, fp32 (INT4) or converter scales (MXFP4)
template <int DT, int FMT, int D>
__device__ __forceinline__ float value_scale(const u32x4* sc, int i, int g) {
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
    const unsigned w = D == 128 ? sc[i / 4][i % 4] >> (8 * g) : sc[0][i / 2] >> (16 * (i % 2) + 8 * g);
    return mx_scale<DT>(w & 255u);
  } else {
    const unsigned w = D == 128 ? sc[i / 4][i % 4] >> (16 * g) : sc[0][i / 2] >> (16 * (i % 2));
    return h2f<SVDQ_F16>(w & 0xFFFFu);
  }
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

// the same for INT4, from fp8 words: c s rounded to 16 bits once (fp32 product
// for bf16, f16 product for f16)
template <int DT, bool HI>
__device__ __forceinline__ void value_pair_int4(const unsigned* v8, const float* s, u32x4* f0, u32x4* f1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SVDQ_BF16) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v8[2 * i], 512.0f, HI);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v8[2 * i + 1], 512.0f, HI);
      (*f0)[i] = pack2<DT>(a[0] * s[2 * i], b[0] * s[2 * i + 1]);
      (*f1)[i] = pack2<DT>(a[1] * s[2 * i], b[1] * s[2 * i + 1]);
    } else {
      const _Float16 s0 = (_Float16)s[2 * i], s1 = (_Float16)s[2 * i + 1];
      const f16x2 a = __builtin_bit_cast(f16x2, cvt_int4<DT, HI>(v8[2 * i])) * f16x2{s0, s0};
      const f16x2 b = __builtin_bit_cast(f16x2, cvt_int4<DT, HI>(v8[2 * i + 1])) * f16x2{s1, s1};
      const unsigned x0 = __builtin_bit_cast(unsigned, a), x1 = __builtin_bit_cast(unsigned, b);
      (*f0)[i] = low_halves(x0, x1);
      (*f1)[i] = high_halves(x0, x1);
    }
  }
}

// column of the result that lane row n of value tile x stands for
template <int FMT, int D>
__device__ __forceinline__ constexpr int value_col(int n, int x) {
  // MXFP4: tiles are the lane's elements in order; INT4: nibbles 0 2 4 6 1 3 5 7
  constexpr int PER = D / 16;
  if (FMT == SVDQ_FMT_MXFP4_G32) return PER * n + x;
  return PER * n + (PER == 8 ? (x < 4 ? 2 * x : 2 * (x - 4) + 1) : (x < 2 ? 2 * x : 2 * (x - 2) + 1));
}

template <int DT, int FMT, int D>
struct Rows16 {
  static constexpr int NJ = D / 32, NX = D / 16;
  u32x4 q[NJ];
  f32x4 o[NX];
  float base, sum;          // reference and this lane's part of the sum
  int low, high;            // keys that this lane's row sees

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int x = 0; x < NX; ++x) o[x] = f32x4{0, 0, 0, 0};
    base = LOWEST;
    sum = 0.0f;
  }

  // all: every row sees every key of the tile and both pages are there
  __device__ __forceinline__ void step(const AttnParams& p, const Tile32<FMT, D>& t, int token, int len, bool all, int lane) {
    const int b = lane >> 4;
    float s[8];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      f32x4 acc = {0, 0, 0, 0};
      if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
        const float e = mx_scale<DT>(t.ke[a]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][j], e), q[j], acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * a + i] = acc[i];
      } else {
        acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][0], 0.0f), q[0], acc);
        acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][1], 0.0f), q[1], acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * a + i] = acc[i] * value_scale<DT, FMT, D>(t.ksc, 4 * a + i, 0);
        if constexpr (D == 128) {
          acc = f32x4{0, 0, 0, 0};
          acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][2], 0.0f), q[2], acc);
          acc = mfma16<DT>(key_frag<DT, FMT>(t.k[a][3], 0.0f), q[3], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[4 * a + i] = __builtin_fmaf(acc[i], value_scale<DT, FMT, D>(t.ksc, 4 * a + i, 1), s[4 * a + i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= p.c;
    const bool there = b >= 2 ? t.ok1 : t.ok0;
    if (!all) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = token + 8 * b + i;
        s[i] = there && k >= low && k < high ? s[i] : -__builtin_inff();
      }
    }
    float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    top = quad_max(top) - p_shift<DT>();
    if (__any(top > base + SLACK)) {
      const float next = fmaxf(base, top), alpha = exp2_hw(base - next);
      base = next;
      sum *= alpha;
#pragma unroll
      for (int x = 0; x < NX; ++x) o[x] *= alpha;
    }
    u32x4 pf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = exp2_hw(s[2 * i] - base), p1 = exp2_hw(s[2 * i + 1] - base);
      sum += p0 + p1;
      pf[i] = pack2<DT>(p0, p1);
    }
    // values: keys past the end or on a missing page hold anything, a NaN
    // included, and must be zero, not only weighted with zero
    float sc[8];
    const int m = lane & 15;
    const int g = FMT == SVDQ_FMT_MXFP4_G32 ? (D == 128 ? m >> 2 : m >> 3) : (D == 128 ? m >> 3 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sc[i] = value_scale<DT, FMT, D>(t.vsc, i, g);
      if (DT == SVDQ_F16 && FMT == SVDQ_FMT_INT4_G64) sc[i] = fminf(sc[i], 9352.0f);   // 7 x 9352 is the last that f16 holds
    }
    if (!all) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] = there && token + 8 * b + i < len ? sc[i] : 0.0f;
    }
    unsigned v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = D == 128 ? t.v[i] : t.v[i] >> (16 * (m & 1));
    u32x4 f0, f1;
    if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
      value_pair_mx<DT, 0>(v, sc, &f0, &f1);
      o[0] = mfma16<DT>(f0, pf, o[0]);
      o[1] = mfma16<DT>(f1, pf, o[1]);
      value_pair_mx<DT, 1>(v, sc, &f0, &f1);
      o[2] = mfma16<DT>(f0, pf, o[2]);
      o[3] = mfma16<DT>(f1, pf, o[3]);
      if constexpr (D == 128) {
        value_pair_mx<DT, 2>(v, sc, &f0, &f1);
        o[4] = mfma16<DT>(f0, pf, o[4]);
        o[5] = mfma16<DT>(f1, pf, o[5]);
        value_pair_mx<DT, 3>(v, sc, &f0, &f1);
        o[6] = mfma16<DT>(f0, pf, o[6]);
        o[7] = mfma16<DT>(f1, pf, o[7]);
      }
    } else {
      constexpr int H = D == 128 ? 4 : 2;       // tiles of even nibbles
      unsigned w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = int4_even(v[i]);
      value_pair_int4<DT, false>(w, sc, &f0, &f1);
      o[0] = mfma16<DT>(f0, pf, o[0]);
      o[1] = mfma16<DT>(f1, pf, o[1]);
      if constexpr (D == 128) {
        value_pair_int4<DT, true>(w, sc, &f0, &f1);
        o[2] = mfma16<DT>(f0, pf, o[2]);
        o[3] = mfma16<DT>(f1, pf, o[3]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = int4_odd(v[i]);
      value_pair_int4<DT, false>(w, sc, &f0, &f1);
      o[H] = mfma16<DT>(f0, pf, o[H]);
      o[H + 1] = mfma16<DT>(f1, pf, o[H + 1]);
      if constexpr (D == 128) {
        value_pair_int4<DT, true>(w, sc, &f0, &f1);
        o[6] = mfma16<DT>(f0, pf, o[6]);
        o[7] = mfma16<DT>(f1, pf, o[7]);
      }
    }
  }
};

// the 16 rows of row tile rt: rows are (query, head of the group), head fastest
struct TileRange {
  int first, last;          // queries of the first and last row
  int from, to;             // keys that any row sees, `from` rounded down to 32
  int all_low, all_high;    // keys that every row sees
  int n;                    // chunks in use
  __device__ __forceinline__ TileRange(const AttnParams& p, const Request& r, int rt, int rows_per_tile) {
    first = rt * rows_per_tile / p.group;
    last = min(r.rows - 1, (rt * rows_per_tile + rows_per_tile - 1) / p.group);
    from = r.low(p, first) & ~31;
    to = r.high(p, last);
    all_low = r.low(p, last);
    all_high = r.high(p, first);
    n = to > from ? (to - from + p.chunk - 1) / p.chunk : 0;
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
__global__ __launch_bounds__(256, 2) void k_attn16(AttnParams p) {
  constexpr int NJ = D / 32, NX = D / 16, PER = D / 16, LD = D + 4;
  __shared__ float so[4][16][LD];
  __shared__ float sb[4][16], ss[4][16];
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  // workgroup -> (request, head, row tile, chunk), chunk fastest
  unsigned id = blockIdx.x;
  const int split = int(id % unsigned(p.splits));
  const int64_t item = int64_t(id / unsigned(p.splits));
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
  w.clear();
  w.low = r.low(p, qi);
  w.high = row < rows ? r.high(p, qi) : 0;
  {
    const uint16_t* q = p.q + (r.first + qi) * p.qt + int64_t(qh) * p.qh;
#pragma unroll
    for (int j = 0; j < NJ; ++j) w.q[j] = query_order<FMT>(*reinterpret_cast<const u32x4*>(q + frag_dim<FMT, D>(j, b)));
  }
  const int from = range.from + split * p.chunk, to = min(range.to, from + p.chunk);
  const int32_t* table = p.table + int64_t(req) * p.table_stride;
  const int last_col = (r.len - 1) >> p.page_shift;
  int token = from + 32 * wave;
  Tile32<FMT, D> cur, next;
  if (token < to) {
    cur.load(p, half_tile(p, table, token, last_col, h), half_tile(p, table, token + 16, last_col, h), lane);
    for (;;) {
      const int after = token + 128;
      if (after < to) next.load(p, half_tile(p, table, after, last_col, h), half_tile(p, table, after + 16, last_col, h), lane);
      const bool all = token >= range.all_low && token + 32 <= range.all_high && cur.ok0 && cur.ok1;
      w.step(p, cur, token, r.len, all, lane);
      if (after >= to) break;
      cur = next;
      token = after;
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
    const int64_t at = (item * p.splits + split) * 16 + orow;
    float* y = p.part + at * D + d;
#pragma unroll
    for (int i = 0; i < PER; i += 4) *reinterpret_cast<f32x4*>(y + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
    if ((int(threadIdx.x) & 15) == 0) {
      float* bs = p.part + int64_t(gridDim.x) * 16 * D + at * 2;
      bs[0] = base;
      bs[1] = sum;
    }
    return;
  }
  const int64_t tok = r.first + row_o / p.group;
  const int head = h * p.group + row_o % p.group;
  const float inv = sum == 0.0f ? 0.0f : value_gain<DT, FMT>() / sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] *= inv;
  store_row<DT, D>(p, tok, head, d, f);
  if (p.lse && (int(threadIdx.x) & 15) == 0)
    p.lse[tok * p.q_heads + head] = sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0.69314718055994531f;
}

// Joins the chunks of an item, in chunk order.
template <int DT, int FMT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnParams p) {
  constexpr int PER = D / 16;
  unsigned id = blockIdx.x;
  const int64_t item = id;
  const int rt = int(id % unsigned(p.row_tiles));
  id /= unsigned(p.row_tiles);
  const int h = int(id % unsigned(p.heads)), req = int(id / unsigned(p.heads));
  const Request r(p, req);
  const int rows = r.rows * p.group;
  const int row = rt * 16 + (int(threadIdx.x) >> 4), d = (int(threadIdx.x) & 15) * PER;
  if (row >= rows) return;
  const TileRange range(p, r, rt, 16);
  if (range.n <= 1) return;
  const int64_t at = item * p.splits * 16 + (int(threadIdx.x) >> 4);
  const float* bs = p.part + int64_t(gridDim.x) * p.splits * 16 * D;
  float base = LOWEST;
  for (int s = 0; s < range.n; ++s) base = fmaxf(base, bs[(at + s * 16) * 2]);
  float sum = 0.0f, f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = 0.0f;
  for (int s = 0; s < range.n; ++s) {
    const float a = exp2_hw(bs[(at + s * 16) * 2] - base);
    sum += a * bs[(at + s * 16) * 2 + 1];
    const float* y = p.part + (at + s * 16) * D + d;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(y + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[i + e] += a * v[e];
    }
  }
  const int64_t tok = r.first + row / p.group;
  const int head = h * p.group + row % p.group;
  const float inv = sum == 0.0f ? 0.0f : value_gain<DT, FMT>() / sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] *= inv;
  store_row<DT, D>(p, tok, head, d, f);
  if (p.lse && (int(threadIdx.x) & 15) == 0)
    p.lse[tok * p.q_heads + head] = sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0.69314718055994531f;
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

// How a call is cut: row tiles per request and head, and key chunks.  `most`
// bounds the chunks of any call with these requests, rows and lengths, whatever
// its window, so that one workspace serves them all.
struct Cut {
  int64_t items;
  int row_tiles, splits, chunk, most;
};

svdq_status check_attn(const svdq_attn_desc* d, const svdq_kv_cache* c) {
  if (!d || d->requests < 0 || d->tokens < 0 || !dtype_ok(d->dtype) || (d->flags & ~unsigned(SVDQ_ATTN_CAUSAL)) != 0u ||
      d->max_q < 0 || d->max_kv < 0 || d->window < 0 || d->table_stride < 0 || d->q_heads < 1)
    return SVDQ_ERR_INVALID_ARG;
  if (!(d->scale == d->scale)) return SVDQ_ERR_INVALID_ARG;
  const svdq_status st = check_cache(c);
  if (st != SVDQ_OK) return st;
  return d->q_heads % c->heads != 0 ? SVDQ_ERR_SHAPE : SVDQ_OK;
}

svdq_status cut_of(const svdq_attn_desc* d, const svdq_kv_cache* c, Cut* out) {
  Cut t;
  const int64_t group = d->q_heads / c->heads;
  const int64_t max_q = d->max_q < d->tokens ? d->max_q : d->tokens;
  const int64_t tiles = ceil_div(max_q * group, 16);
  t.items = d->requests * c->heads * tiles;
  int64_t span = d->max_kv;
  const bool causal = (d->flags & SVDQ_ATTN_CAUSAL) != 0u;   // else a row sees up to the end, whatever its window
  if (causal && d->window > 0 && int64_t(d->window) + max_q < span) span = int64_t(d->window) + max_q;
  if (d->window > 0) span += 31;        // the first tile is rounded down to 32
  // Chunks of at least 128 keys (a tile for each wave), as many as fill the
  // chip about four workgroups deep.
  const int64_t want = ceil_div(int64_t(device_cus()) * 4, t.items > 0 ? t.items : 1);
  const int64_t all = ceil_div(int64_t(d->max_kv) + 31, 128), here = ceil_div(span, 128);
  const int64_t n = want < here ? want : here > 0 ? here : 1;
  const int64_t chunk = ceil_div(ceil_div(span > 0 ? span : 1, n), 128) * 128;
  t.splits = int(ceil_div(span > 0 ? span : 1, chunk));
  t.most = int(want < all ? want : all);
  t.chunk = int(chunk);
  t.row_tiles = int(tiles);
  if (t.items * t.most >= (int64_t(1) << 31)) return SVDQ_ERR_UNSUPPORTED;
  *out = t;
  return SVDQ_OK;
}

size_t part_bytes(const Cut& t, int splits, int D) {
  return splits > 1 ? size_t(t.items) * size_t(splits) * 16 * size_t(D + 2) * 4 : 0;
}

template <int DT, int FMT, int D>
void launch_attn(const AttnParams& p, const Cut& t, hipStream_t st) {
  k_attn16<DT, FMT, D><<<dim3(unsigned(t.items * t.splits)), 256, 0, st>>>(p);
  if (t.splits > 1) k_attn_join<DT, FMT, D><<<dim3(unsigned(t.items)), 256, 0, st>>>(p);
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
  if ((st = cut_of(d, c, &t)) != SVDQ_OK) return st;
  *bytes = part_bytes(t, t.most, c->head_dim);
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
  if ((st = cut_of(d, c, &t)) != SVDQ_OK) return st;
  const size_t need = part_bytes(t, t.splits, c->head_dim);
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
  p.tokens = d->tokens; p.table_stride = d->table_stride; p.n_pages = c->n_pages;
  p.requests = int32_t(d->requests); p.q_heads = d->q_heads; p.heads = c->heads; p.group = d->q_heads / c->heads;
  p.max_q = d->max_q; p.max_kv = d->max_kv; p.window = d->window;
  p.causal = (d->flags & SVDQ_ATTN_CAUSAL) != 0u;
  p.page_shift = page_shift(c->page_size);
  p.row_tiles = t.row_tiles; p.splits = t.splits; p.chunk = t.chunk;
  const bool mx = c->fmt == SVDQ_FMT_MXFP4_G32, bf = d->dtype == SVDQ_BF16;
  p.c = d->scale * 1.44269504088896341f * (mx && !bf ? 8.0f : 1.0f);
  if (bf) {
    if (mx) launch_attn<SVDQ_BF16, SVDQ_FMT_MXFP4_G32>(p, t, c->head_dim, stream);
    else launch_attn<SVDQ_BF16, SVDQ_FMT_INT4_G64>(p, t, c->head_dim, stream);
  } else {
    if (mx) launch_attn<SVDQ_F16, SVDQ_FMT_MXFP4_G32>(p, t, c->head_dim, stream);
    else launch_attn<SVDQ_F16, SVDQ_FMT_INT4_G64>(p, t, c->head_dim, stream);
  }
  return launch_ok();
}
