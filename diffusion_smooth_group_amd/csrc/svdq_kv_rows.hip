// svdq_kv_rows.hip -- gfx950 (MI355X) kernels on the rows around the 4-bit
// key/value cache: norm and rotation of q and k (and its gradient), the
// quantizing append, the read-back, and the tables of a step.  The attention
// over the cache is in svdq_kv_attn.hip; include/svdq_kv.h is the C ABI.
//
// Row kernels: a head's row of D elements is shared by L = pow2 >= D / 16
// neighbouring lanes.  Lane j holds two pieces of 8 elements, [8j, 8j + 8)
// and the same in the row's second half, so both rotations (pairs (2i, 2i + 1)
// and (i, i + D/2)) stay inside a lane and every access is 16 bytes; the sums
// of a row are log2(L) lane exchanges.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "svdq_kv_common.h"

namespace {

using namespace svdq_kv;

struct RowOp {             // one operand of a row kernel (device view)
  const uint16_t* x;       // rows in
  uint16_t* y;             // rows out (null: into the cache)
  const uint16_t* g;       // gradient of the rows out (backward)
  const uint16_t* w;       // norm weight or null
  int64_t xt, xh, yt, yh, gt, gh;   // token / head strides
  int32_t heads;
  int32_t norm, rope;
};

struct RowParams {
  RowOp op[3];             // q, k, v
  uint8_t *codes[3], *scales[3];    // cache buffers of operands 1 (K) and 2 (V)
  const float *cos, *sin;
  const int32_t* positions;
  const int32_t* slots;
  float* part[2];          // backward: partial weight gradients [gridDim.x][D] of q, k
  int64_t tokens, n_positions, n_slots;
  float eps;
  int32_t D, page_shift, cache_heads;
  int32_t skip;            // first operand of grid row 0
};

// values 2i, 2i + 1 of a 16-byte piece
template <int DT>
__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = h2f<DT>(v[i] & 0xFFFFu);
    f[2 * i + 1] = h2f<DT>(v[i] >> 16);
  }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
  return v;
}

// Sum over the L lanes of a row (L <= 16): every lane ends with the same bits,
// each step adds the same two numbers in both lanes.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m *= 2) v += __shfl_xor(v, m);
  return v;
}
template <int N>
__device__ __forceinline__ float lane_max(float v) {
#pragma unroll
  for (int m = 1; m < N; m *= 2) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// cos and sin of the lane's 8 pairs.  Halves: pair i = (i, i + D/2), the
// lane's pairs are [8j, 8j + 8).  Else pairs are neighbours: [4j, 4j + 4) in
// the first piece, [D/4 + 4j, ..) in the second.
__device__ __forceinline__ void load_angles(const RowParams& p, int64_t pos, int j, bool halves, float* c, float* s) {
  if (pos < 0 || pos >= p.n_positions) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s[i] = __builtin_nanf("");
    return;
  }
  const int half = p.D / 2;
  const int64_t at = pos * half;
  const int a0 = halves ? 8 * j : 4 * j, a1 = halves ? 8 * j + 4 : p.D / 4 + 4 * j;
  const f32x4 c0 = *reinterpret_cast<const f32x4*>(p.cos + at + a0), c1 = *reinterpret_cast<const f32x4*>(p.cos + at + a1);
  const f32x4 s0 = *reinterpret_cast<const f32x4*>(p.sin + at + a0), s1 = *reinterpret_cast<const f32x4*>(p.sin + at + a1);
#pragma unroll
  for (int i = 0; i < 4; ++i) { c[i] = c0[i]; c[4 + i] = c1[i]; s[i] = s0[i]; s[4 + i] = s1[i]; }
}

// (u, v) turned by the angle of cos c, sin n; BACK: by its negative
template <bool BACK>
__device__ __forceinline__ void turn(float* u, float* v, float c, float n) {
  const float x = *u, y = *v;
  *u = BACK ? __builtin_fmaf(y, n, x * c) : __builtin_fmaf(-y, n, x * c);
  *v = BACK ? __builtin_fmaf(-x, n, y * c) : __builtin_fmaf(x, n, y * c);
}
template <bool BACK>
__device__ __forceinline__ void rotate(float* a, float* b, const float* c, const float* s, bool halves) {
  if (halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn<BACK>(&a[i], &b[i], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn<BACK>(&a[2 * i], &a[2 * i + 1], c[i], s[i]);
      turn<BACK>(&b[2 * i], &b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  }
}
// sum over i of a[i] x[i] + b[i] y[i], two chains
__device__ __forceinline__ float dot16(const float* a, const float* x, const float* b, const float* y) {
  float s = a[0] * x[0], t = b[0] * y[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) { s = __builtin_fmaf(a[i], x[i], s); t = __builtin_fmaf(b[i], y[i], t); }
  return s + t;
}

// 8 nibbles of the MXFP4 piece f under the group's e8m0 exponent e: the
// converter rounds to nearest even and saturates at 6 (as the activation
// kernel's codes)
__device__ __forceinline__ unsigned mx_codes(const float* f, int e) {
  const float scale = __uint_as_float(unsigned(e) << 23);
  unsigned w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], scale, 3);
  return w;
}

// smallest biased exponent e with 2^(e - 127) >= fl32(a / 6); 0 for a = 0.  At
// most 252, so that a held value (6 x 2^125 at most) is finite in bf16 too.
__device__ __forceinline__ int mx_exponent(float a) {
  const float t = a / 6.0f;
  const unsigned b = __float_as_uint(t);
  if (t == 0.0f) return 0;
  const int e = int(b >> 23) + ((b & 0x7FFFFFu) != 0u ? 1 : 0);
  return e > 252 ? 252 : e;
}

// INT4: code = sign, |clamp(rint(fl32(v / s)), 7)|; a zero scale holds zeros
__device__ __forceinline__ unsigned int4_codes(const float* f, float s) {
  unsigned w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = s == 0.0f ? 0.0f : fminf(rintf(fabsf(f[i]) / s), 7.0f);
    const unsigned m = unsigned(r);
    w |= (m | ((f[i] < 0.0f && m != 0u) ? 8u : 0u)) << (4 * i);
  }
  return w;
}

// The lane's two pieces into the cache.  L lanes per row, lane j of it.
template <int FMT, int L>
__device__ __forceinline__ void store_quantized(const RowParams& p, int which, int64_t slot, int h, int j, float* a, float* b) {
  const int D = L * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {        // a NaN is held as zero
    a[i] = a[i] != a[i] ? 0.0f : a[i];
    b[i] = b[i] != b[i] ? 0.0f : b[i];
  }
  float ma = 0.0f, mb = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) { ma = fmaxf(ma, fabsf(a[i])); mb = fmaxf(mb, fabsf(b[i])); }
  const int64_t page = slot >> p.page_shift, in = slot & ((int64_t(1) << p.page_shift) - 1);
  const int64_t row = (((page * p.cache_heads + h) << p.page_shift) + in);
  uint8_t* code = p.codes[which] + row * (D / 2);
  unsigned wa, wb;
  if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
    ma = lane_max<4>(ma);
    mb = lane_max<4>(mb);
    const int ea = mx_exponent(ma), eb = mx_exponent(mb);
    wa = mx_codes(a, ea);
    wb = mx_codes(b, eb);
    if ((j & 3) == 0) {
      uint8_t* sc = p.scales[which] + row * (D / 32);
      sc[j / 4] = uint8_t(ea);
      sc[D / 64 + j / 4] = uint8_t(eb);
    }
  } else {
    if constexpr (L == 4) ma = mb = fmaxf(ma, mb);   // one group of 64
    ma = lane_max<L>(ma);
    mb = lane_max<L>(mb);
    const _Float16 ha = _Float16(fminf(ma / 7.0f, 65504.0f)), hb = _Float16(fminf(mb / 7.0f, 65504.0f));
    wa = int4_codes(a, float(ha));
    wb = int4_codes(b, float(hb));
    if (j == 0) {
      uint16_t* sc = reinterpret_cast<uint16_t*>(p.scales[which]) + row * (D / 64);
      sc[0] = __builtin_bit_cast(uint16_t, ha);
      if constexpr (L == 8) sc[1] = __builtin_bit_cast(uint16_t, hb);
    }
  }
  *reinterpret_cast<unsigned*>(code + 4 * j) = wa;
  *reinterpret_cast<unsigned*>(code + D / 4 + 4 * j) = wb;
}

// Norm, rotation and store of rows.  Grid: x over rows (token-major), y over
// operands.  FMT < 0: every operand goes to 16-bit rows; else operands 1 and 2
// go to the cache (L is 4 or 8 there).
//   y = R(angle) (x w / sqrt(mean x^2 + eps)), 7 operations an element against
// 4 bytes: bound by memory.  One row a lane group and no loop: enough workgroups
// are in flight to cover the loads (two rows a thread: 25.7 us, four 27.6, one
// 24.8), and streaming stores leave the caches to the angles (27.6 us without).
// 4608 tokens x (24 + 24) heads of 128, bf16: 23.5 us, 4.9 TB/s, the rate of a
// large copy.  The append of the same keys and values (MXFP4): 19 us; with norm,
// rotation and the queries in the same launch, 30 us, 4.3 TB/s.
template <int DT, int L, int FMT>
__global__ __launch_bounds__(256) void k_rows(RowParams p) {
  const int which = int(blockIdx.y) + p.skip;
  const RowOp& o = p.op[which];
  constexpr int RPB = 256 / L;
  const int j = int(threadIdx.x) % L;
  const int64_t rows = p.tokens * o.heads, row = int64_t(blockIdx.x) * RPB + int(threadIdx.x) / L;
  const bool lane_on = 16 * j < p.D;             // D / 16 need not be a power of two
  const bool halves = (o.rope & 2) != 0;
  // Lanes past the last row take part in the lane exchanges with zeros and
  // store nothing: a row's lanes are on or off together.
  const bool on = row < rows && lane_on;
  const unsigned r32 = unsigned(row);            // rows < 2^31 (checked by the host)
  const int64_t t = row < rows ? int64_t(r32 / unsigned(o.heads)) : 0;
  const int h = row < rows ? int(r32 % unsigned(o.heads)) : 0;
  const int half = p.D / 2;
  float a[8], b[8];
  u32x4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
  if (on) {
    const uint16_t* x = o.x + t * o.xt + h * o.xh + 8 * j;
    va = *reinterpret_cast<const u32x4*>(x);
    vb = *reinterpret_cast<const u32x4*>(x + half);
  }
  unpack8<DT>(va, a);
  unpack8<DT>(vb, b);
  if (o.norm) {
    const float s = row_sum<L>(dot16(a, a, b, b));
    const float r = 1.0f / sqrtf(s / float(p.D) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) { a[i] *= r; b[i] *= r; }
    if (o.w && lane_on) {
      float wa[8], wb[8];
      unpack8<DT>(*reinterpret_cast<const u32x4*>(o.w + 8 * j), wa);
      unpack8<DT>(*reinterpret_cast<const u32x4*>(o.w + half + 8 * j), wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) { a[i] *= wa[i]; b[i] *= wb[i]; }
    }
  }
  if (o.rope && on) {
    float c[8], s[8];
    load_angles(p, p.positions ? int64_t(p.positions[t]) : t, j, halves, c, s);
    rotate<false>(a, b, c, s, halves);
  }
  if (FMT < 0 || which == 0) {
    if (on) {
      uint16_t* y = o.y + t * o.yt + h * o.yh + 8 * j;
      __builtin_nontemporal_store(pack8<DT>(a), reinterpret_cast<u32x4*>(y));
      __builtin_nontemporal_store(pack8<DT>(b), reinterpret_cast<u32x4*>(y + half));
    }
  } else {
    if constexpr (FMT >= 0 && (L == 4 || L == 8)) {
      // the 16-bit value that the row kernel would have stored is what is held
      unpack8<DT>(pack8<DT>(a), a);
      unpack8<DT>(pack8<DT>(b), b);
      const int64_t slot = on ? int64_t(p.slots[t]) : -1;
      if (slot >= 0 && slot < p.n_slots) store_quantized<FMT, L>(p, which, slot, h, j, a, b);
    }
  }
}

// Gradient of norm and rotation.  Every lane keeps its 16 columns' weight
// gradient over the rows it walks; the workgroup adds its row groups in a
// fixed order and leaves one partial row of D sums.
//   u = w R^T g, n = x r: dx = r (u - n mean(u n)), dw = sum R^T g n
// 6 bytes an element: bound by memory, less closely than the forward because a
// lane's sums and the next row take 144 registers (three waves a SIMD).  4607
// tokens x (24 + 24) heads of 128, bf16: 38 us, 4.5 TB/s, and 5 us for the sums.
// 2048 x (20 + 20) heads of 64, f16: 12 and 4 us, 2.7 TB/s: 640 groups of rows on
// 384 workgroups are two rounds for some, and the sums cost as much as a row.
template <int DT, int L>
__global__ __launch_bounds__(256) void k_rows_grad(RowParams p) {
  const int which = int(blockIdx.y);
  const RowOp& o = p.op[which];
  constexpr int RPB = 256 / L;
  const int j = int(threadIdx.x) % L, grp = int(threadIdx.x) / L;
  const bool lane_on = 16 * j < p.D;
  const bool halves = (o.rope & 2) != 0;
  const int half = p.D / 2;
  const int64_t rows = p.tokens * o.heads;
  float wa[8], wb[8], da[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { wa[i] = wb[i] = 1.0f; da[i] = db[i] = 0.0f; }
  if (o.norm && o.w && lane_on) {
    unpack8<DT>(*reinterpret_cast<const u32x4*>(o.w + 8 * j), wa);
    unpack8<DT>(*reinterpret_cast<const u32x4*>(o.w + half + 8 * j), wb);
  }
  const float inv_d = 1.0f / float(p.D);
  // The next row's values and position are requested before this row's work.
  struct Row {
    u32x4 va, vb, ua, ub;
    int64_t t, pos;
    int h;
    bool on;
  } next;
  auto request = [&](int64_t base) {
    const int64_t row = base + grp;
    next.on = row < rows && lane_on;
    const unsigned r32 = unsigned(row < rows ? row : 0);
    next.t = int64_t(r32 / unsigned(o.heads));
    next.h = int(r32 % unsigned(o.heads));
    next.va = next.vb = next.ua = next.ub = u32x4{0, 0, 0, 0};
    next.pos = next.t;
    if (next.on) {
      const uint16_t* g = o.g + next.t * o.gt + next.h * o.gh + 8 * j;
      next.ua = *reinterpret_cast<const u32x4*>(g);
      next.ub = *reinterpret_cast<const u32x4*>(g + half);
      if (o.norm) {
        const uint16_t* x = o.x + next.t * o.xt + next.h * o.xh + 8 * j;
        next.va = *reinterpret_cast<const u32x4*>(x);
        next.vb = *reinterpret_cast<const u32x4*>(x + half);
      }
      if (p.positions) next.pos = p.positions[next.t];
    }
  };
  const int64_t step = int64_t(gridDim.x) * RPB;
  int64_t base = int64_t(blockIdx.x) * RPB;
  if (base < rows) request(base);
  for (; base < rows; base += step) {
    const u32x4 va = next.va, vb = next.vb, ua = next.ua, ub = next.ub;
    const int64_t t = next.t, pos = next.pos;
    const int h = next.h;
    const bool on = next.on;
    float c[8], sn[8];
    if (o.rope && on) load_angles(p, pos, j, halves, c, sn);
    if (base + step < rows) request(base + step);
    float a[8], b[8], ga[8], gb[8];
    unpack8<DT>(ua, ga);
    unpack8<DT>(ub, gb);
    if (o.rope && on) rotate<true>(ga, gb, c, sn, halves);
    if (o.norm) {
      unpack8<DT>(va, a);
      unpack8<DT>(vb, b);
      const float s = row_sum<L>(dot16(a, a, b, b));
      const float r = 1.0f / sqrtf(s / float(p.D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= r;                       // x r, the unit row
        b[i] *= r;
        da[i] = __builtin_fmaf(ga[i], a[i], da[i]);
        db[i] = __builtin_fmaf(gb[i], b[i], db[i]);
        ga[i] *= wa[i];
        gb[i] *= wb[i];
      }
      // dx = r u - x r (r mean(u x r))
      const float back = r * (row_sum<L>(dot16(ga, a, gb, b)) * inv_d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ga[i] = __builtin_fmaf(-a[i], back, r * ga[i]);
        gb[i] = __builtin_fmaf(-b[i], back, r * gb[i]);
      }
    }
    if (on) {
      uint16_t* y = o.y + t * o.yt + h * o.yh + 8 * j;
      __builtin_nontemporal_store(pack8<DT>(ga), reinterpret_cast<u32x4*>(y));
      __builtin_nontemporal_store(pack8<DT>(gb), reinterpret_cast<u32x4*>(y + half));
    }
  }
  if (!o.norm || p.part[which] == nullptr) return;
  // row groups of a wave: lane exchanges; waves: through LDS
#pragma unroll
  for (int m = L; m < 64; m *= 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { da[i] += __shfl_xor(da[i], m); db[i] += __shfl_xor(db[i], m); }
  }
  __shared__ float red[4][16 * L];
  const int wave = int(threadIdx.x) / 64, lane = int(threadIdx.x) % 64;
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { red[wave][8 * j + i] = da[i]; red[wave][8 * L + 8 * j + i] = db[i]; }
  }
  __syncthreads();
  for (int d = int(threadIdx.x); d < p.D; d += 256) {
    const int at = d < half ? d : 8 * L + d - half;
    p.part[which][int64_t(blockIdx.x) * p.D + d] = (red[0][at] + red[1][at]) + (red[2][at] + red[3][at]);
  }
}

// Weight gradient = sum of the partial rows, in a fixed order: 64 groups of 16
// lanes (a column each) walk the partials, four loads in flight each, then meet
// in LDS.
__global__ __launch_bounds__(1024) void k_rows_grad_sum(const float* pq, const float* pk, float* dq, float* dk, int parts, int D) {
  const float* part = blockIdx.y == 0 ? pq : pk;
  float* out = blockIdx.y == 0 ? dq : dk;
  if (out == nullptr) return;
  const int lane = int(threadIdx.x) % 16, grp = int(threadIdx.x) / 16, col = int(blockIdx.x) * 16 + lane;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (part != nullptr) {
    int i = grp;
    for (; i + 192 < parts; i += 256) {
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += part[int64_t(i + 64 * u) * D + col];
    }
    for (; i < parts; i += 64) s[0] += part[int64_t(i) * D + col];
  }
  __shared__ float red[64][17];
  red[grp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (threadIdx.x >= 256) return;
  float v = (red[grp][lane] + red[grp + 16][lane]) + (red[grp + 32][lane] + red[grp + 48][lane]);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  __shared__ float last[4][16];
  if ((int(threadIdx.x) & 63) < 16) last[int(threadIdx.x) / 64][lane] = v;
  __syncthreads();
  if (threadIdx.x < 16) out[col] = (last[0][lane] + last[1][lane]) + (last[2][lane] + last[3][lane]);
}

struct ReadParams {
  const uint8_t *codes[2], *scales[2];
  uint16_t* y[2];
  int64_t yt[2], yh[2];
  const int32_t* slots;
  int64_t n, n_slots;
  int32_t heads, page_shift;
};

// Cache rows as 16-bit values: a lane turns 8 bytes of codes into 32 bytes.
// Bound by the writes: 4608 slots x 24 heads of 128, K and V: 15 us, 4.8 TB/s.
template <int DT, int FMT, int D>
__global__ __launch_bounds__(256) void k_read(ReadParams p) {
  constexpr int L = D / 16, RPB = 256 / L;
  const int which = p.y[0] == nullptr ? 1 : int(blockIdx.y);
  const int j = int(threadIdx.x) % L;
  const int64_t row = int64_t(blockIdx.x) * RPB + int(threadIdx.x) / L;
  if (row >= p.n * p.heads) return;
  const unsigned r32 = unsigned(row);
  const int64_t t = int64_t(r32 / unsigned(p.heads));
  const int h = int(r32 % unsigned(p.heads));
  const int64_t slot = int64_t(p.slots[t]);
  u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (slot >= 0 && slot < p.n_slots) {
    const int64_t page = slot >> p.page_shift, in = slot & ((int64_t(1) << p.page_shift) - 1);
    const int64_t at = (((page * p.heads + h) << p.page_shift) + in);
    const u32x2 w = *reinterpret_cast<const u32x2*>(p.codes[which] + at * (D / 2) + 8 * j);
    float f[16];
    float s;
    if constexpr (FMT == SVDQ_FMT_MXFP4_G32) {
      const int e = p.scales[which][at * (D / 32) + j / 2];
      s = e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(unsigned(e) << 23);   // 2^(e - 127)
    } else {
      s = h2f<SVDQ_F16>(reinterpret_cast<const uint16_t*>(p.scales[which])[at * (D / 64) + j / 4]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const unsigned c = (w[i / 8] >> (4 * (i % 8))) & 15u, m = c & 7u;
      // E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6: (2 + m % 2) 2^(m / 2 - 2), m / 2 for m < 2
      float v;
      if constexpr (FMT == SVDQ_FMT_MXFP4_G32)
        v = m < 2u ? 0.5f * float(m) : __uint_as_float(((m / 2u + 126u) << 23) | ((m & 1u) << 22));
      else
        v = float(m);
      f[i] = (c & 8u ? -v : v) * s;
    }
    lo = pack8<DT>(f);
    hi = pack8<DT>(f + 8);
  }
  uint16_t* y = p.y[which] + t * p.yt[which] + h * p.yh[which] + 16 * j;
  __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(y));
  __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(y + 8));
}

// ------------------------------------------------------------ step tables
struct PlanParams {
  const int32_t *past, *fresh, *free_pages, *free_count;
  int32_t *block_table, *q_start, *kv_len, *slots, *positions, *free_left, *missing;
  int64_t tokens, table_stride, free_capacity;
  int32_t requests, page_shift;
};

constexpr int PLAN_TOKENS = 1024;   // new tokens a workgroup maps

// last request whose first item is at or before i (first[] rises from 0): the
// one that item i belongs to, since empty requests start where the next does
__device__ __forceinline__ int last_at_or_before(const int* first, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Every workgroup scans all requests (two loads each, from L2 after the first
// workgroup) into LDS: prefix sums of the new tokens and of the new pages.  It
// then maps its own PLAN_TOKENS tokens and its share of the new pages by binary
// search; workgroup 0 writes the totals.  Latency is all: 512 requests of one
// token 5.8 us, 61 prompts of 79000 tokens in all 6.2 us, most of it the scan's
// loads and the launch itself.  No
// workgroup reads what another writes.
__global__ __launch_bounds__(256) void k_plan(PlanParams p) {
  extern __shared__ int lds[];
  int* qs = lds;                        // [requests + 1] first token of each request
  int* ps = lds + p.requests + 1;       // [requests + 1] first new page of each request
  __shared__ int wave_q[4], wave_p[4];
  const int tid = int(threadIdx.x), B = p.requests, page = 1 << p.page_shift;
  int base_q = 0, base_p = 0;
  for (int at = 0; at < B; at += 256) {
    const int r = at + tid;
    int nq = 0, np = 0;
    if (r < B) {
      const int past = max(p.past[r], 0);
      nq = max(p.fresh[r], 0);
      np = int((unsigned(past) + unsigned(nq) + unsigned(page - 1)) >> p.page_shift) -
           int((unsigned(past) + unsigned(page - 1)) >> p.page_shift);
    }
    int sq = nq, sp = np;               // inclusive scan over the wave
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const int uq = __shfl_up(sq, m), up = __shfl_up(sp, m);
      if ((tid & 63) >= m) { sq += uq; sp += up; }
    }
    if ((tid & 63) == 63) { wave_q[tid / 64] = sq; wave_p[tid / 64] = sp; }
    __syncthreads();
    int oq = base_q, op = base_p;
    for (int w = 0; w < 4; ++w) {
      if (w < tid / 64) { oq += wave_q[w]; op += wave_p[w]; }
      base_q += wave_q[w];
      base_p += wave_p[w];
    }
    if (r < B) { qs[r] = oq + sq - nq; ps[r] = op + sp - np; }
    __syncthreads();
  }
  if (tid == 0) { qs[B] = base_q; ps[B] = base_p; }
  __syncthreads();
  const int count = max(0, min(*p.free_count, int(min(p.free_capacity, int64_t(0x7FFFFFFF)))));
  if (blockIdx.x == 0) {
    for (int r = tid; r <= B; r += 256) p.q_start[r] = qs[r];
    for (int r = tid; r < B; r += 256) p.kv_len[r] = max(p.past[r], 0) + (qs[r + 1] - qs[r]);
    if (tid == 0) {
      *p.free_left = count - min(count, base_p);
      *p.missing = max(base_p - count, 0);
    }
  }
  // table entries: a thread per new page of the step
  for (int k = int(blockIdx.x) * 256 + tid; k < base_p; k += int(gridDim.x) * 256) {
    const int r = last_at_or_before(ps, B, k), past = max(p.past[r], 0);
    const int64_t col = int64_t((unsigned(past) + unsigned(page - 1)) >> p.page_shift) + (k - ps[r]);
    if (col >= 0 && col < p.table_stride)
      p.block_table[int64_t(r) * p.table_stride + col] = k < count ? p.free_pages[count - 1 - k] : -1;
  }
  // tokens
  const int64_t from = int64_t(blockIdx.x) * PLAN_TOKENS;
  for (int64_t t = from + tid; t < min(from + PLAN_TOKENS, p.tokens); t += 256) {
    int slot = -1, pos = 0;
    if (t < base_q) {
      const int r = last_at_or_before(qs, B, int(t)), past = max(p.past[r], 0);
      pos = past + int(t) - qs[r];
      const int col = pos >> p.page_shift, before = int((unsigned(past) + unsigned(page - 1)) >> p.page_shift);
      int pg = -1;
      if (col >= 0 && col < p.table_stride) {
        if (col < before) {
          pg = p.block_table[int64_t(r) * p.table_stride + col];
        } else {
          const int k = ps[r] + col - before;
          pg = k >= 0 && k < count ? p.free_pages[count - 1 - k] : -1;
        }
      }
      // a page that no cache has (slots are 31-bit) must not wrap to one that it has
      slot = pg < 0 || pg > (0x7FFFFFFF >> p.page_shift) ? -1 : (pg << p.page_shift) + (pos & (page - 1));
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

struct ReleaseParams {
  const int32_t* done;
  int32_t *block_table, *kv_len, *free_pages, *free_count;
  int64_t table_stride, free_capacity;
  int32_t requests, page_shift;
};

// One workgroup: requests in order, the pages of a request in order, which is the
// order that they have in the list.  Bound by latency, a load of done[r] and then
// of the table a request: 512 requests, every fourth ended with 63 pages, 127 us.
__global__ __launch_bounds__(256) void k_release(ReleaseParams p) {
  __shared__ int wave_n[4];
  const int tid = int(threadIdx.x);
  int64_t at = max(0, *p.free_count);
  for (int r = 0; r < p.requests; ++r) {
    if (p.done[r] == 0) continue;       // the same for every lane
    const int64_t len = int64_t(max(p.kv_len[r], 0));
    const int64_t n = min((len + (int64_t(1) << p.page_shift) - 1) >> p.page_shift, p.table_stride);
    int32_t* row = p.block_table + int64_t(r) * p.table_stride;
    for (int64_t c = 0; c < n; c += 256) {
      const int pg = c + tid < n ? row[c + tid] : -1;
      const unsigned long long b = __ballot(pg >= 0);
      if ((tid & 63) == 0) wave_n[tid / 64] = __popcll(b);
      __syncthreads();
      int64_t to = at + __popcll(b & ((1ull << (tid & 63)) - 1ull));
      for (int w = 0; w < 4; ++w) {
        if (w < tid / 64) to += wave_n[w];
        at += wave_n[w];
      }
      if (pg >= 0 && to < p.free_capacity) p.free_pages[to] = pg;
      if (c + tid < n) row[c + tid] = -1;
      __syncthreads();
    }
    if (tid == 0) p.kv_len[r] = 0;
  }
  if (tid == 0) *p.free_count = int(min(at, p.free_capacity));
}

// ---------------------------------------------------------------- host side
int row_lanes(int D) {
  int l = 1;
  while (16 * l < D) l *= 2;
  return l;
}

constexpr unsigned QK_FLAGS = unsigned(SVDQ_QK_NORM) | unsigned(SVDQ_QK_ROPE) | unsigned(SVDQ_QK_ROPE_HALVES);

svdq_status check_desc(const svdq_qk_desc* d) {
  if (!d || d->tokens < 0 || !dtype_ok(d->dtype) || (d->flags & ~QK_FLAGS) != 0u) return SVDQ_ERR_INVALID_ARG;
  if (d->head_dim < 16 || d->head_dim > 256 || d->head_dim % 16 != 0) return SVDQ_ERR_SHAPE;
  if ((d->flags & SVDQ_QK_NORM) != 0u && !(d->eps >= 0.0f)) return SVDQ_ERR_INVALID_ARG;
  if ((d->flags & SVDQ_QK_ROPE) == 0u) return (d->flags & SVDQ_QK_ROPE_HALVES) != 0u ? SVDQ_ERR_INVALID_ARG : SVDQ_OK;
  if (!d->cos || !d->sin || d->n_positions < 0) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(d->cos, 16) || !aligned(d->sin, 16) || d->head_dim % 16 != 0) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

svdq_status check_weights(const svdq_qk_desc* d) {
  if ((d->flags & SVDQ_QK_NORM) == 0u) return SVDQ_OK;
  return (d->wq && !aligned(d->wq, 16)) || (d->wk && !aligned(d->wk, 16)) ? SVDQ_ERR_SHAPE : SVDQ_OK;
}

RowOp row_op(const svdq_qk_desc* d, const svdq_heads* in, const svdq_heads* out, const void* w, bool key_or_query) {
  RowOp o = {};
  if (!in) return o;
  o.x = static_cast<const uint16_t*>(in->data);
  o.xt = in->token_stride; o.xh = in->head_stride;
  o.heads = in->heads;
  if (out) {
    o.y = static_cast<uint16_t*>(out->data);
    o.yt = out->token_stride; o.yh = out->head_stride;
  }
  if (key_or_query) {
    o.norm = (d->flags & SVDQ_QK_NORM) != 0u;
    o.w = o.norm ? static_cast<const uint16_t*>(w) : nullptr;
    o.rope = (d->flags & SVDQ_QK_ROPE) == 0u ? 0 : (d->flags & SVDQ_QK_ROPE_HALVES) != 0u ? 3 : 1;
  }
  return o;
}

void fill_desc(RowParams* p, const svdq_qk_desc* d) {
  p->cos = d->cos; p->sin = d->sin;
  p->positions = d->positions;
  p->tokens = d->tokens;
  p->n_positions = d->n_positions;
  p->eps = d->eps;
  p->D = d->head_dim;
}

template <int DT>
void launch_rows(const RowParams& p, int lanes, int64_t rows, int ops, hipStream_t st) {
  const dim3 grid(unsigned(ceil_div(rows, 256 / lanes)), unsigned(ops));
  switch (lanes) {
    case 1: k_rows<DT, 1, -1><<<grid, 256, 0, st>>>(p); break;
    case 2: k_rows<DT, 2, -1><<<grid, 256, 0, st>>>(p); break;
    case 4: k_rows<DT, 4, -1><<<grid, 256, 0, st>>>(p); break;
    case 8: k_rows<DT, 8, -1><<<grid, 256, 0, st>>>(p); break;
    default: k_rows<DT, 16, -1><<<grid, 256, 0, st>>>(p); break;
  }
}

template <int DT, int FMT>
void launch_append(const RowParams& p, int lanes, int64_t rows, int ops, hipStream_t st) {
  const dim3 grid(unsigned(ceil_div(rows, 256 / lanes)), unsigned(ops));
  if (lanes == 4) k_rows<DT, 4, FMT><<<grid, 256, 0, st>>>(p);
  else k_rows<DT, 8, FMT><<<grid, 256, 0, st>>>(p);
}

// Workgroups an operand: q's and k's together are three a compute unit, as many
// as the registers hold at once (4607 tokens, 24 heads of 128: 43 us; 512
// blocks, a second round, 50; 1024 47; other shapes were not measured).  The
// weight gradients' partial rows, and with them the workspace, go by this number.
constexpr int64_t GRAD_BLOCKS = 384;
int grad_blocks(int64_t rows, int lanes) {
  const int64_t blocks = ceil_div(rows, 256 / lanes);
  return int(blocks < 1 ? 1 : blocks > GRAD_BLOCKS ? GRAD_BLOCKS : blocks);
}

template <int DT>
void launch_grad(const RowParams& p, int lanes, int blocks, int ops, hipStream_t st) {
  const dim3 grid{unsigned(blocks), unsigned(ops), 1u};
  switch (lanes) {
    case 1: k_rows_grad<DT, 1><<<grid, 256, 0, st>>>(p); break;
    case 2: k_rows_grad<DT, 2><<<grid, 256, 0, st>>>(p); break;
    case 4: k_rows_grad<DT, 4><<<grid, 256, 0, st>>>(p); break;
    case 8: k_rows_grad<DT, 8><<<grid, 256, 0, st>>>(p); break;
    default: k_rows_grad<DT, 16><<<grid, 256, 0, st>>>(p); break;
  }
}

// rows below 2^31, and their lanes within a launch
svdq_status check_rows(const svdq_qk_desc* d, int64_t heads) {
  const int lanes = row_lanes(d->head_dim);
  return product_below(d->tokens, heads, 1, int64_t(1) << 31) < 0 || product_below(d->tokens, heads, lanes, MAX_THREADS - 256 * lanes) < 0
             ? SVDQ_ERR_UNSUPPORTED
             : SVDQ_OK;
}

template <int DT, int FMT>
void launch_read(const ReadParams& p, int D, int outs, hipStream_t st) {
  const dim3 grid(unsigned(ceil_div(p.n * p.heads, 256 / (D / 16))), unsigned(outs));
  if (D == 64) k_read<DT, FMT, 64><<<grid, 256, 0, st>>>(p);
  else k_read<DT, FMT, 128><<<grid, 256, 0, st>>>(p);
}

}  // namespace

extern "C" svdq_status svdq_kv_cache_size(int64_t n_pages, int32_t page_size, int32_t heads, int32_t head_dim,
                                          svdq_format fmt, size_t* code_bytes, size_t* scale_bytes) {
  if (!code_bytes || !scale_bytes) return SVDQ_ERR_INVALID_ARG;
  svdq_kv_cache c = {};
  c.n_pages = n_pages; c.page_size = page_size; c.heads = heads; c.head_dim = head_dim; c.fmt = fmt;
  const svdq_status st = check_cache_shape(&c);
  if (st != SVDQ_OK) return st;
  const size_t rows = size_t(n_pages) * size_t(page_size) * size_t(heads);
  *code_bytes = rows * size_t(head_dim) / 2;
  *scale_bytes = fmt == SVDQ_FMT_MXFP4_G32 ? rows * size_t(head_dim / 32) : rows * size_t(head_dim / 64) * 2;
  return SVDQ_OK;
}

extern "C" svdq_status svdq_qk_norm_rope(const svdq_qk_desc* d, const svdq_heads* q, const svdq_heads* k,
                                         const svdq_heads* q_out, const svdq_heads* k_out, hipStream_t stream) {
  svdq_status st = check_desc(d);
  if (st != SVDQ_OK) return st;
  if (!q || !k || !q_out || !k_out || q->heads < 1 || k->heads < 0) return SVDQ_ERR_INVALID_ARG;
  if (q_out->heads != q->heads || k_out->heads != k->heads) return SVDQ_ERR_SHAPE;
  if (d->tokens == 0) return SVDQ_OK;
  if ((st = check_weights(d)) != SVDQ_OK || (st = check_heads(q, d->head_dim)) != SVDQ_OK ||
      (st = check_heads(q_out, d->head_dim)) != SVDQ_OK || (st = check_rows(d, q->heads)) != SVDQ_OK)
    return st;
  if (k->heads > 0 && ((st = check_heads(k, d->head_dim)) != SVDQ_OK || (st = check_heads(k_out, d->head_dim)) != SVDQ_OK ||
                       (st = check_rows(d, k->heads)) != SVDQ_OK))
    return st;
  RowParams p = {};
  fill_desc(&p, d);
  p.op[0] = row_op(d, q, q_out, d->wq, true);
  p.op[1] = row_op(d, k, k_out, d->wk, true);
  const int64_t most = d->tokens * (q->heads > k->heads ? q->heads : k->heads);
  const int lanes = row_lanes(d->head_dim), ops = k->heads > 0 ? 2 : 1;
  if (d->dtype == SVDQ_BF16) launch_rows<SVDQ_BF16>(p, lanes, most, ops, stream);
  else launch_rows<SVDQ_F16>(p, lanes, most, ops, stream);
  return launch_ok();
}

extern "C" svdq_status svdq_qk_backward_workspace(const svdq_qk_desc* d, int32_t q_heads, int32_t k_heads, size_t* bytes) {
  svdq_status st = check_desc(d);
  if (st != SVDQ_OK) return st;
  if (!bytes || q_heads < 1 || k_heads < 0) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_rows(d, q_heads > k_heads ? q_heads : k_heads)) != SVDQ_OK) return st;
  const int lanes = row_lanes(d->head_dim);
  const int blocks = grad_blocks(d->tokens * (q_heads > k_heads ? q_heads : k_heads), lanes);
  *bytes = size_t(2) * size_t(blocks) * size_t(d->head_dim) * 4;
  return SVDQ_OK;
}

extern "C" svdq_status svdq_qk_norm_rope_backward(const svdq_qk_desc* d, const svdq_heads* q, const svdq_heads* k,
                                                  const svdq_heads* gq, const svdq_heads* gk, const svdq_heads* dq,
                                                  const svdq_heads* dk, float* dwq, float* dwk, void* ws,
                                                  size_t ws_bytes, hipStream_t stream) {
  svdq_status st = check_desc(d);
  if (st != SVDQ_OK) return st;
  if (!q || !k || !gq || !gk || !dq || !dk || q->heads < 1 || k->heads < 0) return SVDQ_ERR_INVALID_ARG;
  if (gq->heads != q->heads || dq->heads != q->heads || gk->heads != k->heads || dk->heads != k->heads) return SVDQ_ERR_SHAPE;
  const int D = d->head_dim;
  size_t need = 0;
  if ((st = svdq_qk_backward_workspace(d, q->heads, k->heads, &need)) != SVDQ_OK) return st;
  const bool norm = (d->flags & SVDQ_QK_NORM) != 0u && d->tokens > 0;
  RowParams p = {};
  int blocks = 0;
  if (d->tokens > 0) {
    if ((st = check_weights(d)) != SVDQ_OK) return st;
    for (const svdq_heads* v : {q, gq, dq})
      if ((st = check_heads(v, D)) != SVDQ_OK) return st;
    for (const svdq_heads* v : {k, gk, dk})
      if (k->heads > 0 && (st = check_heads(v, D)) != SVDQ_OK) return st;
    if ((st = check_rows(d, q->heads)) != SVDQ_OK || (st = check_rows(d, k->heads)) != SVDQ_OK) return st;
    if (norm && (dwq || dwk)) {
      if (!ws) return SVDQ_ERR_INVALID_ARG;
      if (ws_bytes < need) return SVDQ_ERR_CAPACITY;
      if (!aligned(ws, 16)) return SVDQ_ERR_INVALID_ARG;
    }
    fill_desc(&p, d);
    p.op[0] = row_op(d, q, dq, d->wq, true);
    p.op[1] = row_op(d, k, dk, d->wk, true);
    p.op[0].g = static_cast<const uint16_t*>(gq->data);
    p.op[0].gt = gq->token_stride; p.op[0].gh = gq->head_stride;
    p.op[1].g = static_cast<const uint16_t*>(gk->data);
    p.op[1].gt = gk->token_stride; p.op[1].gh = gk->head_stride;
    const int lanes = row_lanes(D), ops = k->heads > 0 ? 2 : 1;
    blocks = grad_blocks(d->tokens * (q->heads > k->heads ? q->heads : k->heads), lanes);
    if (norm && dwq) p.part[0] = static_cast<float*>(ws);
    if (norm && dwk && k->heads > 0) p.part[1] = static_cast<float*>(ws) + int64_t(blocks) * D;
    if (d->dtype == SVDQ_BF16) launch_grad<SVDQ_BF16>(p, lanes, blocks, ops, stream);
    else launch_grad<SVDQ_F16>(p, lanes, blocks, ops, stream);
  }
  if (dwq || dwk) k_rows_grad_sum<<<dim3(unsigned(D / 16), 2), 1024, 0, stream>>>(p.part[0], p.part[1], dwq, dwk, blocks, D);
  return launch_ok();
}

extern "C" svdq_status svdq_kv_append(const svdq_qk_desc* d, const svdq_heads* q, const svdq_heads* k, const svdq_heads* v,
                                      const svdq_heads* q_out, const svdq_kv_cache* cache, const int32_t* slots,
                                      hipStream_t stream) {
  svdq_status st = check_desc(d);
  if (st != SVDQ_OK) return st;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_cache(cache)) != SVDQ_OK) return st;
  if (d->head_dim != cache->head_dim || k->heads != cache->heads || v->heads != cache->heads) return SVDQ_ERR_SHAPE;
  if (q && (q->heads < 1 || q_out->heads != q->heads)) return SVDQ_ERR_SHAPE;
  if (d->tokens == 0) return SVDQ_OK;
  if (!slots) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_weights(d)) != SVDQ_OK || (st = check_heads(k, d->head_dim)) != SVDQ_OK ||
      (st = check_heads(v, d->head_dim)) != SVDQ_OK || (st = check_rows(d, k->heads)) != SVDQ_OK)
    return st;
  if (q && ((st = check_heads(q, d->head_dim)) != SVDQ_OK || (st = check_heads(q_out, d->head_dim)) != SVDQ_OK ||
            (st = check_rows(d, q->heads)) != SVDQ_OK))
    return st;
  RowParams p = {};
  fill_desc(&p, d);
  p.op[0] = row_op(d, q, q_out, d->wq, true);
  p.op[1] = row_op(d, k, nullptr, d->wk, true);
  p.op[2] = row_op(d, v, nullptr, nullptr, false);
  p.codes[1] = static_cast<uint8_t*>(cache->k_codes);
  p.scales[1] = static_cast<uint8_t*>(cache->k_scales);
  p.codes[2] = static_cast<uint8_t*>(cache->v_codes);
  p.scales[2] = static_cast<uint8_t*>(cache->v_scales);
  p.slots = slots;
  p.n_slots = cache->n_pages * cache->page_size;
  p.page_shift = page_shift(cache->page_size);
  p.cache_heads = cache->heads;
  p.skip = q ? 0 : 1;
  const int heads = q && q->heads > k->heads ? q->heads : k->heads;
  const int lanes = d->head_dim / 16, ops = q ? 3 : 2;
  const int64_t most = d->tokens * heads;
  const bool mx = cache->fmt == SVDQ_FMT_MXFP4_G32;
  if (d->dtype == SVDQ_BF16) {
    if (mx) launch_append<SVDQ_BF16, SVDQ_FMT_MXFP4_G32>(p, lanes, most, ops, stream);
    else launch_append<SVDQ_BF16, SVDQ_FMT_INT4_G64>(p, lanes, most, ops, stream);
  } else {
    if (mx) launch_append<SVDQ_F16, SVDQ_FMT_MXFP4_G32>(p, lanes, most, ops, stream);
    else launch_append<SVDQ_F16, SVDQ_FMT_INT4_G64>(p, lanes, most, ops, stream);
  }
  return launch_ok();
}

extern "C" svdq_status svdq_kv_read(const svdq_kv_cache* cache, const int32_t* slots, int64_t n, svdq_dtype dtype,
                                    const svdq_heads* k_out, const svdq_heads* v_out, hipStream_t stream) {
  svdq_status st = check_cache(cache);
  if (st != SVDQ_OK) return st;
  if (n < 0 || !dtype_ok(dtype)) return SVDQ_ERR_INVALID_ARG;
  for (const svdq_heads* o : {k_out, v_out}) {
    if (o && o->heads != cache->heads) return SVDQ_ERR_SHAPE;
    if (o && n > 0 && (st = check_heads(o, cache->head_dim)) != SVDQ_OK) return st;
  }
  if (n == 0 || (!k_out && !v_out)) return SVDQ_OK;
  if (!slots) return SVDQ_ERR_INVALID_ARG;
  if (product_below(n, cache->heads, 1, int64_t(1) << 31) < 0 ||
      product_below(n, cache->heads, cache->head_dim / 16, MAX_THREADS - 4096) < 0)
    return SVDQ_ERR_UNSUPPORTED;
  ReadParams p = {};
  p.codes[0] = static_cast<const uint8_t*>(cache->k_codes);
  p.scales[0] = static_cast<const uint8_t*>(cache->k_scales);
  p.codes[1] = static_cast<const uint8_t*>(cache->v_codes);
  p.scales[1] = static_cast<const uint8_t*>(cache->v_scales);
  const svdq_heads* out[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i)
    if (out[i]) {
      p.y[i] = static_cast<uint16_t*>(out[i]->data);
      p.yt[i] = out[i]->token_stride;
      p.yh[i] = out[i]->head_stride;
    }
  p.slots = slots;
  p.n = n;
  p.n_slots = cache->n_pages * cache->page_size;
  p.heads = cache->heads;
  p.page_shift = page_shift(cache->page_size);
  const int outs = k_out && v_out ? 2 : 1, D = cache->head_dim;
  const bool mx = cache->fmt == SVDQ_FMT_MXFP4_G32;
  if (dtype == SVDQ_BF16) {
    if (mx) launch_read<SVDQ_BF16, SVDQ_FMT_MXFP4_G32>(p, D, outs, stream);
    else launch_read<SVDQ_BF16, SVDQ_FMT_INT4_G64>(p, D, outs, stream);
  } else {
    if (mx) launch_read<SVDQ_F16, SVDQ_FMT_MXFP4_G32>(p, D, outs, stream);
    else launch_read<SVDQ_F16, SVDQ_FMT_INT4_G64>(p, D, outs, stream);
  }
  return launch_ok();
}

extern "C" svdq_status svdq_kv_plan(const int32_t* past, const int32_t* fresh, int64_t requests, int32_t page_size,
                                    int64_t tokens, const int32_t* free_pages, const int32_t* free_count,
                                    int64_t free_capacity, int32_t* block_table, int64_t table_stride, int32_t* q_start,
                                    int32_t* kv_len, int32_t* slots, int32_t* positions, int32_t* free_left,
                                    int32_t* missing, hipStream_t stream) {
  if (requests < 0 || tokens < 0 || free_capacity < 0 || table_stride < 0 || page_shift(page_size) < 0) return SVDQ_ERR_INVALID_ARG;
  if (requests > SVDQ_KV_MAX_REQUESTS || tokens >= (int64_t(1) << 31)) return SVDQ_ERR_UNSUPPORTED;
  if (!q_start || !free_count || !free_left || !missing || free_left == free_count) return SVDQ_ERR_INVALID_ARG;
  if (requests > 0 && (!past || !fresh || !kv_len || (table_stride > 0 && !block_table))) return SVDQ_ERR_INVALID_ARG;
  if ((tokens > 0 && (!slots || !positions)) || (free_capacity > 0 && !free_pages)) return SVDQ_ERR_INVALID_ARG;
  // workgroups read the inputs while another writes: no output may be one of them
  struct Range {
    uintptr_t from, to;
    Range(const int32_t* p, int64_t n) : from(reinterpret_cast<uintptr_t>(p)), to(from + 4 * uintptr_t(n < (int64_t(1) << 40) ? n : int64_t(1) << 40)) {}
  };
  const int64_t cells = product_below(requests, table_stride, 1, int64_t(1) << 40);
  for (const Range out : {Range{q_start, requests + 1}, Range{kv_len, requests}, Range{slots, tokens}, Range{positions, tokens},
                          Range{free_left, 1}, Range{missing, 1}, Range{block_table, cells < 0 ? int64_t(1) << 40 : cells}})
    for (const Range in : {Range{past, requests}, Range{fresh, requests}, Range{free_pages, free_capacity}, Range{free_count, 1}})
      if (out.from < in.to && in.from < out.to) return SVDQ_ERR_INVALID_ARG;
  PlanParams p;
  p.past = past; p.fresh = fresh;
  p.free_pages = free_pages; p.free_count = free_count;
  p.block_table = block_table; p.q_start = q_start; p.kv_len = kv_len;
  p.slots = slots; p.positions = positions; p.free_left = free_left; p.missing = missing;
  p.tokens = tokens; p.table_stride = table_stride; p.free_capacity = free_capacity;
  p.requests = int32_t(requests); p.page_shift = page_shift(page_size);
  const int64_t by_tokens = ceil_div(tokens, PLAN_TOKENS);
  const unsigned grid = unsigned(by_tokens < 1 ? 1 : by_tokens);
  k_plan<<<grid, 256, unsigned(2 * (requests + 1) * 4), stream>>>(p);
  return launch_ok();
}

extern "C" svdq_status svdq_kv_release(const int32_t* done, int64_t requests, int32_t page_size, int32_t* block_table,
                                       int64_t table_stride, int32_t* kv_len, int32_t* free_pages, int32_t* free_count,
                                       int64_t free_capacity, hipStream_t stream) {
  if (requests < 0 || free_capacity < 0 || table_stride < 0 || page_shift(page_size) < 0 || !free_count) return SVDQ_ERR_INVALID_ARG;
  if (requests > SVDQ_KV_MAX_REQUESTS) return SVDQ_ERR_UNSUPPORTED;
  if (requests == 0) return SVDQ_OK;
  if (!done || !kv_len || (table_stride > 0 && !block_table) || (free_capacity > 0 && !free_pages)) return SVDQ_ERR_INVALID_ARG;
  ReleaseParams p;
  p.done = done;
  p.block_table = block_table; p.kv_len = kv_len; p.free_pages = free_pages; p.free_count = free_count;
  p.table_stride = table_stride; p.free_capacity = free_capacity;
  p.requests = int32_t(requests); p.page_shift = page_shift(page_size);
  k_release<<<1, 256, 0, stream>>>(p);
  return launch_ok();
}
