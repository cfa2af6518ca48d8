// svdq_image_attn.hip -- gfx950 (MI355X) cross attention to an encoder's 16-bit
// keys and values, and its gradient (include/svdq_image.h).
//
//   s_it = scale q_i . k_t,  p_it = exp(s_it - lse_i),  out_i = sum_t p_it v_t
//   dv_t = sum_i p_it g_i,   ds_it = p_it (g_i . v_t - delta_i),  delta_i = g_i . out_i
//   dq_i = scale sum_t ds_it k_t,  dk_t = scale sum_i ds_it q_i
//
// A pair is a request and a key head; its rows are (query, head of the group),
// heads fastest.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "svdq_image.h"
#include "svdq_image_cut.h"
#include "svdq_kv_common.h"

namespace {

using namespace svdq_kv;
using namespace svdq_image;

struct Rows {               // an operand of heads
  uint16_t* data;
  int64_t token, head;
};

struct CrossParams {
  Rows q, k, v, out, g, dq, dk, dv;
  float *lse, *delta, *part, *key_part;
  const int32_t *q_start, *k_start;
  const uint8_t* mask;
  int32_t tokens, states, max_q, max_k, q_heads, heads, group, pairs, D;
  int32_t row_slots, row_tiles, splits, chunk;
  int32_t key_tiles, row_splits, row_chunk;
  unsigned by_group;        // 2^32 / group, rounded up (group > 1)
  float c, scale;           // c = scale log2(e); forward: |scale|, and q's signs are turned
  unsigned turn;            // bits of two 16-bit values to turn
  bool past;                // rows of the result (out, dq) are whole lines

  // row / group: the product may be one too high
  __device__ __forceinline__ int token_of(int row) const {
    if (group == 1) return row;
    const int t = int(__umulhi(unsigned(row), by_group));
    return t * group > row ? t - 1 : t;
  }
};

constexpr float LOWEST = -3.0e38f;   // reference of a row that has seen no key
constexpr float LOG2E = 1.44269504088896341f;
// Elements of a row in LDS: 36, 52 or 72 words, so that eight rows' 16 bytes and
// four rows' 32 lie in banks of their own.
template <int DP>
constexpr int row_of() { return DP + (DP == 128 ? 16 : 8); }

template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A block of 16-bit values in LDS, four rows of 16 for every 16 lanes (lane i
// names row i / 4, columns 4 (i % 4) ..), transposed: lane i gets column i's
// four rows.
typedef short i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_turned(const uint16_t* at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(at)));
}
__device__ __forceinline__ u32x4 joined(u32x2 a, u32x2 b) { return u32x4{a[0], a[1], b[0], b[1]}; }

// The reads of N times M matrix instructions, R each time, run ahead of them:
// EXTRA and those of the first AHEAD, then R behind each (left alone, the compiler
// waits for nearly every read right where it is used).
template <int N, int R, int AHEAD, int M = 1, int EXTRA = 0>
__device__ __forceinline__ void reads_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * R + EXTRA, 0);
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, AHEAD * M, 0);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// NaN if either is one: one instruction for three, where fmaxf has to quiet its
// operands first.  A row with a NaN gives NaN by its probabilities.
__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// over the two lanes l, l ^ 32, and over the four l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float half_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float quad_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_max(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_sum(__uint_as_float(a[0]) + __uint_as_float(a[1]));
}

__device__ __forceinline__ float row_lse(float base, float sum) {
  return sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0.69314718055994531f;
}

// A row's reference is raised only when its maximum has passed it by 2^SLACK;
// between that no accumulator is touched.  f16: probabilities are held at 2^6 of
// their size, so that f16's subnormals start far below any that counts.
template <int DT>
constexpr float p_shift() { return DT == SVDQ_F16 ? 6.0f : 0.0f; }
constexpr float SLACK = 8.0f;

// f16, gradient: ds is rounded under a power of two, `gain`, that is lowered
// where the row's (or state's) largest passes 2^15, so that all but what is
// 2^-21 below the largest of its sum keeps f16's 11 bits.  top: largest |ds|.
__device__ __forceinline__ float lower_gain(float top) {      // 2^7 / 2^floor(log2 top)
  return __uint_as_float((261u - (__float_as_uint(top) >> 23)) << 23);
}
constexpr float FIRST_GAIN = 0x1p100f, MOST = 0x1p15f;
constexpr float P_UP = 10.0f;           // f16, gradient of values: probabilities are held at 2^10 of their size

// the two 16-bit values of a word as floats
template <int DT>
__device__ __forceinline__ float first_half(unsigned w) { return h2f<DT>(w & 0xFFFFu); }
template <int DT>
__device__ __forceinline__ float second_half(unsigned w) {
  if constexpr (DT == SVDQ_BF16) return __uint_as_float(w & 0xFFFF0000u);
  else return h2f<DT>(w >> 16);
}

// 16-bit values of the columns of a 32 x 32 result (lane: column lane % 32, rows
// 8 (i / 4) + 4 (lane / 32) + i % 4) as they are stored: eight neighbouring rows,
// [16 y + 8 (lane / 32), ..), in w[4 y ..].
template <int DT>
__device__ __forceinline__ void columns(const f32x16& o, float by, unsigned* w) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const unsigned a0 = pack2<DT>(o[8 * y] * by, o[8 * y + 1] * by), a1 = pack2<DT>(o[8 * y + 2] * by, o[8 * y + 3] * by);
    const unsigned b0 = pack2<DT>(o[8 * y + 4] * by, o[8 * y + 5] * by), b1 = pack2<DT>(o[8 * y + 6] * by, o[8 * y + 7] * by);
    const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
    w[4 * y] = s0[0];
    w[4 * y + 1] = s1[0];
    w[4 * y + 2] = s0[1];
    w[4 * y + 3] = s1[1];
  }
}

// Rows on their way into LDS by buffer loads, whose addresses are a scalar base
// and a lane's fixed offset, and which give zeros for the offset OUT: no vector
// instruction a stage but for the last.
constexpr unsigned OUT = 0x80000000u;   // = the buffers' size: host checks keep every other offset below it
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t from, unsigned at, unsigned base = 0) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at, base, 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint16_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, OUT, 0x00020000);
}

// KT rows of an operand, 256 threads
template <int DP, int KT>
struct Piece {
  static constexpr int CH = DP / 8, N = KT * CH / 256;   // 16-byte pieces a row, pieces a thread
  static constexpr bool EVEN = 256 % CH == 0;            // a thread's pieces are whole rows apart: one offset, and a scalar for the rest
  static constexpr int LD = row_of<DP>();
  static_assert(KT * CH % 256 == 0, "whole pieces");
  u32x4 v[N];
  unsigned off[EVEN ? 1 : N], step;
  static __device__ __forceinline__ int row(int tid, int i) { return EVEN ? tid / CH + 256 / CH * i : (tid + 256 * i) / CH; }
  static __device__ __forceinline__ int col(int tid, int i) { return (EVEN ? tid : tid + 256 * i) % CH * 8; }
  // rows `stride` elements apart
  __device__ __forceinline__ void rows(int64_t stride, int D, int tid) {
    step = EVEN ? unsigned(256 / CH) * unsigned(stride) * 2u : 0u;
#pragma unroll
    for (int i = 0; i < (EVEN ? 1 : N); ++i)
      off[i] = col(tid, i) < D ? unsigned(row(tid, i)) * unsigned(stride) * 2u + unsigned(col(tid, i)) * 2u : OUT;
  }
  // the `n` first rows from `base` on; zeros behind them
  __device__ __forceinline__ void load(const uint16_t* base, int n, int tid) {
    const __amdgpu_buffer_rsrc_t from = buffer(base);
    if (n >= KT) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = load16(from, off[EVEN ? 0 : i], i * step);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = load16(from, row(tid, i) < n ? off[EVEN ? 0 : i] : OUT, i * step);
    }
  }
  __device__ __forceinline__ void write(uint16_t* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + row(tid, i) * LD + col(tid, i)) = v[i];
  }
  // rows whose bit in `see` is not set become zeros
  __device__ __forceinline__ void hide(uint64_t see, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!((see >> row(tid, i)) & 1u)) v[i] = u32x4{0, 0, 0, 0};
  }
};

// The same for rows (query, head of a group): every piece has its own offset.
template <int DP, int KT>
struct RowPiece {
  static constexpr int CH = DP / 8, N = KT * CH / 256, LD = row_of<DP>();
  static_assert(KT * CH % 256 == 0, "whole pieces");
  u32x4 v[N];
  unsigned off[N];
  static __device__ __forceinline__ int row(int tid, int i) { return (tid + 256 * i) / CH; }
  static __device__ __forceinline__ int col(int tid, int i) { return (tid + 256 * i) % CH * 8; }
  __device__ __forceinline__ void load(const uint16_t* base, int n, int tid) {
    const __amdgpu_buffer_rsrc_t from = buffer(base);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load16(from, n >= KT || row(tid, i) < n ? off[i] : OUT);
  }
  __device__ __forceinline__ void write(uint16_t* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + row(tid, i) * LD + col(tid, i)) = v[i];
  }
};

// The 128 rows of a tile, by way of LDS: in memory they are whole lines (8 lanes a
// row of 64), as operands and results 32 bytes of every row at a time, for which the
// memory system takes longer (dq, q, g and out so: 2 x 4096 rows, 10 heads of 64,
// over 77: 20.3 us, 16 of them without any key, and 16.4 by way of LDS; 1023 rows
// over 2049, 32 heads of 128: 256 and 226).
template <int DP>
struct TileRows {
  static constexpr int CH = DP / 8, N = 128 * CH / 256, LD = row_of<DP>();
  u32x4 v[N];
  __device__ __forceinline__ void load(const CrossParams& p, const CrossRange& r, const Rows& from, int first, int h, int tid) {
    const int rows = r.rows * p.group;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int rw = first + (tid + 256 * i) / CH, d = (tid + 256 * i) % CH * 8;
      v[i] = u32x4{0, 0, 0, 0};
      if (rw < rows && d < p.D) {
        const int t = p.token_of(rw);
        v[i] = *reinterpret_cast<const u32x4*>(from.data + (int64_t(r.q_first) + t) * from.token + (h * p.group + rw - t * p.group) * from.head + d);
      }
    }
  }
  __device__ __forceinline__ void write(uint16_t* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + (tid + 256 * i) / CH * LD + (tid + 256 * i) % CH * 8) = v[i];
  }
};

// A wave's 32 rows of a result (its transpose in o, times `by`) to memory by way of
// its part of LDS, which no other wave uses; past the caches where a row is whole
// 64-byte parts of lines (the call by itself: 2 x 4096 rows of 64 over 77, 11.3 us and
// 12.2 through them; in a view 64 bytes on 10.8 and 11.6, in one 16 bytes on 12.7 and
// 12.4; 2 x 16384 rows so 21.8 and 19.9; 3 x 2047 rows of 72 over 300 21.1 and 19.7).
// What reads the result next finds it in memory: with a 4-bit linear behind it 2 x 4096
// x 10 heads take 32.4 us and 33.9 through the caches, 2 x 16384 x 6 60.6 and 58.0, 4608
// x 24 of 128 over 512 79.7 and 77.6; with an elementwise pass no more than through them.
template <int DT, int DP>
__device__ __forceinline__ void store_rows(const CrossParams& p, const CrossRange& r, const Rows& to, uint16_t* lds, const f32x16* o, float by,
                                           int first, int h, int lane) {
  constexpr int CH = DP / 8, LD = row_of<DP>();
  const int m = lane & 31, hb = lane >> 5, rows = r.rows * p.group;
#pragma unroll
  for (int x = 0; x < DP / 32; ++x) {
    unsigned w[8];
    columns<DT>(o[x], by, w);
#pragma unroll
    for (int y = 0; y < 2; ++y)
      *reinterpret_cast<u32x4*>(lds + m * LD + 32 * x + 16 * y + 8 * hb) = u32x4{w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]};
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  auto put = [&](auto past) {
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; ++i) {
      const int row = (lane + 64 * i) / CH, d = (lane + 64 * i) % CH * 8, rw = first + row;
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * LD + d);
      if (rw >= rows || d >= p.D) continue;
      const int t = p.token_of(rw);
      u32x4* at = reinterpret_cast<u32x4*>(to.data + (int64_t(r.q_first) + t) * to.token + (h * p.group + rw - t * p.group) * to.head + d);
      if constexpr (decltype(past)::value) __builtin_nontemporal_store(v, at);
      else *at = v;
    }
    if constexpr (decltype(past)::value) asm volatile("" ::: "memory");    // else the last store of both forms becomes one
  };
  if (p.past) put(std::true_type());
  else put(std::false_type());
}

// bit t: state `at` + t of the request is seen, t < 64
__device__ __forceinline__ uint64_t seen(const CrossParams& p, const CrossRange& r, int at, int lane) {
  bool on = at + lane < r.keys;
  if (p.mask && on) on = p.mask[int64_t(r.k_first) + at + lane] != 0;
  return __ballot(on);
}

// Logits of 32 keys; what is not seen becomes -infinity.  see: the keys' bits from
// the lane half's first on.
__device__ __forceinline__ void hide16(f32x16& s, unsigned see) {
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = (see >> (8 * (i / 4) + i % 4)) & 1u ? s[i] : -__builtin_inff();
}

// A stage's keys as what their logits start from, 0 or (not seen) -infinity, or
// +infinity where they are multiplied by a negative number: the matrix core adds it,
// so that a mask costs no vector instruction.  By one wave.
__device__ __forceinline__ void leave_bias(float* bias, uint64_t see, float c, int lane) {
  bias[lane] = (see >> lane) & 1u ? 0.0f : c < 0.0f ? __builtin_inff() : -__builtin_inff();
}
// the 16 rows of a lane of a 32 x 32 result
__device__ __forceinline__ f32x16 rows16(const float* at, int hb) {
  f32x16 v;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(at + 8 * y + 4 * hb);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * y + i] = u[i];
  }
  return v;
}

// ------------------------------------------------------------ forward, many rows
// 32 rows a wave on 32x32x16: S^T = K Q^T leaves a lane with 16 of 32 keys of
// one row, two runs of four neighbours for every 16, which is the operand of
// O^T = V^T P^T as it stands; V^T comes out of LDS by transposing reads of four
// keys each.  128 rows a workgroup share stages of 64 keys, the next one in
// registers on its way; two workgroups a compute unit (three with heads up to 96: 3 x
// 2047 rows over 300, 16 heads of 72, 20 us against 25).  One request, 4608 rows over
// 4096, 24 heads of 128: 254 us, 910 TFLOP/s.  What bounds that: matrix and vector
// instructions of two waves a SIMD that hardly overlap (without the exponentials 256
// us of then 276, without the loads 254), and 864 tiles on 512 places.  Measured and
// not kept: the reference raised by the probabilities' sum instead of a maximum (the
// compiler copies the accumulators, 362 us against 298), the second tile's
// exponentials between the first's products (325 against 281), masks as the logits'
// start, from LDS (290 against 275 without a mask).
template <int DT, int DP>
__global__ __launch_bounds__(256, DP == 128 ? 2 : 3) void k_cross_rows(CrossParams p) {
  constexpr int KT = 64, NE = DP / 16, NX = DP / 32, LD = row_of<DP>();
  __shared__ __attribute__((aligned(16))) uint16_t sk[2][KT * LD];     // 128 rows' room in all
  __shared__ __attribute__((aligned(16))) uint16_t sv[2][KT * LD];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 31, hb = lane >> 5;
  const PairWork work(blockIdx.x, p.pairs, p.row_tiles * p.splits);
  const int tile = work.tile / p.splits, split = work.tile % p.splits, req = work.pair / p.heads, h = work.pair % p.heads;
  const CrossRange r(p, req);
  const int rows = r.rows * p.group;
  if (tile * 128 >= rows) return;
  const int chunks = (r.keys + p.chunk - 1) / p.chunk;
  if (split > 0 && split >= chunks) return;
  const int from = split * p.chunk, to = smaller(r.keys, from + p.chunk);
  const int row = tile * 128 + wave * 32 + m;
  const bool active = tile * 128 + wave * 32 < rows;     // of the wave
  const int64_t tok = int64_t(r.q_first) + (row < rows ? p.token_of(row) : 0);
  const int head = h * p.group + (row < rows ? row % p.group : 0);
  // the first keys are on their way before the rows
  const uint16_t* kp = p.k.data + (int64_t(r.k_first) + from) * p.k.token + h * p.k.head;
  const uint16_t* vp = p.v.data + (int64_t(r.k_first) + from) * p.v.token + h * p.v.head;
  Piece<DP, KT> pk, pv;
  pk.rows(p.k.token, p.D, tid);
  pv.rows(p.v.token, p.D, tid);
  uint64_t see = 0;
  if (from < to) {
    pk.load(kp, to - from, tid);
    pv.load(vp, to - from, tid);
    see = seen(p, r, from, lane);
  }
  u32x4 q[NE];
  {
    TileRows<DP> all;
    all.load(p, r, p.q, tile * 128, h, tid);
    all.write(sk[0], tid);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      q[e] = *reinterpret_cast<const u32x4*>(&sk[0][(wave * 32 + m) * LD + 16 * e + 8 * hb]);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[e][i] ^= p.turn;
    }
    __syncthreads();
  }
  f32x16 o[NX];
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[x][i] = 0.0f;
  float base = 0.0f, limit = -__builtin_inff(), sum = 0.0f;

  if (from < to) {
    if (see != ~uint64_t(0)) pv.hide(see, tid);
    pk.write(sk[0], tid);
    pv.write(sv[0], tid);
  }
  __syncthreads();
  int buf = 0;
  for (int at = from; at < to; at += KT) {
    const bool more = at + KT < to;
    uint64_t next = 0;
    if (more) {
      kp += KT * p.k.token;
      vp += KT * p.v.token;
      pk.load(kp, to - at - KT, tid);
      pv.load(vp, to - at - KT, tid);
    }
    if (see != 0 && active) {
      constexpr int T = 2;              // tiles of 32 keys
      f32x16 s[T];
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(&sk[buf][(32 * t + m) * LD + 16 * e + 8 * hb]);
          s[t] = mfma32<DT>(a, q[e], s[t]);
        }
        reads_ahead<NE, 1, DP == 96 ? 3 : 4>();
      }
      __builtin_amdgcn_s_setprio(0);
      if (see != ~uint64_t(0)) {
        hide16(s[0], unsigned(see) >> (4 * hb));
        hide16(s[1], unsigned(see >> 32) >> (4 * hb));
      }
      float top = s[0][0];
#pragma unroll
      for (int i = 1; i < 16 * T; ++i) top = maximum(top, s[i / 16][i % 16]);
      top = __builtin_fmaf(half_max(top), p.c, -base);
      if (__any(top > limit)) {
        const bool first_keys = limit < 0.0f, some = top > -__builtin_inff();
        const float up = first_keys ? (some ? top - p_shift<DT>() : 0.0f) : fmaxf(top - p_shift<DT>(), 0.0f);
        const float alpha = first_keys ? 1.0f : exp2_hw(-up);
        base += up;
        limit = first_keys && !some ? limit : p_shift<DT>() + SLACK;
        sum *= alpha;
#pragma unroll
        for (int x = 0; x < NX; ++x) o[x] *= alpha;
      }
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 16 * T; ++i) {
        s[i / 16][i % 16] = exp2_hw(__builtin_fmaf(s[i / 16][i % 16], p.c, -base));
        part += s[i / 16][i % 16];
      }
      sum += part;
      u32x4 pf[2 * T];
#pragma unroll
      for (int i = 0; i < 8 * T; ++i) pf[i / 4][i % 4] = pack2<DT>(s[i / 8][2 * i % 16], s[i / 8][2 * i % 16 + 1]);
      const int g = lane >> 4, i4 = lane & 15;
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int x = 0; x < NX; ++x) {
#pragma unroll
        for (int j = 0; j < 2 * T; ++j) {
          const uint16_t* b = &sv[buf][(16 * j + 4 * (g >> 1) + (i4 >> 2)) * LD + 32 * x + 16 * (g & 1) + 4 * (i4 & 3)];
          o[x] = mfma32<DT>(joined(read_turned(b), read_turned(b + 8 * LD)), pf[j], o[x]);
        }
      }
      reads_ahead<2 * T * NX, 2, DP == 96 ? 3 : 4>();
      __builtin_amdgcn_s_setprio(0);
    }
    if (more) {
      next = seen(p, r, at + KT, lane);
      if (next != ~uint64_t(0)) pv.hide(next, tid);
      pk.write(sk[buf ^ 1], tid);
      pv.write(sv[buf ^ 1], tid);
    }
    see = next;
    buf ^= 1;
    __syncthreads();
  }
  sum = half_sum(sum);
  if (limit < 0.0f) base = LOWEST;
  const bool whole = chunks <= 1;
  if (whole) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    store_rows<DT, DP>(p, r, p.out, sk[0] + wave * 32 * LD, o, inv, tile * 128 + wave * 32, h, lane);
    if (p.lse && row < rows && hb == 0) p.lse[tok * p.q_heads + head] = row_lse(base, sum);
    return;
  }
  if (row >= rows) return;
  const int64_t slot = (int64_t(work.pair) * p.row_slots + row) * p.splits + split;
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (32 * x + 8 * y + 4 * hb < p.D)
        *reinterpret_cast<f32x4*>(p.part + slot * p.D + 32 * x + 8 * y + 4 * hb) =
            f32x4{o[x][4 * y], o[x][4 * y + 1], o[x][4 * y + 2], o[x][4 * y + 3]};
  if (hb == 0)
    *reinterpret_cast<f32x2*>(p.part + int64_t(p.pairs) * p.row_slots * p.splits * p.D + slot * 2) = f32x2{base, sum};
}

// ------------------------------------------------------------- forward, few rows
// 16 rows a workgroup on 16x16x32, 32 keys a wave and step, straight from memory:
// K as operands, V through a piece of LDS of the wave's own for its transposition.
// The waves meet at the end.  The states' bytes bound it: 64 requests with up to 4096,
// 8 heads of 128 and four query heads each, 143 us, 4.8 TB/s; with the same loads
// through 64-bit addresses of their own it needed all registers of one wave a SIMD
// (184 us), at three waves with spills 159.
template <int DT, int DP>
__global__ __launch_bounds__(256, DP == 64 ? 4 : 2) void k_cross_few(CrossParams p) {
  constexpr int NJ = DP / 32, NX = DP / 16, LD = row_of<DP>(), CH = DP / 8, NV = 32 * CH / 64;
  __shared__ __attribute__((aligned(16))) uint16_t sv[4][32 * LD];
  __shared__ float wave_base[4][16], wave_sum[4][16];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 15, b = lane >> 4;
  const PairWork work(blockIdx.x, p.pairs, p.row_tiles * p.splits);
  const int tile = work.tile / p.splits, split = work.tile % p.splits, req = work.pair / p.heads, h = work.pair % p.heads;
  const CrossRange r(p, req);
  const int rows = r.rows * p.group;
  if (tile * 16 >= rows) return;
  const int chunks = (r.keys + p.chunk - 1) / p.chunk;
  if (split > 0 && split >= chunks) return;
  const int from = split * p.chunk, to = smaller(r.keys, from + p.chunk);
  const int row = tile * 16 + m;
  u32x4 q[NJ];
  {
    const int64_t tok = int64_t(r.q_first) + (row < rows ? p.token_of(row) : 0);
    const int head = h * p.group + (row < rows ? row % p.group : 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      q[j] = u32x4{0, 0, 0, 0};
      if (row < rows && 32 * j + 8 * b < p.D) {
        q[j] = *reinterpret_cast<const u32x4*>(p.q.data + tok * p.q.token + head * p.q.head + 32 * j + 8 * b);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[j][i] ^= p.turn;
      }
    }
  }
  f32x4 o[NX];
#pragma unroll
  for (int x = 0; x < NX; ++x) o[x] = f32x4{0, 0, 0, 0};
  float base = 0.0f, limit = -__builtin_inff(), sum = 0.0f;
  uint16_t* mine = sv[wave];
  u32x4 kf[2][NJ], vf[NV];
  bool on = false;
  // offsets of a lane's pieces; pieces of V are whole rows apart where CH divides 64
  constexpr bool EVEN = 64 % CH == 0;
  unsigned koff[NJ], voff[EVEN ? 1 : NV];
#pragma unroll
  for (int j = 0; j < NJ; ++j) koff[j] = 32 * j + 8 * b < p.D ? (unsigned(m) * unsigned(p.k.token) + unsigned(32 * j + 8 * b)) * 2u : OUT;
  auto vrow = [&](int i) { return EVEN ? lane / CH + 64 / CH * i : (lane + 64 * i) / CH; };
  auto vcol = [&](int i) { return (EVEN ? lane : lane + 64 * i) % CH * 8; };
#pragma unroll
  for (int i = 0; i < (EVEN ? 1 : NV); ++i)
    voff[i] = vcol(i) < p.D ? (unsigned(vrow(i)) * unsigned(p.v.token) + unsigned(vcol(i))) * 2u : OUT;
  const unsigned kstep = 32u * unsigned(p.k.token), vstep = EVEN ? unsigned(64 / CH) * unsigned(p.v.token) * 2u : 0u;
  auto fetch = [&](int at) {            // keys at .. at + 31, within [from, to)
    const __amdgpu_buffer_rsrc_t kb = buffer(p.k.data + (int64_t(r.k_first) + at) * p.k.token + h * p.k.head);
    const __amdgpu_buffer_rsrc_t vb = buffer(p.v.data + (int64_t(r.k_first) + at) * p.v.token + h * p.v.head);
    const int n = to - at;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int j = 0; j < NJ; ++j) kf[a][j] = load16(kb, 16 * a + m < n ? koff[j] : OUT, a * kstep);
#pragma unroll
    for (int i = 0; i < NV; ++i) vf[i] = load16(vb, vrow(i) < n ? voff[EVEN ? 0 : i] : OUT, i * vstep);
    on = lane < 32 && lane < n;
    if (p.mask && on) on = p.mask[int64_t(r.k_first) + at + lane] != 0;
  };
  int at = from + 32 * wave;
  if (at < to) fetch(at);
  for (; at < to; at += 128) {
    const unsigned see = unsigned(__ballot(on));
    f32x4 s[2];
    if (see != 0u) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int t = vrow(i), d = vcol(i);
        if (see != ~0u && !((see >> t) & 1u)) vf[i] = u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(mine + t * LD + d) = vf[i];
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        s[a] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[a] = mfma16<DT>(kf[a][j], q[j], s[a]);
      }
    }
    if (at + 128 < to) fetch(at + 128);
    if (see == 0u) continue;
    if (see != ~0u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i / 4][i % 4] = (see >> (16 * (i / 4) + 4 * b + i % 4)) & 1u ? s[i / 4][i % 4] : -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = maximum(top, s[i / 4][i % 4]);
    top = __builtin_fmaf(quad_max(top), p.c, -base);
    if (__any(top > limit)) {
      const bool first_keys = limit < 0.0f, some = top > -__builtin_inff();
      const float up = first_keys ? (some ? top - p_shift<DT>() : 0.0f) : fmaxf(top - p_shift<DT>(), 0.0f);
      const float alpha = first_keys ? 1.0f : exp2_hw(-up);
      base += up;
      limit = first_keys && !some ? limit : p_shift<DT>() + SLACK;
      sum *= alpha;
#pragma unroll
      for (int x = 0; x < NX; ++x) o[x] *= alpha;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i / 4][i % 4] = exp2_hw(__builtin_fmaf(s[i / 4][i % 4], p.c, -base));
      sum += s[i / 4][i % 4];
    }
    const u32x4 pf = {pack2<DT>(s[0][0], s[0][1]), pack2<DT>(s[0][2], s[0][3]), pack2<DT>(s[1][0], s[1][1]), pack2<DT>(s[1][2], s[1][3])};
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const uint16_t* t = mine + (4 * b + (m >> 2)) * LD + 16 * x + 4 * (m & 3);
      o[x] = mfma16<DT>(joined(read_turned(t), read_turned(t + 16 * LD)), pf, o[x]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  sum = quad_sum(sum);
  if (limit < 0.0f) base = LOWEST;
  float* mo = reinterpret_cast<float*>(mine);             // [16][DP], what was the wave's V
#pragma unroll
  for (int x = 0; x < NX; ++x) *reinterpret_cast<f32x4*>(mo + m * DP + 16 * x + 4 * b) = o[x];
  if (b == 0) {
    wave_base[wave][m] = base;
    wave_sum[wave][m] = sum;
  }
  __syncthreads();
  const bool whole = chunks <= 1;
  for (int u = tid; u < 16 * DP / 4; u += 256) {
    const int i = u / (DP / 4), d = u % (DP / 4) * 4, rw = tile * 16 + i;
    if (rw >= rows || d >= p.D) continue;
    float top = wave_base[0][i], total = 0.0f;
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, wave_base[w][i]);
    f32x4 f = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float a = exp2_hw(wave_base[w][i] - top);
      const f32x4 y = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(sv[w]) + i * DP + d);
      total += a * wave_sum[w][i];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += a * y[e];
    }
    const int64_t tok = int64_t(r.q_first) + rw / p.group;
    const int head = h * p.group + rw % p.group;
    if (whole) {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      *reinterpret_cast<u32x2*>(p.out.data + tok * p.out.token + head * p.out.head + d) =
          u32x2{pack2<DT>(f[0] * inv, f[1] * inv), pack2<DT>(f[2] * inv, f[3] * inv)};
      if (p.lse && d == 0) p.lse[tok * p.q_heads + head] = row_lse(top, total);
    } else {
      const int64_t slot = (int64_t(work.pair) * p.row_slots + rw) * p.splits + split;
      *reinterpret_cast<f32x4*>(p.part + slot * p.D + d) = f;
      if (d == 0) *reinterpret_cast<f32x2*>(p.part + int64_t(p.pairs) * p.row_slots * p.splits * p.D + slot * 2) = f32x2{top, total};
    }
  }
}

// Joins a row's chunks: a wave a row, 32 lanes for its columns, the two halves
// take every other chunk.  GRAD: partial rows of dq, which are only added.
template <int DT, bool GRAD>
__global__ __launch_bounds__(256) void k_cross_join(CrossParams p) {
  const int lane = int(threadIdx.x) & 63;
  const int64_t slot = int64_t(blockIdx.x) * 4 + (int(threadIdx.x) >> 6), slots = int64_t(p.pairs) * p.row_slots;
  if (slot >= slots) return;
  const int pair = int(slot / p.row_slots), row = int(slot % p.row_slots);
  const CrossRange r(p, pair / p.heads);
  if (row >= r.rows * p.group) return;
  const int n = (r.keys + p.chunk - 1) / p.chunk;
  if (n <= 1) return;
  const int d = (lane & 31) * 4, half = lane >> 5;
  const int64_t at = slot * p.splits;
  const float* y = p.part + at * p.D + (d < p.D ? d : 0);
  f32x4 f = {0, 0, 0, 0};
  float top = LOWEST, total = 0.0f;
  if constexpr (!GRAD) {
    const f32x2* bs = reinterpret_cast<const f32x2*>(p.part + slots * p.splits * p.D) + at;
    for (int i = lane; i < n; i += 64) top = fmaxf(top, bs[i][0]);
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
#pragma unroll 4
    for (int i = half; i < n; i += 2) {
      const f32x2 v = bs[i];
      const f32x4 u = *reinterpret_cast<const f32x4*>(y + int64_t(i) * p.D);
      const float a = exp2_hw(v[0] - top);
      total += a * v[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += a * u[e];
    }
    total = half_sum(total);
  } else {
#pragma unroll 4
    for (int i = half; i < n; i += 2) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(y + int64_t(i) * p.D);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += u[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = half_sum(f[e]);
  if (half != 0 || d >= p.D) return;
  const int64_t tok = int64_t(r.q_first) + row / p.group;
  const int head = pair % p.heads * p.group + row % p.group;
  const float inv = GRAD ? 1.0f : total == 0.0f ? 0.0f : 1.0f / total;
  const Rows& to = GRAD ? p.dq : p.out;
  *reinterpret_cast<u32x2*>(to.data + tok * to.token + head * to.head + d) =
      u32x2{pack2<DT>(f[0] * inv, f[1] * inv), pack2<DT>(f[2] * inv, f[3] * inv)};
  if (!GRAD && p.lse && d == 0) p.lse[tok * p.q_heads + head] = row_lse(top, total);
}

// --------------------------------------------------------------- gradient of q
// As k_cross_rows, with dP^T = V G^T beside S^T; dQ^T += K^T dS^T, K^T by
// transposing reads.  Leaves delta for k_cross_dkv.  SHORT: all keys (up to 128) are
// in LDS at once, and delta_i = sum_t p_it (g_i . v_t) comes from a pass over them,
// not from `out`, whose bytes are not read and whose rounding, which counts most over
// few keys, does not enter.  5 x up to 1023 rows over 2049, 32 heads in groups of
// four: 222 us of the call's 442; 4608 rows over 512, 24 heads, f16: 86 of 180; 2 x
// 4096 over 77, 10 heads of 64: 15 of 33.  Bound as k_cross_rows.
template <int DT, int DP, bool SHORT>
__global__ __launch_bounds__(256, 2) void k_cross_dq(CrossParams p) {
  constexpr int KT = 64, NE = DP / 16, NX = DP / 32, LD = row_of<DP>();
  __shared__ __attribute__((aligned(16))) uint16_t sk[2][KT * LD];
  __shared__ __attribute__((aligned(16))) uint16_t sv[2][KT * LD];
  __shared__ __attribute__((aligned(16))) float sb[2][KT];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 31, hb = lane >> 5;
  const PairWork work(blockIdx.x, p.pairs, p.row_tiles * p.splits);
  const int tile = work.tile / p.splits, split = work.tile % p.splits, req = work.pair / p.heads, h = work.pair % p.heads;
  const CrossRange r(p, req);
  const int rows = r.rows * p.group;
  if (tile * 128 >= rows) return;
  const int chunks = (r.keys + p.chunk - 1) / p.chunk;
  if (split > 0 && split >= chunks) return;
  const int from = split * p.chunk, to = smaller(r.keys, from + p.chunk);
  const int row = tile * 128 + wave * 32 + m;
  const bool active = tile * 128 + wave * 32 < rows;
  const int64_t tok = int64_t(r.q_first) + (row < rows ? p.token_of(row) : 0);
  const int head = h * p.group + (row < rows ? row % p.group : 0);
  // the first keys are on their way before the rows
  const uint16_t* kp = p.k.data + (int64_t(r.k_first) + from) * p.k.token + h * p.k.head;
  const uint16_t* vp = p.v.data + (int64_t(r.k_first) + from) * p.v.token + h * p.v.head;
  Piece<DP, KT> pk, pv, pk1, pv1;
  pk.rows(p.k.token, p.D, tid);
  pv.rows(p.v.token, p.D, tid);
  uint64_t see = 0, see1 = 0;
  if (from < to) {
    pk.load(kp, to - from, tid);
    pv.load(vp, to - from, tid);
    see = seen(p, r, from, lane);
    if constexpr (SHORT) {
      pk1.rows(p.k.token, p.D, tid);
      pv1.rows(p.v.token, p.D, tid);
      pk1.load(kp + KT * p.k.token, to - from - KT, tid);
      pv1.load(vp + KT * p.v.token, to - from - KT, tid);
      see1 = seen(p, r, from + KT, lane);
    }
  }
  u32x4 q[NE], g[NE];
  float delta = 0.0f;
  {
    TileRows<DP> all, of_g, of_out;
    all.load(p, r, p.q, tile * 128, h, tid);
    of_g.load(p, r, p.g, tile * 128, h, tid);
    if constexpr (!SHORT) of_out.load(p, r, p.out, tile * 128, h, tid);
    all.write(sk[0], tid);
    of_g.write(sv[0], tid);
    __syncthreads();
    const int mine = (wave * 32 + m) * LD + 8 * hb;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      q[e] = *reinterpret_cast<const u32x4*>(&sk[0][mine + 16 * e]);
      g[e] = *reinterpret_cast<const u32x4*>(&sv[0][mine + 16 * e]);
    }
    __syncthreads();
    if constexpr (!SHORT) {
      of_out.write(sk[0], tid);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const u32x4 y = *reinterpret_cast<const u32x4*>(&sk[0][mine + 16 * e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          delta = __builtin_fmaf(first_half<DT>(g[e][i]), first_half<DT>(y[i]), delta);
          delta = __builtin_fmaf(second_half<DT>(g[e][i]), second_half<DT>(y[i]), delta);
        }
      }
      __syncthreads();
    }
  }
  float lse = __builtin_inff();
  if (row < rows) {
    const float l = p.lse[tok * p.q_heads + head];
    lse = l == -__builtin_inff() ? __builtin_inff() : l * LOG2E;
  }
  f32x16 acc[NX];
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[x][i] = 0.0f;
  float gain = FIRST_GAIN;

  if (from < to) {
    if (see != ~uint64_t(0)) { pk.hide(see, tid); pv.hide(see, tid); }
    if (wave == 0) leave_bias(sb[0], see, p.c, lane);
    pk.write(sk[0], tid);
    pv.write(sv[0], tid);
    if constexpr (SHORT) {
      if (see1 != ~uint64_t(0)) { pk1.hide(see1, tid); pv1.hide(see1, tid); }
      if (wave == 0) leave_bias(sb[1], see1, p.c, lane);
      pk1.write(sk[1], tid);
      pv1.write(sv[1], tid);
    }
  }
  __syncthreads();
  // logits, probabilities in their place, and g . v of 32 keys
  auto products = [&](int buf, int t, f32x16& s, f32x16& dp) {
    s = rows16(&sb[buf][32 * t], hb);
#pragma unroll
    for (int i = 0; i < 16; ++i) dp[i] = 0.0f;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      s = mfma32<DT>(*reinterpret_cast<const u32x4*>(&sk[buf][(32 * t + m) * LD + 16 * e + 8 * hb]), q[e], s);
      dp = mfma32<DT>(*reinterpret_cast<const u32x4*>(&sv[buf][(32 * t + m) * LD + 16 * e + 8 * hb]), g[e], dp);
    }
    reads_ahead<2 * NE, 1, 4>();
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = exp2_hw(__builtin_fmaf(s[i], p.c, -lse));
  };
  if constexpr (SHORT) {
    if (active) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint64_t of = t < 2 ? see : see1;
        if (unsigned(of >> (32 * (t & 1))) == 0u) continue;
        f32x16 s, dp;
        products(t / 2, t & 1, s, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) delta = __builtin_fmaf(s[i], dp[i], delta);
      }
    }
  }
  delta = half_sum(delta);
  if (row < rows && split == 0 && hb == 0) p.delta[tok * p.q_heads + head] = delta;
  int buf = 0;
  for (int at = from; at < to; at += KT) {
    const bool more = at + KT < to;
    uint64_t next = see1;
    if (!SHORT && more) {
      kp += KT * p.k.token;
      vp += KT * p.v.token;
      pk.load(kp, to - at - KT, tid);
      pv.load(vp, to - at - KT, tid);
    }
    if (see != 0 && active) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const unsigned bits = t ? unsigned(see >> 32) : unsigned(see);
        if (bits == 0u) continue;
        f32x16 s, dp;
        products(buf, t, s, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[i] = s[i] * (dp[i] - delta);
        if constexpr (DT == SVDQ_F16) {
          float top = __builtin_fabsf(dp[0]);
#pragma unroll
          for (int i = 1; i < 16; ++i) top = maximum(top, __builtin_fabsf(dp[i]));
          top = half_max(top);
          const bool over = top * gain > MOST;
          if (__any(over)) {
            const float lower = over ? lower_gain(top) : gain, by = lower / gain;
            gain = lower;
#pragma unroll
            for (int x = 0; x < NX; ++x) acc[x] *= by;
          }
          dp *= gain;
        }
        // Two terms of 16 bits where delta comes from `out`: one alone and the rounding
        // of `out` cost more precision together than the result's own rounding.
        constexpr int NT = SHORT ? 1 : 2;
        u32x4 ds[NT][2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned w = pack2<DT>(dp[2 * i], dp[2 * i + 1]);
          ds[0][i / 4][i % 4] = w;
          if constexpr (!SHORT) ds[NT - 1][i / 4][i % 4] = pack2<DT>(dp[2 * i] - first_half<DT>(w), dp[2 * i + 1] - second_half<DT>(w));
        }
        const int gr = lane >> 4, i4 = lane & 15;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint16_t* b = &sk[buf][(32 * t + 16 * j + 4 * (gr >> 1) + (i4 >> 2)) * LD + 32 * x + 16 * (gr & 1) + 4 * (i4 & 3)];
            const u32x4 a = joined(read_turned(b), read_turned(b + 8 * LD));
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[x] = mfma32<DT>(a, ds[n][j], acc[x]);
          }
        }
        reads_ahead<2 * NX, 2, 4, NT>();
        __builtin_amdgcn_s_setprio(0);
      }
    }
    if (!SHORT && more) {
      next = seen(p, r, at + KT, lane);
      if (next != ~uint64_t(0)) { pk.hide(next, tid); pv.hide(next, tid); }
      if (wave == 0) leave_bias(sb[buf ^ 1], next, p.c, lane);
      pk.write(sk[buf ^ 1], tid);
      pv.write(sv[buf ^ 1], tid);
    }
    see = next;
    buf ^= 1;
    if constexpr (!SHORT) __syncthreads();
  }
  if constexpr (SHORT) {
    __syncthreads();                    // before results take the keys' place
  }
  const float by = DT == SVDQ_F16 ? p.scale / gain : p.scale;
  if (chunks <= 1) {
    store_rows<DT, DP>(p, r, p.dq, sk[0] + wave * 32 * LD, acc, by, tile * 128 + wave * 32, h, lane);
    return;
  }
  if (row >= rows) return;
  const int64_t slot = (int64_t(work.pair) * p.row_slots + row) * p.splits + split;
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (32 * x + 8 * y + 4 * hb < p.D)
        *reinterpret_cast<f32x4*>(p.part + slot * p.D + 32 * x + 8 * y + 4 * hb) =
            f32x4{acc[x][4 * y] * by, acc[x][4 * y + 1] * by, acc[x][4 * y + 2] * by, acc[x][4 * y + 3] * by};
}

// -------------------------------------------------------- gradient of k and v
// 32 keys a wave, whose K and V stay in registers as operands, KEY_TILE a
// workgroup; rows pass by in LDS, RT a stage.  S = Q K^T leaves a lane with 16
// rows of one key: the operand of dV^T += G^T P and dK^T += Q^T dS, G^T and Q^T
// by transposing reads.  A key that is not seen spoils only its own lane's sums,
// which are not stored.  delta is what the products with V start from.  5 x up to
// 1023 rows over 2049, 32 heads of 128 in groups of four: 253 us; 4608 rows over 512,
// 24 heads, f16: 87 and 13 for the join; 2 x 4096 over 77: 15 and 6.  LDS reads and
// matrix instructions bound it (each row tile is read four times a wave).  64 keys a
// wave would halve the reads but take all registers of one wave a SIMD: 10 heads of
// 64, 2 x 4096 rows over 300, 99 us a call against 61; heads of 128 spill.
template <int DT, int DP>
__global__ __launch_bounds__(256, 2) void k_cross_dkv(CrossParams p) {
  constexpr int RT = DP == 128 ? 32 : 64, NE = DP / 16, NX = DP / 32, LD = row_of<DP>();
  __shared__ __attribute__((aligned(16))) uint16_t sq[2][RT * LD];
  __shared__ __attribute__((aligned(16))) uint16_t sg[2][RT * LD];
  __shared__ __attribute__((aligned(16))) float sl[2][RT], sd[2][RT];
  // Of the NE operands of K and V each, the last LE lie in LDS: what does not fit
  // the registers of two waves a SIMD would otherwise come back from scratch memory
  // every stage, behind the rows that are on their way.
  constexpr int LE = DP == 64 ? 0 : DP == 96 ? 2 : 4, HE = NE - LE;
  __shared__ u32x4 sx[4][2 * LE + 1][64];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 31, hb = lane >> 5;
  const PairWork work(blockIdx.x, p.pairs, p.key_tiles * p.row_splits);
  const int tile = work.tile / p.row_splits, split = work.tile % p.row_splits, req = work.pair / p.heads, h = work.pair % p.heads;
  const CrossRange r(p, req);
  if (tile * KEY_TILE >= r.keys) return;
  const int rows = r.rows * p.group, chunks = (rows + p.row_chunk - 1) / p.row_chunk;
  if (split > 0 && split >= chunks) return;
  const int from = split * p.row_chunk, to = smaller(rows, from + p.row_chunk);
  const int first = tile * KEY_TILE + wave * 32;
  const bool active = first < r.keys;
  u32x4 k[HE], v[HE];
  const int key = first + m;
  const bool held = key < r.keys;
  const int64_t state = int64_t(r.k_first) + (held ? key : 0);
  const bool shown = held && (!p.mask || p.mask[state] != 0);
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    u32x4 a = {0, 0, 0, 0}, c = {0, 0, 0, 0};
    const int d = 16 * e + 8 * hb;
    if (shown && d < p.D) {
      a = *reinterpret_cast<const u32x4*>(p.k.data + state * p.k.token + h * p.k.head + d);
      c = *reinterpret_cast<const u32x4*>(p.v.data + state * p.v.token + h * p.v.head + d);
    }
    if (e < HE) {
      k[e < HE ? e : 0] = a;
      v[e < HE ? e : 0] = c;
    } else {                          // the wave's own: it reads them itself
      sx[wave][e - HE][lane] = a;
      sx[wave][LE + e - HE][lane] = c;
    }
  }
  f32x16 dk[NX], dv[NX];
  float gain = FIRST_GAIN;
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[x][i] = dv[x][i] = 0.0f;

  RowPiece<DP, RT> pq, pg;
  // a row's offset from its stage's first; where heads of a group divide the
  // stage it is the same for all stages
  const bool fixed = RT % p.group == 0;
  auto offsets = [&](int at) {
    const int t0 = p.token_of(at);
#pragma unroll
    for (int i = 0; i < pq.N; ++i) {
      const int rw = at + pq.row(tid, i), t = p.token_of(rw), gh = rw - t * p.group, d = pq.col(tid, i);
      pq.off[i] = d < p.D ? (unsigned(t - t0) * unsigned(p.q.token) + unsigned(gh) * unsigned(p.q.head) + unsigned(d)) * 2u : OUT;
      pg.off[i] = d < p.D ? (unsigned(t - t0) * unsigned(p.g.token) + unsigned(gh) * unsigned(p.g.head) + unsigned(d)) * 2u : OUT;
    }
  };
  if (fixed) offsets(from);
  float l = 0.0f, dl = 0.0f;
  auto fetch = [&](int at) {
    if (!fixed) offsets(at);
    const int64_t tok = int64_t(r.q_first) + p.token_of(at);
    pq.load(p.q.data + tok * p.q.token + h * p.group * p.q.head, to - at, tid);
    pg.load(p.g.data + tok * p.g.token + h * p.group * p.g.head, to - at, tid);
    if (tid < RT) {
      l = __builtin_inff();
      dl = 0.0f;
      const int rw = at + tid;
      if (rw < to) {
        const int t = p.token_of(rw);
        const int64_t i = (int64_t(r.q_first) + t) * p.q_heads + h * p.group + rw - t * p.group;
        const float y = p.lse[i];
        if (y != -__builtin_inff()) l = y * LOG2E - (DT == SVDQ_F16 ? P_UP : 0.0f);
        dl = p.delta[i];
      }
    }
  };
  auto write = [&](int buf) {
    pq.write(sq[buf], tid);
    pg.write(sg[buf], tid);
    if (tid < RT) {
      sl[buf][tid] = l;
      sd[buf][tid] = -dl;
    }
  };
  if (from < to) {
    fetch(from);
    write(0);
  }
  __syncthreads();
  int buf = 0;
  for (int at = from; at < to; at += RT) {
    const bool more = at + RT < to;
    if (more) fetch(at + RT);
    if (active) {
#pragma unroll
      for (int t = 0; t < RT / 32; ++t) {
        if (at + 32 * t >= to) continue;
        f32x16 s, dp = rows16(&sd[buf][32 * t], hb);      // - delta
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(&sq[buf][(32 * t + m) * LD + 16 * e + 8 * hb]);
          s = mfma32<DT>(a, e < HE ? k[e < HE ? e : 0] : sx[wave][e < HE ? 0 : e - HE][lane], s);
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(&sg[buf][(32 * t + m) * LD + 16 * e + 8 * hb]);
          dp = mfma32<DT>(a, e < HE ? v[e < HE ? e : 0] : sx[wave][e < HE ? 0 : LE + e - HE][lane], dp);
        }
        reads_ahead<2 * NE, 1, DP == 96 ? 2 : 3, 1, DP == 96 ? 0 : 4>();
        __builtin_amdgcn_s_setprio(0);
        u32x4 pf[2], ds[2];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f32x4 ll = *reinterpret_cast<const f32x4*>(&sl[buf][32 * t + 8 * y + 4 * hb]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[4 * y + i] = exp2_hw(__builtin_fmaf(s[4 * y + i], p.c, -ll[i]));
            dp[4 * y + i] *= s[4 * y + i];
          }
        }
        if constexpr (DT == SVDQ_F16) {
          float top = __builtin_fabsf(dp[0]);
#pragma unroll
          for (int i = 1; i < 16; ++i) top = maximum(top, __builtin_fabsf(dp[i]));
          top = half_max(top);
          const bool over = top * gain > MOST;
          if (__any(over)) {
            const float lower = over ? lower_gain(top) : gain, by = lower / gain;
            gain = lower;
#pragma unroll
            for (int x = 0; x < NX; ++x) dk[x] *= by;
          }
          dp *= gain;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pf[i / 4][i % 4] = pack2<DT>(s[2 * i], s[2 * i + 1]);
          ds[i / 4][i % 4] = pack2<DT>(dp[2 * i], dp[2 * i + 1]);
        }
        const int gr = lane >> 4, i4 = lane & 15;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int b = (32 * t + 16 * j + 4 * (gr >> 1) + (i4 >> 2)) * LD + 32 * x + 16 * (gr & 1) + 4 * (i4 & 3);
            const u32x4 ga = joined(read_turned(&sg[buf][b]), read_turned(&sg[buf][b + 8 * LD]));
            const u32x4 qa = joined(read_turned(&sq[buf][b]), read_turned(&sq[buf][b + 8 * LD]));
            dv[x] = mfma32<DT>(ga, pf[j], dv[x]);
            dk[x] = mfma32<DT>(qa, ds[j], dk[x]);
          }
        }
        reads_ahead<4 * NX, 2, DP == 96 ? 2 : 3>();
        __builtin_amdgcn_s_setprio(0);
      }
    }
    if (more) write(buf ^ 1);
    buf ^= 1;
    __syncthreads();
  }
  if (!active) return;
  const float kby = !shown ? 0.0f : DT == SVDQ_F16 ? p.scale / gain * 0x1p-10f : p.scale, vby = DT == SVDQ_F16 ? 0x1p-10f : 1.0f;
  if (!shown) {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) dk[x][i] = dv[x][i] = 0.0f;
  }
  if (chunks <= 1) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      unsigned wk[8], wv[8];
      columns<DT>(dk[x], kby, wk);
      columns<DT>(dv[x], vby, wv);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int d = 32 * x + 16 * y + 8 * hb;
        if (held && d < p.D) {
          *reinterpret_cast<u32x4*>(p.dk.data + state * p.dk.token + h * p.dk.head + d) = u32x4{wk[4 * y], wk[4 * y + 1], wk[4 * y + 2], wk[4 * y + 3]};
          *reinterpret_cast<u32x4*>(p.dv.data + state * p.dv.token + h * p.dv.head + d) = u32x4{wv[4 * y], wv[4 * y + 1], wv[4 * y + 2], wv[4 * y + 3]};
        }
      }
    }
  } else if (held) {
    // [pair][split][key of the tiles][2][D]
    float* part = p.key_part + ((int64_t(work.pair) * p.row_splits + split) * (int64_t(p.key_tiles) * KEY_TILE) + key) * 2 * p.D;
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int d = 32 * x + 8 * y + 4 * hb;
        if (d < p.D) {
          const f32x16 &a = dk[x], &b = dv[x];
          *reinterpret_cast<f32x4*>(part + d) = f32x4{a[4 * y] * kby, a[4 * y + 1] * kby, a[4 * y + 2] * kby, a[4 * y + 3] * kby};
          *reinterpret_cast<f32x4*>(part + p.D + d) = f32x4{b[4 * y] * vby, b[4 * y + 1] * vby, b[4 * y + 2] * vby, b[4 * y + 3] * vby};
        }
      }
  }
}

// Adds the chunks of a key's gradients: a wave a key, the lower half dk, the
// upper dv.
template <int DT>
__global__ __launch_bounds__(256) void k_cross_key_join(CrossParams p) {
  const int lane = int(threadIdx.x) & 63, width = p.key_tiles * KEY_TILE;
  const int64_t slot = int64_t(blockIdx.x) * 4 + (int(threadIdx.x) >> 6);
  if (slot >= int64_t(p.pairs) * width) return;
  const int pair = int(slot / width), key = int(slot % width);
  const CrossRange r(p, pair / p.heads);
  if (key >= r.keys) return;
  const int n = (r.rows * p.group + p.row_chunk - 1) / p.row_chunk;
  if (n <= 1) return;
  const int d = (lane & 31) * 4, half = lane >> 5;
  if (d >= p.D) return;
  const float* y = p.key_part + (int64_t(pair) * p.row_splits * width + key) * 2 * p.D + half * p.D + d;
  f32x4 f = {0, 0, 0, 0};
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(y + int64_t(i) * width * 2 * p.D);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] += u[e];
  }
  const Rows& to = half ? p.dv : p.dk;
  *reinterpret_cast<u32x2*>(to.data + (int64_t(r.k_first) + key) * to.token + pair % p.heads * to.head + d) =
      u32x2{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])};
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

svdq_status check_cross(const svdq_cross_desc* d, int q_heads, int k_heads) {
  if (!d || d->requests < 0 || d->tokens < 0 || d->states < 0 || !dtype_ok(d->dtype) || d->max_q < 0 || d->max_k < 0 || q_heads < 1 ||
      k_heads < 1 || !(d->scale - d->scale == 0.0f))
    return SVDQ_ERR_INVALID_ARG;
  if (d->head_dim < 8 || d->head_dim % 8 != 0 || q_heads % k_heads != 0) return SVDQ_ERR_SHAPE;
  if (d->head_dim > 128) return SVDQ_ERR_UNSUPPORTED;
  if (d->requests >= (int64_t(1) << 30) || d->tokens >= (int64_t(1) << 31) - 512 || d->states >= (int64_t(1) << 31) - 512)
    return SVDQ_ERR_UNSUPPORTED;
  if (!d->q_start && d->tokens != d->requests * d->max_q) return SVDQ_ERR_SHAPE;
  if (!d->k_start && d->states != d->requests * d->max_k) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

// rows that are written: no element lies on another, whether a token's heads or a
// head's tokens are the outer ones
svdq_status check_result(const svdq_heads* h, int D, int64_t n) {
  const svdq_status st = check_heads(h, D);
  if (st != SVDQ_OK || n <= 1) return st;
  const int64_t far = h->heads > 1 ? h->head_stride : 0;
  const __int128 heads = __int128(h->heads - 1) * far + D, tokens = __int128(n - 1) * h->token_stride + D;
  return h->token_stride >= heads || (h->heads > 1 && far >= tokens && h->token_stride >= D) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

// every row of 64 or 128 columns is whole 64-byte parts of lines
bool whole_lines(const svdq_heads* h, int D) {
  return D % 64 == 0 && aligned(h->data, 64) && h->token_stride % 32 == 0 && (h->heads == 1 || h->head_stride % 32 == 0);
}

Rows rows_of(const svdq_heads* h) { return Rows{static_cast<uint16_t*>(h->data), h->token_stride, h->head_stride}; }

svdq_status check_scratch(const void* ws, size_t have, size_t need) {
  if (need == 0) return SVDQ_OK;
  if (!ws) return SVDQ_ERR_INVALID_ARG;
  if (have < need) return SVDQ_ERR_CAPACITY;
  return aligned(ws, 256) ? SVDQ_OK : SVDQ_ERR_INVALID_ARG;
}

// 64 rows and a group's heads apart stay below OUT bytes
bool strides_fit(std::initializer_list<const svdq_heads*> of, int group) {
  for (const svdq_heads* h : of) {
    const int64_t heads = h->heads > 1 ? h->head_stride : 0;
    if (h->token_stride >= (int64_t(1) << 23) || (group > 1 && product_below(heads, group, 1, int64_t(1) << 28) < 0)) return false;
  }
  return true;
}

CrossParams params_of(const svdq_cross_desc* d, const CrossCut& t, int q_heads, int k_heads) {
  CrossParams p = {};
  p.q_start = d->q_start; p.k_start = d->k_start; p.mask = d->mask;
  p.tokens = t.tokens; p.states = t.states; p.max_q = d->max_q; p.max_k = d->max_k;
  p.q_heads = q_heads; p.heads = k_heads; p.group = t.group; p.pairs = t.pairs; p.D = d->head_dim;
  p.row_slots = t.row_slots; p.row_tiles = t.row_tiles; p.splits = t.splits; p.chunk = t.chunk;
  p.key_tiles = t.key_tiles; p.row_splits = t.row_splits; p.row_chunk = t.row_chunk;
  p.by_group = t.group > 1 ? unsigned((uint64_t(1) << 32) / unsigned(t.group)) + 1 : 0;
  p.scale = d->scale;
  p.c = d->scale * LOG2E;
  if (p.c == 0.0f) p.c = 1.2e-38f;      // every logit is zero to fp32, and a hidden -infinity stays one
  return p;
}

template <int DT, int DP>
void launch_forward(const CrossParams& p, const CrossCut& t, hipStream_t st) {
  const dim3 grid(unsigned(t.pairs) * unsigned(t.row_tiles) * unsigned(t.splits));
  if (t.rows == 16) k_cross_few<DT, DP><<<grid, 256, 0, st>>>(p);
  else k_cross_rows<DT, DP><<<grid, 256, 0, st>>>(p);
  if (t.splits > 1) k_cross_join<DT, false><<<dim3(unsigned(ceil_div(int64_t(t.pairs) * t.row_slots, 4))), 256, 0, st>>>(p);
}

template <int DT, int DP>
void launch_backward(const CrossParams& p, const CrossCut& t, hipStream_t st) {
  if (t.row_tiles > 0) {
    const dim3 grid(unsigned(t.pairs) * unsigned(t.row_tiles) * unsigned(t.splits));
    if (t.few_keys) k_cross_dq<DT, DP, true><<<grid, 256, 0, st>>>(p);
    else k_cross_dq<DT, DP, false><<<grid, 256, 0, st>>>(p);
    if (t.splits > 1) k_cross_join<DT, true><<<dim3(unsigned(ceil_div(int64_t(t.pairs) * t.row_slots, 4))), 256, 0, st>>>(p);
  }
  if (t.key_tiles == 0) return;
  const dim3 grid(unsigned(t.pairs) * unsigned(t.key_tiles) * unsigned(t.row_splits));
  k_cross_dkv<DT, DP><<<grid, 256, 0, st>>>(p);
  if (t.row_splits > 1)
    k_cross_key_join<DT><<<dim3(unsigned(int64_t(t.pairs) * t.key_tiles * (KEY_TILE / 4))), 256, 0, st>>>(p);
}

template <int DT>
void launch(const CrossParams& p, const CrossCut& t, bool grad, hipStream_t st) {
  if (p.D <= 64) grad ? launch_backward<DT, 64>(p, t, st) : launch_forward<DT, 64>(p, t, st);
  else if (p.D <= 96) grad ? launch_backward<DT, 96>(p, t, st) : launch_forward<DT, 96>(p, t, st);
  else grad ? launch_backward<DT, 128>(p, t, st) : launch_forward<DT, 128>(p, t, st);
}

}  // namespace

extern "C" svdq_status svdq_cross_attention_workspace(const svdq_cross_desc* d, int32_t q_heads, int32_t k_heads, size_t* bytes) {
  svdq_status st = check_cross(d, q_heads, k_heads);
  if (st != SVDQ_OK) return st;
  if (!bytes) return SVDQ_ERR_INVALID_ARG;
  CrossCut t;
  if ((st = cross_cut(d, q_heads, k_heads, device_cus(), false, &t)) != SVDQ_OK) return st;
  *bytes = size_t(cross_part_floats(d, t, false)) * 4;
  return SVDQ_OK;
}

extern "C" svdq_status svdq_cross_attention(const svdq_cross_desc* d, const svdq_heads* q, const svdq_heads* k, const svdq_heads* v,
                                            const svdq_heads* out, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!q || !k || !v || !out) return SVDQ_ERR_INVALID_ARG;
  svdq_status st = check_cross(d, q->heads, k->heads);
  if (st != SVDQ_OK) return st;
  if (v->heads != k->heads || out->heads != q->heads) return SVDQ_ERR_SHAPE;
  if (d->requests == 0 || d->tokens == 0 || d->max_q == 0) return SVDQ_OK;
  CrossCut t;
  if ((st = cross_cut(d, q->heads, k->heads, device_cus(), false, &t)) != SVDQ_OK) return st;
  if ((st = check_heads(q, d->head_dim)) != SVDQ_OK || (st = check_result(out, d->head_dim, d->tokens)) != SVDQ_OK) return st;
  if (d->states > 0)                    // without states there need be none
    for (const svdq_heads* h : {k, v})
      if ((st = check_heads(h, d->head_dim)) != SVDQ_OK) return st;
  if (!strides_fit({k, v}, 1)) return SVDQ_ERR_UNSUPPORTED;
  if ((st = check_scratch(ws, ws_bytes, size_t(cross_part_floats(d, t, false)) * 4)) != SVDQ_OK) return st;
  CrossParams p = params_of(d, t, q->heads, k->heads);
  p.q = rows_of(q); p.k = rows_of(k); p.v = rows_of(v); p.out = rows_of(out);
  p.past = whole_lines(out, d->head_dim);
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  if (p.c < 0.0f) {                     // so that a row's largest logit is that of its largest product
    p.c = -p.c;
    p.turn = 0x80008000u;
  }
  if (d->dtype == SVDQ_BF16) launch<SVDQ_BF16>(p, t, false, stream);
  else launch<SVDQ_F16>(p, t, false, stream);
  return launch_ok();
}

extern "C" svdq_status svdq_cross_attention_backward_workspace(const svdq_cross_desc* d, int32_t q_heads, int32_t k_heads, size_t* bytes) {
  svdq_status st = check_cross(d, q_heads, k_heads);
  if (st != SVDQ_OK) return st;
  if (!bytes) return SVDQ_ERR_INVALID_ARG;
  CrossCut t;
  if ((st = cross_cut(d, q_heads, k_heads, device_cus(), true, &t)) != SVDQ_OK) return st;
  *bytes = size_t(cross_delta_floats(t, q_heads) + ceil_div(cross_part_floats(d, t, true), 64) * 64 + cross_key_floats(d, t)) * 4;
  return SVDQ_OK;
}

extern "C" svdq_status svdq_cross_attention_backward(const svdq_cross_desc* d, const svdq_heads* q, const svdq_heads* k,
                                                     const svdq_heads* v, const svdq_heads* out, const float* lse,
                                                     const svdq_heads* g, const svdq_heads* dq, const svdq_heads* dk,
                                                     const svdq_heads* dv, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!q || !k || !v || !out || !g || !dq || !dk || !dv) return SVDQ_ERR_INVALID_ARG;
  svdq_status st = check_cross(d, q->heads, k->heads);
  if (st != SVDQ_OK) return st;
  if (out->heads != q->heads || g->heads != q->heads || dq->heads != q->heads || v->heads != k->heads || dk->heads != k->heads ||
      dv->heads != k->heads)
    return SVDQ_ERR_SHAPE;
  if (d->requests == 0) return SVDQ_OK;
  CrossCut t;
  if ((st = cross_cut(d, q->heads, k->heads, device_cus(), true, &t)) != SVDQ_OK) return st;
  if (d->tokens > 0) {
    for (const svdq_heads* h : {q, out, g})
      if ((st = check_heads(h, d->head_dim)) != SVDQ_OK) return st;
    if ((st = check_result(dq, d->head_dim, d->tokens)) != SVDQ_OK) return st;
    if (!lse) return SVDQ_ERR_INVALID_ARG;
  }
  if (d->states > 0) {
    for (const svdq_heads* h : {k, v})
      if ((st = check_heads(h, d->head_dim)) != SVDQ_OK) return st;
    for (const svdq_heads* h : {dk, dv})
      if ((st = check_result(h, d->head_dim, d->states)) != SVDQ_OK) return st;
  }
  if (!strides_fit({q, g}, t.group) || !strides_fit({k, v}, 1)) return SVDQ_ERR_UNSUPPORTED;
  const int64_t delta = cross_delta_floats(t, q->heads), part = ceil_div(cross_part_floats(d, t, true), 64) * 64;
  if ((st = check_scratch(ws, ws_bytes, size_t(delta + part + cross_key_floats(d, t)) * 4)) != SVDQ_OK) return st;
  CrossParams p = params_of(d, t, q->heads, k->heads);
  p.q = rows_of(q); p.k = rows_of(k); p.v = rows_of(v); p.out = rows_of(out); p.g = rows_of(g);
  p.dq = rows_of(dq); p.dk = rows_of(dk); p.dv = rows_of(dv);
  p.past = whole_lines(dq, d->head_dim);
  p.lse = const_cast<float*>(lse);
  p.delta = static_cast<float*>(ws);
  p.part = p.delta + delta;
  p.key_part = p.part + part;
  if (d->dtype == SVDQ_BF16) launch<SVDQ_BF16>(p, t, true, stream);
  else launch<SVDQ_F16>(p, t, true, stream);
  return launch_ok();
}
