// svdq_image_norm.hip -- gfx950 (MI355X) group norm with an activation over a
// channels-last map, and its gradient (include/svdq_image.h).
//
// A thread has eight neighbouring channels (16 bytes) of every R-th pixel, so
// weights, sums and scales of a channel stay in its registers.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "svdq_image.h"
#include "svdq_image_cut.h"
#include "svdq_kv_common.h"

namespace {

using namespace svdq_kv;
using namespace svdq_image;

struct NormParams {
  const uint16_t *x, *g;
  uint16_t* y;              // or dx
  const uint16_t *w, *b;
  float* stats;             // [samples][groups][2]
  float* part;              // [samples][chunks][groups][2]: mean and square deviations (gradient: sums of u and u xh)
  float* chan;              // gradient: [samples][chunks][channels][2], sums of dz and dz xh
  float *dw, *db;
  int64_t xs, xp, gs, gp, ys, yp;
  int64_t pixels, chunk;    // pixels of a chunk
  int32_t each, last_each, last_over;   // and of a row of a chunk, a row of the last one, rows of that with one more
  int32_t samples, channels, groups, per;   // per = channels / groups
  int32_t cv, rows;         // 8-channel pieces of a pixel that a workgroup takes; pixels in flight in it
  int32_t block;            // groups a workgroup takes (k_norm_whole)
  int32_t chunks, act;
  float eps;
};

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SVDQ_BF16) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    } else {
      f[2 * i] = h2f<DT>(v[i] & 0xFFFFu);
      f[2 * i + 1] = h2f<DT>(v[i] >> 16);
    }
  }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  return u32x4{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7])};
}

// The last read of a map and the write of the result pass the caches by: the call by
// itself takes 44.5 us for 1 x 512 x 512 x 128, 48.6 through them, 2 x 128 x 128 x 384
// 25.6 and 27.5; with an elementwise pass over the result behind it 66.9 and 69.4, 35.1
// and 35.8.  A 4-bit linear behind it reads the result slower from memory than it is
// written faster: 286 us and 279, 76.9 and 75.0; up to 2 x 64 x 64 x 384 (6 MB) the same.
__device__ __forceinline__ u32x4 last_read(const uint16_t* at) { return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at)); }
__device__ __forceinline__ void write_past(u32x4 v, uint16_t* at) { __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(at)); }

constexpr float LOG2E = 1.44269504088896341f;

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * z)); }

// Phi(z), the normal distribution: of erfc, since 1 + erf(z / sqrt 2) has lost every
// digit at z = -5.5, where bf16 holds z Phi(z) to 2^-9 (1 x 512 x 512 x 128: 65 us, by
// erf 53; its gradient 119, 111).
__device__ __forceinline__ float normal_below(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == SVDQ_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == SVDQ_ACT_GELU) return z * normal_below(z);
  return z;
}
// derivative of the activation
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if constexpr (ACT == SVDQ_ACT_SILU) {
    const float p = sigmoid(z);
    return __builtin_fmaf(z * p, 1.0f - p, p);
  }
  if constexpr (ACT == SVDQ_ACT_GELU)
    return __builtin_fmaf(z * 0.39894228040143268f, __builtin_amdgcn_exp2f(-0.5f * LOG2E * z * z), normal_below(z));
  return 1.0f;
}

// groups of the channels c .. c + 7
__device__ __forceinline__ void groups8(const NormParams& p, int c, int* g) {
  const bool one = p.per % 8 == 0;      // the same for all threads
  g[0] = int(unsigned(c) / unsigned(p.per));
#pragma unroll
  for (int e = 1; e < 8; ++e) g[e] = one ? g[0] : int(unsigned(c + e) / unsigned(p.per));
}

// a square deviation's rounding below zero is zero; a NaN stays one
__device__ __forceinline__ float not_negative(float x) { return __builtin_elementwise_maximum(x, 0.0f); }

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
  return x;
}

// The middle one of three: a reference that one value far from the rest does not
// move (a NaN or an infinity among them reaches the sums by itself).
__device__ __forceinline__ float middle(float a, float b, float c) { return __builtin_amdgcn_fmed3f(a, b, c); }

// Weights of eight channels; ones and zeros where there are none.
template <int DT>
__device__ __forceinline__ void weights8(const uint16_t* w, int c, float none, float* f) {
  if (w) unpack8<DT>(*reinterpret_cast<const u32x4*>(w + c), f);
  else
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = none;
}

// What a group sums over a workgroup: every thread leaves its eight channels'
// values in LDS as [channel][row of pixels], so that a group's are contiguous;
// a wave a group adds them up, in a fixed order.  Two sums at once.
__device__ __forceinline__ void leave8(float* red, int stride, const float* v, int piece, int row, bool on) {
  if (!on) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[(8 * piece + i) * stride + row] = v[i];
}

// Both sums of channel c over the rows that leave8 left, by `lanes` lanes (all of
// them get the sums): one up to 32 rows, where there are many channels (24 rows of
// 320: 14.0 us against 16.9 for the whole kernel), else 16 (one thread a channel and
// 102 rows are the longest part of a small call).
__device__ __forceinline__ int sum_lanes(int rows) { return rows <= 32 ? 1 : 16; }
__device__ __forceinline__ float2 channel_sums(const float* red, int size, int ld, int rows, int c, int lane, int lanes) {
  float2 v = {0.0f, 0.0f};
#pragma unroll 4
  for (int i = lane & (lanes - 1); i < rows; i += lanes) {
    v.x += red[c * ld + i];
    v.y += red[size + c * ld + i];
  }
  for (int m = 1; m < lanes; m *= 2) {
    v.x += __shfl_xor(v.x, m);
    v.y += __shfl_xor(v.y, m);
  }
  return v;
}

// ------------------------------------------------------------ one launch
// A workgroup has `block` groups of a sample: reads them once into registers
// (NV pieces of 16 bytes a thread), mean first and square deviations after it,
// writes them once.  1 x 8 x 8 x 1280: 6.0 us, latency (loads, two sums with a barrier
// each, stores), under the call's 9.2 on the host.
template <int DT, int ACT, int NV>
__global__ __launch_bounds__(1024) void k_norm_whole(NormParams p) {
  extern __shared__ float red[];
  __shared__ float sm[NORM_MAX_BLOCK];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, waves = (int(blockDim.x) + 63) >> 6;
  const int blocks = p.groups / p.block, sample = int(blockIdx.x) / blocks, first = int(blockIdx.x) % blocks * p.block;
  const int row = tid / p.cv, piece = tid % p.cv;
  const bool on = row < p.rows;
  const int c0 = first * p.per + 8 * piece;
  const uint16_t* x = p.x + int64_t(sample) * p.xs + c0;
  u32x4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t at = row + int64_t(i) * p.rows;
    v[i] = u32x4{0, 0, 0, 0};
    if (on && at < p.pixels) v[i] = *reinterpret_cast<const u32x4*>(x + at * p.xp);
  }
  float w[8], b[8];
  if (on) {
    weights8<DT>(p.w, c0, 1.0f, w);
    weights8<DT>(p.b, c0, 0.0f, b);
  }
  const float inv_n = 1.0f / (float(p.pixels) * float(p.per));
  const bool even = p.per % 8 == 0;     // then a thread's channels are of one group: it leaves one sum
  const int span = even ? p.per / 8 * p.rows : p.per * p.rows;
  float s[8] = {}, mean[8], f[8];
  int gi[8];                            // group within the block
  groups8(p, on ? 8 * piece : 0, gi);
  // about the group's first value, so that a mean far from zero costs nothing
#pragma unroll
  for (int e = 0; e < 8; ++e) mean[e] = h2f<DT>(p.x[int64_t(sample) * p.xs + (first + gi[e]) * p.per]);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!on || row + int64_t(i) * p.rows >= p.pixels) continue;
    unpack8<DT>(v[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e] - mean[e];
  }
  auto sums = [&]() {                   // sm[group] = sums of s
    if (!even) leave8(red, p.rows, s, piece, row, on);
    else if (on) red[piece * p.rows + row] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    for (int g = wave; g < p.block; g += waves) {
      float t = 0.0f;
#pragma unroll 4
      for (int e = lane; e < span; e += 64) t += red[g * span + e];
      t = wave_sum(t);
      if (lane == 0) sm[g] = t;
    }
    __syncthreads();
  };
  sums();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mean[e] = __builtin_fmaf(sm[gi[e]], inv_n, mean[e]);
    s[e] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (on && row + int64_t(i) * p.rows < p.pixels) {
      unpack8<DT>(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = f[e] - mean[e];
        s[e] = __builtin_fmaf(d, d, s[e]);
      }
    }
  }
  __syncthreads();                      // the means have been read
  sums();
  float a[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sm[gi[e]], inv_n, p.eps));
    if (p.stats && on && row == 0 && 8 * piece + e == gi[e] * p.per) {
      float* st = p.stats + (int64_t(sample) * p.groups + first + gi[e]) * 2;
      st[0] = mean[e];
      st[1] = rstd;
    }
    a[e] = rstd * w[e];
  }
  uint16_t* y = p.y + int64_t(sample) * p.ys + c0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t at = row + int64_t(i) * p.rows;
    if (!on || at >= p.pixels) continue;
    unpack8<DT>(v[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = activate<ACT>(__builtin_fmaf(f[e] - mean[e], a[e], b[e]));
    *reinterpret_cast<u32x4*>(y + at * p.yp) = pack8<DT>(f);
  }
}

// ----------------------------------------------------------- two launches
// Statistics of a chunk of pixels, all channels.  A thread takes its pixels in runs
// of RUN, each about the mean of those before it (the first about its first pixel),
// so that neither a mean far from zero nor a pixel far from the rest costs digits:
// about the chunk's first pixel alone, one at zero among 65536 pixels of 512 +- 2 made
// rstd wrong by 5 to 30 %.  With s and q the sums of d = x - mean and d^2 over a run and
// n pixels after it, mean += s / n and the square deviations grow by q - s s / n.
// Threads, channels of a group and chunks are joined by their means, square
// deviations about the joined mean.  1 x 512 x 512 x 128 takes 18 us (3.7 TB/s from
// memory; 16.5 about the first pixel) and k_norm_apply 24: it moves 134 MB at 5.6 TB/s,
// above a copy's 4.9, since a map of up to 256 MB still lies in the memory-side cache.
constexpr int RUN = 32, AHEAD = 4;      // pixels of a run, and of those read at once

// sum over `lanes` neighbouring lanes, a power of two
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
  for (int m = 1; m < lanes; m *= 2) x += __shfl_xor(x, m);
  return x;
}

template <int DT>
__global__ __launch_bounds__(1024) void k_norm_stats(NormParams p) {
  extern __shared__ float red[];        // [2][channels][rows]
  const int tid = int(threadIdx.x), lane = tid & 63;
  const int sample = int(blockIdx.x) / p.chunks, chunk = int(blockIdx.x) % p.chunks;
  const int row = tid / p.cv, piece = tid % p.cv;
  const bool on = row < p.rows, last = chunk + 1 == p.chunks;
  // pixels of row r of the chunk: every p.rows-th one, one more in the first `over` rows
  const int each = last ? p.last_each : p.each, over = last ? p.last_over : 0, n = each * p.rows + over;
  auto pixels = [&](int r) { return each + (r < over ? 1 : 0); };
  float m[8] = {}, dev[8] = {};
  if (on) {
    const uint16_t* x = p.x + int64_t(sample) * p.xs + (int64_t(chunk) * p.chunk + row) * p.xp + 8 * piece;
    const int64_t step = int64_t(p.rows) * p.xp;
    const int mine = pixels(row);
    float k[8] = {}, f[8];              // the first pixel, which the mean is held from
    for (int done = 0; done < mine; done += RUN) {
      const int run = min(RUN, mine - done);
      float s[8] = {}, q[8] = {};
      for (int i = 0; i < run; i += AHEAD, x += AHEAD * step) {
        u32x4 v[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (i + j < run) v[j] = *reinterpret_cast<const u32x4*>(x + j * step);
        if (done + i == 0) unpack8<DT>(v[0], k);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          if (i + j >= run) continue;
          unpack8<DT>(v[j], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = (f[e] - k[e]) - m[e];
            s[e] += d;
            q[e] = __builtin_fmaf(d, d, q[e]);
          }
        }
      }
      const float inv = 1.0f / float(done + run);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float by = s[e] * inv;
        m[e] += by;
        dev[e] += not_negative(__builtin_fmaf(-s[e], by, q[e]));
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] += k[e];
  }
  // channels: a row's mean counts by its pixels (rows of none hold zeros)
  const int ld = p.rows | 1, size = p.channels * ld;
  leave8(red, ld, m, piece, row, on);
  leave8(red + size, ld, dev, piece, row, on);
  __syncthreads();
  const float inv = 1.0f / float(n);
  const int lanes = sum_lanes(p.rows);
  for (int c = tid / lanes; c < p.channels; c += int(blockDim.x) / lanes) {
    const int from = lane & (lanes - 1);
    const float m0 = red[c * ld];       // row 0's: there is always one
    float t = 0.0f, u = 0.0f, d = 0.0f;
#pragma unroll 4
    for (int r = from; r < p.rows; r += lanes) {
      t = __builtin_fmaf(float(pixels(r)), red[c * ld + r] - m0, t);
      d += red[size + c * ld + r];
    }
    const float mean = lanes_sum(t, lanes) * inv;
#pragma unroll 4
    for (int r = from; r < p.rows; r += lanes) {
      const float e = (red[c * ld + r] - m0) - mean;
      u = __builtin_fmaf(float(pixels(r)) * e, e, u);
    }
    u = lanes_sum(u + d, lanes);
    if (from != 0) continue;
    // in the places of the channel's own first row: nobody else reads these
    red[c * ld] = m0 + mean;
    red[size + c * ld] = u;
  }
  __syncthreads();
  // groups: as many lanes as a power of two from their channels on, so that groups of
  // few are summed side by side
  int wide = 8;
  while (wide < p.per && wide < 64) wide *= 2;
  for (int g = tid / wide; g < p.groups; g += int(blockDim.x) / wide) {
    const int from = lane & (wide - 1);
    const float* m0 = red + g * p.per * ld;
    const float* d0 = m0 + size;
    const float k0 = m0[0];
    float t = 0.0f, u = 0.0f, d = 0.0f;
    for (int c = from; c < p.per; c += wide) {
      t += m0[c * ld] - k0;
      d += d0[c * ld];
    }
    t = lanes_sum(t, wide) / float(p.per);
    for (int c = from; c < p.per; c += wide) {
      const float e = (m0[c * ld] - k0) - t;
      u = __builtin_fmaf(e, e, u);
    }
    u = lanes_sum(__builtin_fmaf(float(n), u, d), wide);
    if (from != 0) continue;
    float* out = p.part + (int64_t(blockIdx.x) * p.groups + g) * 2;
    out[0] = k0 + t;
    out[1] = u;
  }
}

// What the means of a group's chunks are joined about: their middle one of three.
__device__ __forceinline__ float reference(const float2* of, const NormParams& p) {
  return middle(of[int64_t(p.chunks / 4) * p.groups].x, of[int64_t(p.chunks / 2) * p.groups].x, of[int64_t(p.chunks * 3LL / 4) * p.groups].x);
}

// Adds two values a chunk and group over a sample's chunks: all threads at once,
// thread t has group t % groups and every (threads / groups)-th chunk, so that
// few loads wait for another; add(group, chunk, value, sums of three).  In LDS
// the sums of a group end up at sm[3 group ..].
template <class F>
__device__ __forceinline__ void join_chunks(const NormParams& p, int sample, int tid, float* sm, F add) {
  const int threads = int(blockDim.x), wide = min(p.groups, threads), walks = threads / wide;
  const float2* part = reinterpret_cast<const float2*>(p.part) + int64_t(sample) * p.chunks * p.groups;
  for (int g0 = 0; g0 < p.groups; g0 += wide) {
    const int g = g0 + tid % wide, walk = tid / wide;
    float s[3] = {0.0f, 0.0f, 0.0f};
    const bool on = walk < walks && g < p.groups;
    if (on) {
      const float2* q = part + g;
      const float first = reference(q, p);
#pragma unroll 8
      for (int i = walk; i < p.chunks; i += walks) add(first, i, q[int64_t(i) * p.groups], s);
    }
    float* mine = sm + 3 * p.groups;
    if (walks > 1) {
      if (g0 > 0) __syncthreads();
      if (on)
        for (int e = 0; e < 3; ++e) mine[3 * tid + e] = s[e];
      __syncthreads();
      if (on && walk == 0)
        for (int w = 1; w < walks; ++w)
          for (int e = 0; e < 3; ++e) s[e] += mine[3 * (tid + w * wide) + e];
    }
    if (on && walk == 0)
      for (int e = 0; e < 3; ++e) sm[3 * g + e] = s[e];
  }
  __syncthreads();
}

// Mean and rstd of every group of a sample from its chunks' (in LDS, [groups][3]).
// All chunks but the last have the same number of pixels.
__device__ __forceinline__ void join_stats(const NormParams& p, int sample, int tid, float* sm) {
  const int64_t tail = p.pixels - int64_t(p.chunks - 1) * p.chunk;
  const float share = float(double(p.chunk) / double(p.pixels)), last = float(double(tail) / double(p.pixels));
  join_chunks(p, sample, tid, sm, [&](float first, int i, float2 v, float* s) {
    const float wt = i + 1 < p.chunks ? share : last, e = v.x - first;
    s[0] = __builtin_fmaf(wt, e, s[0]);
    s[1] = __builtin_fmaf(wt * e, e, s[1]);
    s[2] += v.y;
  });
  const float2* part = reinterpret_cast<const float2*>(p.part) + int64_t(sample) * p.chunks * p.groups;
  for (int g = tid; g < p.groups; g += int(blockDim.x)) {
    const float m = sm[3 * g], u = sm[3 * g + 1], d = sm[3 * g + 2];
    const float between = not_negative(__builtin_fmaf(-m, m, u));
    const float within = d / (float(p.per) * float(p.pixels));
    sm[3 * g] = reference(part + g, p) + m;
    sm[3 * g + 1] = 1.0f / __builtin_sqrtf(between + within + p.eps);
  }
  __syncthreads();
}

template <int DT, int ACT>
__global__ __launch_bounds__(1024) void k_norm_apply(NormParams p) {
  extern __shared__ float sm[];         // [groups][3], and three a thread
  const int tid = int(threadIdx.x);
  const int sample = int(blockIdx.x) / p.chunks, chunk = int(blockIdx.x) % p.chunks;
  join_stats(p, sample, tid, sm);
  if (p.stats && chunk == 0)
    for (int i = tid; i < 2 * p.groups; i += int(blockDim.x)) p.stats[int64_t(sample) * p.groups * 2 + i] = sm[i / 2 * 3 + i % 2];
  const int row = tid / p.cv, piece = tid % p.cv;
  if (row >= p.rows) return;
  float w[8], b[8], a[8], m[8], f[8];
  weights8<DT>(p.w, 8 * piece, 1.0f, w);
  weights8<DT>(p.b, 8 * piece, 0.0f, b);
  int g[8];
  groups8(p, 8 * piece, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = sm[3 * g[e]];
    a[e] = sm[3 * g[e] + 1] * w[e];
  }
  const int64_t from = int64_t(chunk) * p.chunk, n = min(p.pixels - from, p.chunk);
  const uint16_t* x = p.x + int64_t(sample) * p.xs + (from + row) * p.xp + 8 * piece;
  uint16_t* y = p.y + int64_t(sample) * p.ys + (from + row) * p.yp + 8 * piece;
  const int64_t xstep = int64_t(p.rows) * p.xp, ystep = int64_t(p.rows) * p.yp;
  int64_t at = row;
  for (; at + 3 * int64_t(p.rows) < n; at += 4 * int64_t(p.rows), x += 4 * xstep, y += 4 * ystep) {
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = last_read(x + i * xstep);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack8<DT>(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = activate<ACT>(__builtin_fmaf(f[e] - m[e], a[e], b[e]));
      write_past(pack8<DT>(f), y + i * ystep);
    }
  }
  for (; at < n; at += p.rows, x += xstep, y += ystep) {
    unpack8<DT>(last_read(x), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = activate<ACT>(__builtin_fmaf(f[e] - m[e], a[e], b[e]));
    write_past(pack8<DT>(f), y);
  }
}

// ------------------------------------------------------------- gradient
// dz and xh of eight elements
template <int DT, int ACT>
__device__ __forceinline__ void back8(u32x4 xv, u32x4 gv, const float* m, const float* r, const float* w, const float* b,
                                      float* dz, float* xh) {
  float f[8];
  unpack8<DT>(xv, f);
  unpack8<DT>(gv, dz);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    xh[e] = (f[e] - m[e]) * r[e];
    if constexpr (ACT != SVDQ_ACT_NONE) dz[e] *= slope<ACT>(__builtin_fmaf(xh[e], w[e], b[e]));
  }
}

// One launch: as k_norm_whole.  Few samples: a workgroup takes its groups of all of
// them, one after the other, and ends with dw and db; many: of one, whose channel
// sums go to `chan` for k_norm_sum.
template <int DT, int ACT, int NV>
__global__ __launch_bounds__(512) void k_norm_grad_whole(NormParams p) {
  extern __shared__ float red[];        // [2][channels of the block][rows]
  __shared__ float sm[2 * NORM_MAX_BLOCK];
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, waves = (int(blockDim.x) + 63) >> 6;
  const int blocks = p.groups / p.block, first = int(blockIdx.x) % blocks * p.block;
  const bool every = int(gridDim.x) == blocks;
  const int from = every ? 0 : int(blockIdx.x) / blocks, to = every ? p.samples : from + 1;
  const int row = tid / p.cv, piece = tid % p.cv;
  const bool on = row < p.rows;
  const int c0 = first * p.per + 8 * piece;
  const int wide = 8 * p.cv, ld = p.rows | 1, size = wide * ld;
  float* total = red + 2 * size;        // [2][channels of the block]
  float w[8] = {}, b[8] = {};
  int gi[8] = {};
  if (on) {
    weights8<DT>(p.w, c0, 1.0f, w);
    weights8<DT>(p.b, c0, 0.0f, b);
    groups8(p, 8 * piece, gi);
  }
  for (int sample = from; sample < to; ++sample) {
    u32x4 xv[NV], gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = row + int64_t(i) * p.rows;
      xv[i] = gv[i] = u32x4{0, 0, 0, 0};
      if (on && at < p.pixels) {
        xv[i] = *reinterpret_cast<const u32x4*>(p.x + int64_t(sample) * p.xs + at * p.xp + c0);
        gv[i] = *reinterpret_cast<const u32x4*>(p.g + int64_t(sample) * p.gs + at * p.gp + c0);
      }
    }
    float m[8] = {}, r[8] = {}, s[8] = {}, q[8] = {}, dz[8], xh[8];
    if (on) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* st = p.stats + (int64_t(sample) * p.groups + first + gi[e]) * 2;
        m[e] = st[0];
        r[e] = st[1];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on || row + int64_t(i) * p.rows >= p.pixels) continue;
      back8<DT, ACT>(xv[i], gv[i], m, r, w, b, dz, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[e] += dz[e];
        q[e] = __builtin_fmaf(dz[e], xh[e], q[e]);
      }
    }
    leave8(red, ld, s, piece, row, on);
    leave8(red + size, ld, q, piece, row, on);
    __syncthreads();
    const int lanes = sum_lanes(p.rows);
    for (int c = tid / lanes; c < wide; c += int(blockDim.x) / lanes) {
      const float2 v = channel_sums(red, size, ld, p.rows, c, lane, lanes);
      if ((lane & (lanes - 1)) != 0) continue;
      const float s0 = v.x, q0 = v.y;
      const int ch = first * p.per + c;
      if (!every) {
        *reinterpret_cast<float2*>(p.chan + (int64_t(sample) * p.channels + ch) * 2) = float2{s0, q0};
      } else {                            // (the same thread for every sample)
        const float s1 = sample > 0 ? total[c] + s0 : s0, q1 = sample > 0 ? total[wide + c] + q0 : q0;
        total[c] = s1;
        total[wide + c] = q1;
        if (sample + 1 == to) {
          if (p.db) p.db[ch] = s1;
          if (p.dw) p.dw[ch] = q1;
        }
      }
      const float wc = p.w ? h2f<DT>(p.w[ch]) : 1.0f;
      red[c * ld] = s0 * wc;          // (the channel's own places: nobody else reads these)
      red[size + c * ld] = q0 * wc;
    }
    __syncthreads();
    const float inv_n = 1.0f / (float(p.pixels) * float(p.per));
    for (int g = wave; g < p.block; g += waves) {
      float t = 0.0f, u = 0.0f;
      for (int c = lane; c < p.per; c += 64) {
        t += red[(g * p.per + c) * ld];
        u += red[size + (g * p.per + c) * ld];
      }
      t = wave_sum(t);
      u = wave_sum(u);
      if (lane == 0) {
        sm[2 * g] = t * inv_n;
        sm[2 * g + 1] = u * inv_n;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = row + int64_t(i) * p.rows;
      if (!on || at >= p.pixels) continue;
      back8<DT, ACT>(xv[i], gv[i], m, r, w, b, dz, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dz[e] = r[e] * (__builtin_fmaf(dz[e], w[e], -sm[2 * gi[e]]) - xh[e] * sm[2 * gi[e] + 1]);
      *reinterpret_cast<u32x4*>(p.y + int64_t(sample) * p.ys + at * p.yp + c0) = pack8<DT>(dz);
    }
    __syncthreads();                    // sums and means have been read
  }
}

// Two launches: channel and group sums of a chunk (2 x 128 x 128 x 320: 14.3 us, 2.9
// TB/s: memory, and the activation's slope, about 120 vector instructions for eight
// elements of a lane, of which the sums need it, too) ...
template <int DT, int ACT>
__global__ __launch_bounds__(1024) void k_norm_grad_sums(NormParams p) {
  extern __shared__ float red[];        // [2][channels][rows]
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, waves = (int(blockDim.x) + 63) >> 6;
  const int sample = int(blockIdx.x) / p.chunks, chunk = int(blockIdx.x) % p.chunks;
  const int64_t from = int64_t(chunk) * p.chunk, n = min(p.pixels - from, p.chunk);
  const int row = tid / p.cv, piece = tid % p.cv;
  const bool on = row < p.rows;
  float s[8] = {}, q[8] = {};
  if (on) {
    float w[8], b[8], m[8], r[8], dz[8], xh[8];
    weights8<DT>(p.w, 8 * piece, 1.0f, w);
    weights8<DT>(p.b, 8 * piece, 0.0f, b);
    int gi[8];
    groups8(p, 8 * piece, gi);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float* st = p.stats + (int64_t(sample) * p.groups + gi[e]) * 2;
      m[e] = st[0];
      r[e] = st[1];
    }
    const uint16_t* x = p.x + int64_t(sample) * p.xs + (from + row) * p.xp + 8 * piece;
    const uint16_t* g = p.g + int64_t(sample) * p.gs + (from + row) * p.gp + 8 * piece;
    const int64_t xstep = int64_t(p.rows) * p.xp, gstep = int64_t(p.rows) * p.gp;
    auto add = [&](u32x4 xv, u32x4 gv) {
      back8<DT, ACT>(xv, gv, m, r, w, b, dz, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[e] += dz[e];
        q[e] = __builtin_fmaf(dz[e], xh[e], q[e]);
      }
    };
    int64_t at = row;
    for (; at + int64_t(p.rows) < n; at += 2 * int64_t(p.rows), x += 2 * xstep, g += 2 * gstep) {
      const u32x4 x0 = *reinterpret_cast<const u32x4*>(x), g0 = *reinterpret_cast<const u32x4*>(g);
      const u32x4 x1 = *reinterpret_cast<const u32x4*>(x + xstep), g1 = *reinterpret_cast<const u32x4*>(g + gstep);
      add(x0, g0);
      add(x1, g1);
    }
    if (at < n) add(*reinterpret_cast<const u32x4*>(x), *reinterpret_cast<const u32x4*>(g));
  }
  const int ld = p.rows | 1, size = p.channels * ld;
  leave8(red, ld, s, piece, row, on);
  leave8(red + size, ld, q, piece, row, on);
  __syncthreads();
  const int lanes = sum_lanes(p.rows);
  for (int c = tid / lanes; c < p.channels; c += int(blockDim.x) / lanes) {
    const float2 v = channel_sums(red, size, ld, p.rows, c, lane, lanes);
    if ((lane & (lanes - 1)) != 0) continue;
    const float s0 = v.x, q0 = v.y;
    *reinterpret_cast<float2*>(p.chan + (int64_t(blockIdx.x) * p.channels + c) * 2) = float2{s0, q0};
    const float wc = p.w ? h2f<DT>(p.w[c]) : 1.0f;
    red[c * ld] = s0 * wc;          // (the channel's own places: nobody else reads these)
    red[size + c * ld] = q0 * wc;
  }
  __syncthreads();
  for (int g = wave; g < p.groups; g += waves) {
    float t = 0.0f, u = 0.0f;
    for (int c = lane; c < p.per; c += 64) {
      t += red[(g * p.per + c) * ld];
      u += red[size + (g * p.per + c) * ld];
    }
    t = wave_sum(t);
    u = wave_sum(u);
    if (lane == 0) *reinterpret_cast<float2*>(p.part + (int64_t(blockIdx.x) * p.groups + g) * 2) = float2{t, u};
  }
}

// dw and db of 32 channels: sums over `n` rows of [channels][2], eight walks and
// then one thread a channel.  A walk adds 256 rows up before it adds them to the rest
// (125000 equal rows one after the other are up to 4e-4 off, so 3e-6).
__device__ __forceinline__ void sum_channels(const NormParams& p, int64_t n, int c0, int tid, float* red) {
  const int c = c0 + (tid & 31), walk = tid >> 5;
  const bool on = walk < 8 && c < p.channels;
  if (on) {
    float s = 0.0f, q = 0.0f;
    const float2* at = reinterpret_cast<const float2*>(p.chan) + c;
    for (int64_t i = walk; i < n;) {
      float2 part = {0.0f, 0.0f};
      const int64_t to = min(n, i + 8 * 256);
#pragma unroll 4
      for (; i < to; i += 8) {
        const float2 v = at[i * p.channels];
        part.x += v.x;
        part.y += v.y;
      }
      s += part.x;
      q += part.y;
    }
    red[2 * tid] = s;
    red[2 * tid + 1] = q;
  }
  __syncthreads();
  if (!on || walk != 0) return;
  float s = 0.0f, q = 0.0f;
  for (int i = 0; i < 8; ++i) {
    s += red[2 * (tid + 32 * i)];
    q += red[2 * (tid + 32 * i) + 1];
  }
  if (p.db) p.db[c] = s;
  if (p.dw) p.dw[c] = q;
}

__global__ __launch_bounds__(256) void k_norm_sum(NormParams p) {
  __shared__ float red[512];
  sum_channels(p, int64_t(p.samples) * p.chunks, int(blockIdx.x) * 32, int(threadIdx.x), red);
}

// ... and the map's gradient (14.5 us there, 4.3 TB/s); workgroups past the chunks'
// have the channels' sums.
template <int DT, int ACT>
__global__ __launch_bounds__(1024) void k_norm_grad_apply(NormParams p) {
  extern __shared__ float sm[];         // [groups][3], and three a thread
  const int tid = int(threadIdx.x);
  const int work = p.samples * p.chunks;
  if (int(blockIdx.x) >= work) {
    sum_channels(p, work, (int(blockIdx.x) - work) * 32, tid, sm);
    return;
  }
  const int sample = int(blockIdx.x) / p.chunks, chunk = int(blockIdx.x) % p.chunks;
  const float inv_n = 1.0f / (float(p.pixels) * float(p.per));
  join_chunks(p, sample, tid, sm, [](float, int, float2 v, float* s) {
    s[0] += v.x;
    s[1] += v.y;
  });
  const int row = tid / p.cv, piece = tid % p.cv;
  if (row >= p.rows) return;
  float w[8], b[8], m[8], r[8], t[8], u[8];
  weights8<DT>(p.w, 8 * piece, 1.0f, w);
  weights8<DT>(p.b, 8 * piece, 0.0f, b);
  int gi[8];
  groups8(p, 8 * piece, gi);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float* st = p.stats + (int64_t(sample) * p.groups + gi[e]) * 2;
    m[e] = st[0];
    r[e] = st[1];
    t[e] = sm[3 * gi[e]] * inv_n;
    u[e] = sm[3 * gi[e] + 1] * inv_n;
  }
  const int64_t from = int64_t(chunk) * p.chunk, n = min(p.pixels - from, p.chunk);
  const uint16_t* x = p.x + int64_t(sample) * p.xs + (from + row) * p.xp + 8 * piece;
  const uint16_t* g = p.g + int64_t(sample) * p.gs + (from + row) * p.gp + 8 * piece;
  uint16_t* y = p.y + int64_t(sample) * p.ys + (from + row) * p.yp + 8 * piece;
  const int64_t xstep = int64_t(p.rows) * p.xp, gstep = int64_t(p.rows) * p.gp, ystep = int64_t(p.rows) * p.yp;
  auto one = [&](u32x4 xv, u32x4 gv, uint16_t* to) {
    float dz[8], xh[8];
    back8<DT, ACT>(xv, gv, m, r, w, b, dz, xh);
#pragma unroll
    for (int e = 0; e < 8; ++e) dz[e] = r[e] * (__builtin_fmaf(dz[e], w[e], -t[e]) - xh[e] * u[e]);
    write_past(pack8<DT>(dz), to);
  };
  int64_t at = row;
  for (; at + int64_t(p.rows) < n; at += 2 * int64_t(p.rows), x += 2 * xstep, g += 2 * gstep, y += 2 * ystep) {
    const u32x4 x0 = last_read(x), g0 = last_read(g);
    const u32x4 x1 = last_read(x + xstep), g1 = last_read(g + gstep);
    one(x0, g0, y);
    one(x1, g1, y + ystep);
  }
  if (at < n) one(last_read(x), last_read(g), y);
}

// dw = db = 0 (a call without samples)
__global__ void k_norm_zero(float* dw, float* db, int n) {
  const int i = int(blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= n) return;
  if (dw) dw[i] = 0.0f;
  if (db) db[i] = 0.0f;
}

// ---------------------------------------------------------------- host side
svdq_status check_norm(const svdq_norm_desc* d) {
  if (!d || d->samples < 0 || d->pixels < 0 || !dtype_ok(d->dtype) || d->groups < 1 || d->channels < 1 || d->act < SVDQ_ACT_NONE ||
      d->act > SVDQ_ACT_GELU || !(d->eps >= 0.0f) || !(d->eps <= 3.0e38f))
    return SVDQ_ERR_INVALID_ARG;
  if (d->samples > 0 && d->pixels < 1) return SVDQ_ERR_INVALID_ARG;
  if (d->channels % 8 != 0 || d->channels % d->groups != 0 || !aligned(d->weight, 16) || !aligned(d->bias, 16)) return SVDQ_ERR_SHAPE;
  if (d->channels > SVDQ_NORM_MAX_CHANNELS) return SVDQ_ERR_UNSUPPORTED;
  if (d->samples >= (int64_t(1) << 31) || product_below(d->samples, d->pixels, d->channels, int64_t(1) << 60) < 0) return SVDQ_ERR_UNSUPPORTED;
  return SVDQ_OK;
}

svdq_status check_map(const svdq_norm_desc* d, const svdq_map* m) {
  if (!m || !m->data) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(m->data, 16) || m->sample_stride % 8 != 0 || m->pixel_stride % 8 != 0 || m->sample_stride < 0 || m->pixel_stride < 0)
    return SVDQ_ERR_SHAPE;
  if (d->pixels > 1 && m->pixel_stride < d->channels) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

// a map that is written: no element lies on another
svdq_status check_result(const svdq_norm_desc* d, const svdq_map* m) {
  const svdq_status st = check_map(d, m);
  if (st != SVDQ_OK || d->samples <= 1) return st;
  const __int128 pixels = __int128(d->pixels - 1) * m->pixel_stride + d->channels, samples = __int128(d->samples - 1) * m->sample_stride + d->channels;
  return m->sample_stride >= pixels || (d->pixels > 1 && m->pixel_stride >= samples && m->sample_stride >= d->channels) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

svdq_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return SVDQ_OK;
  if (!ws) return SVDQ_ERR_INVALID_ARG;
  if (have < need) return SVDQ_ERR_CAPACITY;
  return aligned(ws, 16) ? SVDQ_OK : SVDQ_ERR_INVALID_ARG;
}

NormParams params_of(const svdq_norm_desc* d, const NormCut& t) {
  NormParams p = {};
  p.w = static_cast<const uint16_t*>(d->weight);
  p.b = static_cast<const uint16_t*>(d->bias);
  p.pixels = d->pixels; p.chunk = t.chunk;
  p.samples = int32_t(d->samples); p.channels = d->channels; p.groups = d->groups; p.per = d->channels / d->groups;
  const int64_t tail = d->pixels - int64_t(t.chunks - 1) * t.chunk;
  p.each = int32_t(t.chunk / t.rows); p.last_each = int32_t(tail / t.rows); p.last_over = int32_t(tail % t.rows);
  p.cv = t.cv; p.rows = t.rows; p.block = t.block; p.chunks = t.chunks; p.act = d->act; p.eps = d->eps;
  return p;
}

template <int DT, int ACT>
void launch_norm(const NormParams& p, const NormCut& t, hipStream_t st) {
  const size_t red = norm_lds(t);
  if (t.block > 0) {
    const dim3 grid(unsigned(p.samples) * unsigned(p.groups / t.block));
    if (t.pieces <= 1) k_norm_whole<DT, ACT, 1><<<grid, t.threads, red, st>>>(p);
    else if (t.pieces <= 2) k_norm_whole<DT, ACT, 2><<<grid, t.threads, red, st>>>(p);
    else if (t.pieces <= 4) k_norm_whole<DT, ACT, 4><<<grid, t.threads, red, st>>>(p);
    else k_norm_whole<DT, ACT, 8><<<grid, t.threads, red, st>>>(p);
    return;
  }
  const dim3 grid(unsigned(p.samples) * unsigned(t.chunks));
  k_norm_stats<DT><<<grid, t.threads, 2 * red, st>>>(p);
  k_norm_apply<DT, ACT><<<grid, t.threads, norm_join_lds(p.groups, t.threads), st>>>(p);
}

template <int DT, int ACT>
void launch_norm_grad(const NormParams& p, const NormCut& t, hipStream_t st) {
  const size_t red = 2 * norm_lds(t);
  const bool sums = p.dw || p.db;
  const unsigned tiles = unsigned((p.channels + 31) / 32);
  if (t.block > 0) {
    const bool every = p.samples <= NORM_FEW_SAMPLES;
    const dim3 grid((every ? 1u : unsigned(p.samples)) * unsigned(p.groups / t.block));
    const size_t lds = red + size_t(t.cv) * 16 * 4;
    if (t.pieces <= 1) k_norm_grad_whole<DT, ACT, 1><<<grid, t.threads, lds, st>>>(p);
    else if (t.pieces <= 2) k_norm_grad_whole<DT, ACT, 2><<<grid, t.threads, lds, st>>>(p);
    else k_norm_grad_whole<DT, ACT, 4><<<grid, t.threads, lds, st>>>(p);
    if (!every && sums) k_norm_sum<<<dim3(tiles), 256, 0, st>>>(p);
    return;
  }
  const unsigned work = unsigned(p.samples) * unsigned(t.chunks);
  k_norm_grad_sums<DT, ACT><<<dim3(work), t.threads, red, st>>>(p);
  k_norm_grad_apply<DT, ACT><<<dim3(work + (sums ? tiles : 0)), t.threads, norm_join_lds(p.groups, t.threads), st>>>(p);
}

template <int DT>
void launch(const NormParams& p, const NormCut& t, bool grad, hipStream_t st) {
  if (p.act == SVDQ_ACT_NONE) grad ? launch_norm_grad<DT, SVDQ_ACT_NONE>(p, t, st) : launch_norm<DT, SVDQ_ACT_NONE>(p, t, st);
  else if (p.act == SVDQ_ACT_SILU) grad ? launch_norm_grad<DT, SVDQ_ACT_SILU>(p, t, st) : launch_norm<DT, SVDQ_ACT_SILU>(p, t, st);
  else grad ? launch_norm_grad<DT, SVDQ_ACT_GELU>(p, t, st) : launch_norm<DT, SVDQ_ACT_GELU>(p, t, st);
}

}  // namespace

extern "C" svdq_status svdq_group_norm_workspace(const svdq_norm_desc* d, size_t* bytes) {
  svdq_status st = check_norm(d);
  if (st != SVDQ_OK) return st;
  if (!bytes) return SVDQ_ERR_INVALID_ARG;
  NormCut t;
  if ((st = norm_cut(d, false, &t)) != SVDQ_OK) return st;
  *bytes = norm_bytes(d, t, false);
  return SVDQ_OK;
}

extern "C" svdq_status svdq_group_norm(const svdq_norm_desc* d, const svdq_map* x, const svdq_map* y, float* stats, void* ws,
                                       size_t ws_bytes, hipStream_t stream) {
  svdq_status st = check_norm(d);
  if (st != SVDQ_OK) return st;
  if (!x || !y) return SVDQ_ERR_INVALID_ARG;
  if (d->samples == 0) return SVDQ_OK;
  if ((st = check_map(d, x)) != SVDQ_OK || (st = check_result(d, y)) != SVDQ_OK) return st;
  NormCut t;
  if ((st = norm_cut(d, false, &t)) != SVDQ_OK || (st = check_ws(ws, ws_bytes, norm_bytes(d, t, false))) != SVDQ_OK) return st;
  NormParams p = params_of(d, t);
  p.x = static_cast<const uint16_t*>(x->data);
  p.y = static_cast<uint16_t*>(y->data);
  p.xs = x->sample_stride; p.xp = x->pixel_stride; p.ys = y->sample_stride; p.yp = y->pixel_stride;
  p.stats = stats;
  p.part = static_cast<float*>(ws);
  if (d->dtype == SVDQ_BF16) launch<SVDQ_BF16>(p, t, false, stream);
  else launch<SVDQ_F16>(p, t, false, stream);
  return launch_ok();
}

extern "C" svdq_status svdq_group_norm_backward_workspace(const svdq_norm_desc* d, size_t* bytes) {
  svdq_status st = check_norm(d);
  if (st != SVDQ_OK) return st;
  if (!bytes) return SVDQ_ERR_INVALID_ARG;
  NormCut t;
  if ((st = norm_cut(d, true, &t)) != SVDQ_OK) return st;
  *bytes = norm_bytes(d, t, true);
  return SVDQ_OK;
}

extern "C" svdq_status svdq_group_norm_backward(const svdq_norm_desc* d, const svdq_map* x, const svdq_map* g, const float* stats,
                                                const svdq_map* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                                                hipStream_t stream) {
  svdq_status st = check_norm(d);
  if (st != SVDQ_OK) return st;
  if (!x || !g || !dx) return SVDQ_ERR_INVALID_ARG;
  if (d->samples == 0) {
    if (!dw && !db) return SVDQ_OK;
    k_norm_zero<<<dim3(unsigned((d->channels + 255) / 256)), 256, 0, stream>>>(dw, db, d->channels);
    return launch_ok();
  }
  if (!stats) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_map(d, x)) != SVDQ_OK || (st = check_map(d, g)) != SVDQ_OK || (st = check_result(d, dx)) != SVDQ_OK) return st;
  NormCut t;
  if ((st = norm_cut(d, true, &t)) != SVDQ_OK || (st = check_ws(ws, ws_bytes, norm_bytes(d, t, true))) != SVDQ_OK) return st;
  NormParams p = params_of(d, t);
  p.x = static_cast<const uint16_t*>(x->data);
  p.g = static_cast<const uint16_t*>(g->data);
  p.y = static_cast<uint16_t*>(dx->data);
  p.xs = x->sample_stride; p.xp = x->pixel_stride; p.gs = g->sample_stride; p.gp = g->pixel_stride;
  p.ys = dx->sample_stride; p.yp = dx->pixel_stride;
  p.stats = const_cast<float*>(stats);
  p.chan = static_cast<float*>(ws);
  p.part = p.chan + (t.block > 0 ? 0 : int64_t(d->samples) * t.chunks * d->channels * 2);
  p.dw = dw; p.db = db;
  if (d->dtype == SVDQ_BF16) launch<SVDQ_BF16>(p, t, true, stream);
  else launch<SVDQ_F16>(p, t, true, stream);
  return launch_ok();
}
