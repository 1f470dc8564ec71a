// Residual addition and root-mean-square norm of rows, and the backward.
//
//   h = bf16(x + residual),  y = bf16(h w r),  r = 1 / sqrt(mean(h^2) + eps)
//   dx = bf16(dh + r (w dy - h r^2 mean(w dy h))),  dw = sum over rows of dy h r
//
// Bound by HBM: 4 to 8 B per element in either direction: forward of 4096 x 4096 with a residual 20.4 us = 6.6 TB/s, backward with dh
// 22.3 us = 6.0 TB/s and 3.9 for the weight's gradient, whose 256 partials are 4 MB more (2048 x 8192, 512 partials: 24.7 + 4.4 us).  For a few rows by a
// launch and two dependent round trips (16 x 8192: 3.8 us).  A row stays in the registers of the T threads that
// hold it (a wave for short rows, a workgroup for long ones), 8 elements to a load, so each tensor is read or written once.
// The backward walks over rows with the weight's gradient in registers, one partial per workgroup, summed by a second
// kernel in a fixed order.
#include "kernels.h"
#include "rows.h"

namespace qlora {

namespace {

constexpr int NT = 256;   // threads of a workgroup of several rows

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

__device__ __forceinline__ const u32x4* row_of(const RowsView& v, int64_t row) {
  return reinterpret_cast<const u32x4*>(v.data + row * v.stride);
}
__device__ __forceinline__ u32x4* out_row(const RowsView& v, int64_t row) {
  return reinterpret_cast<u32x4*>(v.data + row * v.stride);
}

// Sums of N values over the T threads of a row, the same in all of them.  `buf`: [T / 64][N] floats, free again
// after the barrier of the next call but one (two buffers).
template <int T, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (T > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[w * N + i] = v[i];
    }
    __syncthreads();
    buf += threadIdx.x / T * (T / 64 * N);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = buf[i];
#pragma unroll
      for (int j = 1; j < T / 64; ++j) v[i] += buf[j * N + i];
    }
  }
}

template <int T, int C, bool RES>
__global__ __launch_bounds__(T < NT ? NT : T) void k_rms_norm(NormArgs a) {
  __shared__ float buf[T / 64];
  const int t = threadIdx.x % T, chunks = a.dim >> 3;
  const int64_t row = (int64_t)blockIdx.x * (T < NT ? NT / T : 1) + threadIdx.x / T;
  if (row >= a.rows) return;   // (a whole wave, and never one of several that wait for each other)
  const u32x4 zero = u32x4{0, 0, 0, 0}, one = u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  u32x4 xv[C], rv[C], wv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    const bool in = c < chunks;
    xv[i] = in ? row_of(a.x, row)[c] : zero;
    if (RES) rv[i] = in ? row_of(a.res, row)[c] : zero;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    wv[i] = one;
    if (a.w && c < chunks) wv[i] = reinterpret_cast<const u32x4*>(a.w)[c];
  }
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float f[8];
    unpack8(xv[i], f);
    if (RES) {
      float g[8];
      unpack8(rv[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      xv[i] = pack8(f);   // the norm is that of the sum as it is kept
      if (t + i * T < chunks) out_row(a.sum, row)[t + i * T] = xv[i];
      unpack8(xv[i], f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(f[j], f[j], ss[0]);
  }
  row_sum<T, 1>(ss, buf);
  const float r = 1.0f / sqrtf(ss[0] * a.inv_dim + a.eps);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (t + i * T >= chunks) continue;
    float f[8], w[8];
    unpack8(xv[i], f);
    unpack8(wv[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * r * w[j];
    out_row(a.y, row)[t + i * T] = pack8(f);
  }
}

// AHEAD: the next row's loads are issued before this row's sums are waited for (4096 x 4096 with dh 25.4 -> 24 us, without 20.3 ->
// 18.7), where the registers leave eight waves to a CU all the same (2048 x 8192 with dh, both kernels: 33.5 us without, 34.4 with).
constexpr bool bwd_ahead(int c, bool dh) { return c <= 2 || !dh; }
// Threads of a workgroup, rows of t threads.  Two rows of 256, which halves the partial weight gradients (2048 x 8192 27.0 -> 23.7 us
// in all, 1531 x 5000 16.2 -> 15.1, 4096 x 4096 with dh 26.5 -> 25.5), where the next rows' loads bridge the wait for each other
// (2048 x 8192 with dh: 33.5 us apart, 33.2 in pairs, no more than two runs differ).
constexpr int bwd_threads(int t, int c, bool dh) { return t < NT ? NT : t == 256 && bwd_ahead(c, dh) ? 512 : t; }

// The loads of a row in the backward.
template <int T, int C, bool DH>
struct BwdRow {
  u32x4 g[C], h[C], d[DH ? C : 1];
  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int t, int chunks) {
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = t + i * T;
      const bool in = c < chunks;
      g[i] = in ? row_of(a.x, row)[c] : zero;
      h[i] = in ? row_of(a.res, row)[c] : zero;
      if constexpr (DH) d[i] = in ? row_of(a.dh, row)[c] : zero;
    }
  }
};

template <int T, int C, bool DH>
__global__ __launch_bounds__(bwd_threads(T, C, DH)) void k_rms_norm_bwd(NormArgs a) {
  constexpr bool AHEAD = bwd_ahead(C, DH);
  constexpr int G = bwd_threads(T, C, DH) / T;   // rows of a workgroup at a time
  __shared__ float buf[2][T / 64 * 2 * G];
  __shared__ float sum[G > 1 ? (G - 1) * T * C * 8 : 1];
  const int t = threadIdx.x % T, chunks = a.dim >> 3;
  const u32x4 one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  float acc[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  u32x4 wv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    wv[i] = one;
    if (a.w && c < chunks) wv[i] = reinterpret_cast<const u32x4*>(a.w)[c];
  }
  const int64_t first = (int64_t)blockIdx.x * G + threadIdx.x / T, step = (int64_t)gridDim.x * G;
  BwdRow<T, C, DH> now, next;
  if (AHEAD && first < a.rows) next.load(a, first, t, chunks);
  int turn = 0;
  // (rows of several waves wait for each other's: as many turns for all)
  const int64_t lead = T > 64 ? threadIdx.x / T : 0;
  for (int64_t row = first; row - lead < a.rows; row += step, turn ^= 1) {
    const bool real = row < a.rows;
    if constexpr (AHEAD) {
      now = next;
      if (row + step < a.rows) next.load(a, row + step, t, chunks);
    } else if (real) {
      now.load(a, row, t, chunks);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float g[8], h[8], w[8];
      unpack8(now.g[i], g);
      unpack8(now.h[i], h);
      unpack8(wv[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = __builtin_fmaf(h[j], h[j], s[0]);
        s[1] = __builtin_fmaf(g[j] * h[j], w[j], s[1]);
      }
    }
    row_sum<T, 2>(s, buf[turn]);
    if (!real) break;
    const float r = 1.0f / sqrtf(s[0] * a.inv_dim + a.eps);
    const float m = s[1] * a.inv_dim * r * r;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float g[8], h[8], w[8], d[8];
      unpack8(now.g[i], g);
      unpack8(now.h[i], h);
      unpack8(wv[i], w);
      if constexpr (DH) unpack8(now.d[i], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = __builtin_fmaf(g[j] * h[j], r, acc[i][j]);
        const float v = __builtin_fmaf(-h[j], m, g[j] * w[j]);
        g[j] = DH ? __builtin_fmaf(r, v, d[j]) : r * v;
      }
      if (t + i * T < chunks) out_row(a.y, row)[t + i * T] = pack8(g);
    }
  }
  if (!a.part) return;
  if constexpr (G > 1) {   // the workgroup's waves, in their order
    const int w = threadIdx.x / T;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (w > 0) sum[((w - 1) * C * 8 + i * 8 + j) * T + t] = acc[i][j];
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < G - 1; ++k) acc[i][j] += sum[(k * C * 8 + i * 8 + j) * T + t];
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    if (c >= chunks) continue;
    float* const p = a.part + (int64_t)blockIdx.x * a.dim + c * 8;
    *reinterpret_cast<f32x4*>(p) = f32x4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
  }
}

// Rows too long for the registers of a workgroup: dy and h are read a second time (from the caches) after the sums
// (500 x 32768 with dh: 34.5 us, and 6.9 for the weight's gradient: 256 partials are 34 MB out and back beside 131 MB of operands; held in
// registers, most of which spill, 102).
template <bool DH>
__global__ __launch_bounds__(1024) void k_rms_norm_bwd_long(NormArgs a) {
  constexpr int T = 1024, C = 4;
  __shared__ float buf[2][T / 64 * 2];
  const int t = threadIdx.x, chunks = a.dim >> 3;
  const u32x4* const wp = reinterpret_cast<const u32x4*>(a.w);
  float acc[C][8] = {};
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = t + i * T;
      if (c >= chunks) continue;
      float g[8], h[8], w[8];
      unpack8(row_of(a.x, row)[c], g);
      unpack8(row_of(a.res, row)[c], h);
      if (a.w) unpack8(wp[c], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = __builtin_fmaf(h[j], h[j], s[0]);
        s[1] = __builtin_fmaf(g[j] * h[j], a.w ? w[j] : 1.0f, s[1]);
      }
    }
    row_sum<T, 2>(s, buf[turn]);
    const float r = 1.0f / sqrtf(s[0] * a.inv_dim + a.eps);
    const float m = s[1] * a.inv_dim * r * r;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = t + i * T;
      if (c >= chunks) continue;
      float g[8], h[8], w[8], d[8];
      unpack8(row_of(a.x, row)[c], g);
      unpack8(row_of(a.res, row)[c], h);
      if (a.w) unpack8(wp[c], w);
      if (DH) unpack8(row_of(a.dh, row)[c], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = __builtin_fmaf(g[j] * h[j], r, acc[i][j]);
        const float v = __builtin_fmaf(-h[j], m, g[j] * (a.w ? w[j] : 1.0f));
        g[j] = DH ? __builtin_fmaf(r, v, d[j]) : r * v;
      }
      out_row(a.y, row)[c] = pack8(g);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = t + i * T;
    if (c >= chunks) continue;
    float* const p = a.part + (int64_t)blockIdx.x * a.dim + c * 8;
    *reinterpret_cast<f32x4*>(p) = f32x4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
  }
}

// dw[c] = sum over n partials [n][dim]: 32 columns per workgroup (128 B of a partial), 32 threads per column.
constexpr int WT = 1024, WC = 32, WR = WT / WC, WL = 16;
__global__ __launch_bounds__(WT) void k_norm_weight_grad(const float* __restrict__ part, int n, int dim, float* __restrict__ dw) {
  __shared__ float sum[WR][WC + 1];
  const int c = threadIdx.x % WC, r = threadIdx.x / WC, col = blockIdx.x * WC + c;
  const int cc = col < dim ? col : dim - 1;
  float s = 0.0f;
  for (int i0 = r; i0 < n; i0 += WR * WL) {
    float v[WL];
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      const int i = i0 + j * WR;
      v[j] = i < n ? part[(int64_t)i * dim + cc] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < WL; ++j) s += v[j];
  }
  sum[r][c] = s;
  __syncthreads();
  if (r == 0 && col < dim) {
#pragma unroll
    for (int j = 1; j < WR; ++j) s += sum[j][c];
    dw[col] = s;
  }
}

// threads and loads of a row
struct Shape {
  int t, c;
};
Shape shape_of(int32_t dim) {
  const int chunks = dim / 8;
  if (chunks <= 64) return {64, 1};
  if (chunks <= 128) return {64, 2};
  if (chunks <= 256) return {64, 4};
  if (chunks <= 512) return {256, 2};
  if (chunks <= 768) return {256, 3};
  if (chunks <= 1024) return {256, 4};
  if (chunks <= 2048) return {1024, 2};
  return {1024, 4};
}

// of the backward
Shape bwd_shape_of(int32_t dim) {
  const Shape sh = shape_of(dim);
  return sh.t == 1024 && sh.c == 2 ? Shape{512, 4} : sh;
}
int64_t bwd_wgs(int64_t rows, const Shape& s, bool dh) {
  const int threads = bwd_threads(s.t, s.c, dh), per = threads / s.t;
  const int64_t wgs = (rows + per - 1) / per, most = threads >= 512 ? 256 : 512;
  return wgs < most ? wgs : most;
}

}  // namespace

// a launch with the flag, in workgroups of W1 and W0 threads with and without it, where the run-time shape is T x C
#define NORM_CASE(T, C, W1, W0, KT, KF)                               \
  if (sh.t == T && sh.c == C) {                                       \
    if (flag) hipLaunchKernelGGL(KT, g, dim3(W1), 0, s, a);           \
    else hipLaunchKernelGGL(KF, g, dim3(W0), 0, s, a);                \
  }
#define FWD_CASE(T, C) \
  NORM_CASE(T, C, T < NT ? NT : T, T < NT ? NT : T, (k_rms_norm<T, C, true>), (k_rms_norm<T, C, false>))
#define BWD_CASE(T, C)                                                             \
  NORM_CASE(T, C, bwd_threads(T, C, true), bwd_threads(T, C, false), (k_rms_norm_bwd<T, C, true>), \
            (k_rms_norm_bwd<T, C, false>))

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  const Shape sh = shape_of(a.dim);
  const int per = sh.t < NT ? NT / sh.t : 1;
  const dim3 g((unsigned)((a.rows + per - 1) / per));
  const bool flag = a.res.data != nullptr;
  ProfScope ps("k_rms_norm", s);
  FWD_CASE(64, 1)
  FWD_CASE(64, 2)
  FWD_CASE(64, 4)
  FWD_CASE(256, 2)
  FWD_CASE(256, 3)
  FWD_CASE(256, 4)
  FWD_CASE(1024, 2)
  FWD_CASE(1024, 4)
  return hipGetLastError();
}

// (with dh there are as many workgroups as without, or more)
size_t norm_part_floats(int64_t rows, int32_t dim) { return (size_t)bwd_wgs(rows, bwd_shape_of(dim), true) * dim; }

hipError_t launch_rms_norm_bwd(const NormArgs& a, float* dw, hipStream_t s) {
  const Shape sh = bwd_shape_of(a.dim);
  const int64_t wgs = bwd_wgs(a.rows, sh, a.dh.data != nullptr);
  {
    const dim3 g((unsigned)wgs);
    const bool flag = a.dh.data != nullptr;
    ProfScope ps("k_rms_norm_bwd", s);
    BWD_CASE(64, 1)
    BWD_CASE(64, 2)
    BWD_CASE(64, 4)
    BWD_CASE(256, 2)
    BWD_CASE(256, 3)
    BWD_CASE(256, 4)
    BWD_CASE(512, 4)
    NORM_CASE(1024, 4, 1024, 1024, (k_rms_norm_bwd_long<true>), (k_rms_norm_bwd_long<false>))
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.part) return hipSuccess;
  ProfScope ps("k_norm_weight_grad", s);
  hipLaunchKernelGGL(k_norm_weight_grad, dim3((unsigned)((a.dim + WC - 1) / WC)), dim3(WT), 0, s, a.part, (int)wgs, a.dim, dw);
  return hipGetLastError();
}

}  // namespace qlora
