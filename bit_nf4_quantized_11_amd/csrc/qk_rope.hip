// Norm of each head of q and k, and rotation by position, in one pass; and the backward.
//
//   r = 1 / sqrt(mean(x^2) + eps),  u = x r w  (u = x without a weight)
//   y = R(t) u:  (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * freq[i]
//   backward:  g = R(-t) dy,  dw = sum g x r,  dx = r (w g - x r^2 mean(w g x))
//
// 2 B read and 2 B written per element (4 B read in the backward): bound by HBM, for a few tokens
// by the launch and one memory round trip.  D / 16 lanes hold a head, 16 elements each: with pairs
// (i, i + rot / 2) the 16-byte chunks j and j + rot / 16, so that both members of a pair are in one
// lane and the same lane can take adjacent pairs just as well.  A wave holds 64 / (D / 16) heads of
// one row at a time and walks over the row's heads, so a lane's 8 angles are formed once per row
// and used for all of them.  The angle is reduced in float64, in revolutions (the unit of the sine
// instruction): pos * freq is exact to 2^-53 however far the position, the fraction is then
// exact in fp32 to 2^-25 revolutions, where an fp32 product at position 10^6 is off by 0.06 radians.
//
// Measured: 4096 rows of 32 + 32 heads of 128 with norms 26 us = 5.1 TB/s (a copy of 2 GiB: 4.8; part of the data is still in the
// 256 MB cache here), their backward at 2048 rows of 64 + 64 heads 38.6 us = 5.2 TB/s; 16 rows of 64 + 64 heads 3.7 us, which
// is one launch and two dependent loads.
#include "kernels.h"
#include "kv.h"

namespace qlora {

namespace {

constexpr int QT = 256;
constexpr int QW = QT / 64;
constexpr double kInv2Pi = 0.15915494309189533577;

struct Rot {
  float c[8], s[8];
};

// the 16 elements of a lane: chunk c0 in v[0..7], chunk c1 in v[8..15]
__device__ __forceinline__ void load16(const uint16_t* p, int c0, int c1, float (&v)[16]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p + c0 * 8), b = *reinterpret_cast<const uint4*>(p + c1 * 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store16(uint16_t* p, int c0, int c1, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p + c0 * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + c1 * 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Lane `sub` of a head: its two chunks.  Rotated ones first (j and j + rot / 16 for j < rot / 16),
// then what is left, two neighbours each.
__device__ __forceinline__ void chunks_of(int sub, int rot, int& c0, int& c1) {
  const int n = rot >> 4;
  c0 = sub < n ? sub : 2 * sub;
  c1 = sub < n ? sub + n : 2 * sub + 1;
}

template <bool INTER>
__device__ __forceinline__ Rot angles(const QkArgs& a, int64_t row, int c0, int c1, bool turn) {
  Rot r;
  const double p = (turn && a.pos) ? (double)a.pos[row] : 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // pair i of the lane: (v[i], v[8 + i]), or (v[2i], v[2i + 1])
    const int f = INTER ? (i < 4 ? 4 * c0 + i : 4 * c1 + i - 4) : 8 * c0 + i;
    const double t = turn ? p * ((double)a.freq[f] * kInv2Pi) : 0.0;
    const float x = (float)(t - rint(t));
    r.c[i] = __builtin_amdgcn_cosf(x);
    r.s[i] = __builtin_amdgcn_sinf(x);
  }
  return r;
}

template <bool INTER>
__device__ __forceinline__ void rotate(float (&v)[16], const Rot& r, float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 8 + i;
    const float x = v[ia], y = v[ib], s = r.s[i] * sign;
    v[ia] = __builtin_fmaf(x, r.c[i], -(y * s));
    v[ib] = __builtin_fmaf(y, r.c[i], x * s);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// sum over the L lanes of a head: lanes 1 and 2 away, then the other half of 8 and of 16 (mirrored)
template <int L>
__device__ __forceinline__ float head_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  if (L >= 8) v = dpp_add<0x141>(v);
  if (L >= 16) v = dpp_add<0x140>(v);
  return v;
}

template <int L>
__device__ __forceinline__ float inv_rms(const float (&v)[16], float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
  return 1.0f / sqrtf(head_sum<L>(ss) * (1.0f / (16 * L)) + eps);
}

// Wave items are (row, slice): slice i of a row takes its head groups i, i + slices, ...  (q's first).
template <int L, bool INTER>
__global__ __launch_bounds__(QT) void k_qk_norm_rope(QkArgs a) {
  constexpr int HP = 64 / L;
  const int lane = threadIdx.x & 63, sub = lane & (L - 1), hl = lane / L;
  const int64_t item = (int64_t)blockIdx.x * QW + (threadIdx.x >> 6);
  const int64_t row = item / a.slices;
  if (row >= a.rows) return;
  int c0, c1;
  chunks_of(sub, a.rot, c0, c1);
  const bool turn = sub < (a.rot >> 4);
  const Rot R = angles<INTER>(a, row, c0, c1, turn);
  const int gq = (a.q.n + HP - 1) / HP, gk = (a.k.n + HP - 1) / HP;
  for (int g = (int)(item - row * a.slices); g < gq + gk; g += a.slices) {
    const bool isq = g < gq;
    const Heads& in = isq ? a.q : a.k;
    const Heads& out = isq ? a.qo : a.ko;
    const uint16_t* w = isq ? a.wq : a.wk;
    const int h = (isq ? g : g - gq) * HP + hl;
    if (h >= in.n) continue;   // the lanes of a head leave together
    float v[16];
    load16(in.data + row * in.rs + h * in.hs, c0, c1, v);
    if (w) {
      const float r = inv_rms<L>(v, a.eps);
      float wv[16];
      load16(w, c0, c1, wv);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * r * wv[i];
    }
    if (turn) rotate<INTER>(v, R, 1.0f);
    store16(out.data + row * out.rs + h * out.hs, c0, c1, v);
  }
}

// The backward walks over the items with a fixed grid: each lane sums the weight gradients of its 16
// columns over all heads and rows it meets, the workgroup adds its lanes and waves in a fixed order
// and writes one partial of both; k_qk_weight_grad adds the partials.
template <int L, bool INTER>
__global__ __launch_bounds__(QT, 4) void k_qk_norm_rope_bwd(QkArgs a) {
  constexpr int HP = 64 / L, D = 16 * L;
  __shared__ __attribute__((aligned(16))) float sum[QW][2][D];
  const int lane = threadIdx.x & 63, sub = lane & (L - 1), hl = lane / L, wave = threadIdx.x >> 6;
  int c0, c1;
  chunks_of(sub, a.rot, c0, c1);
  const bool turn = sub < (a.rot >> 4);
  const int gq = (a.q.n + HP - 1) / HP, gk = (a.k.n + HP - 1) / HP;
  float dw[2][16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[0][i] = dw[1][i] = 0.0f;
  const int64_t items = a.rows * a.slices, step = (int64_t)gridDim.x * QW;
  for (int64_t item = (int64_t)blockIdx.x * QW + wave; item < items; item += step) {
    const int64_t row = item / a.slices;
    const Rot R = angles<INTER>(a, row, c0, c1, turn);
    for (int g = (int)(item - row * a.slices); g < gq + gk; g += a.slices) {
      const bool isq = g < gq;
      const Heads& in = isq ? a.q : a.k;
      const Heads& xin = isq ? a.xq : a.xk;
      const Heads& out = isq ? a.qo : a.ko;
      const uint16_t* w = isq ? a.wq : a.wk;
      const int h = (isq ? g : g - gq) * HP + hl;
      if (h >= in.n) continue;
      float v[16];
      load16(in.data + row * in.rs + h * in.hs, c0, c1, v);
      if (w) {
        float x[16], wv[16];
        load16(xin.data + row * xin.rs + h * xin.hs, c0, c1, x);
        load16(w, c0, c1, wv);
        if (turn) rotate<INTER>(v, R, -1.0f);
        const float r = inv_rms<L>(x, a.eps);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float gx = v[i] * x[i];
          if (isq) dw[0][i] = __builtin_fmaf(gx, r, dw[0][i]);
          else dw[1][i] = __builtin_fmaf(gx, r, dw[1][i]);
          v[i] *= wv[i];
          dot = __builtin_fmaf(gx, wv[i], dot);
        }
        const float m = head_sum<L>(dot) * (1.0f / D) * r * r;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = r * __builtin_fmaf(-x[i], m, v[i]);
      } else if (turn) {
        rotate<INTER>(v, R, -1.0f);
      }
      store16(out.data + row * out.rs + h * out.hs, c0, c1, v);
    }
  }
  if (!a.part) return;
  // The wave's heads, halving the values with each exchange: lanes 32 .. 63 go on with the keys' weight, then odd rows of
  // 16 lanes with the second chunk.  (Through LDS, 32 values over 64 / L heads each, it was 4 us of a call that takes 10.)
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(dw[0][i]), __float_as_uint(dw[1][i]), false, false);
    v[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 8]), false, false);
    v[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    if (L <= 8) v[i] = dpp_add<0x128>(v[i]);   // row_ror 8
    if (L <= 4) v[i] = dpp_add<0x124>(v[i]);   // row_ror 4
  }
  if ((lane & 15) < L) {
    float* const p = &sum[wave][lane >> 5][(lane & 16 ? c1 : c0) * 8];
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += QT) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < QW; ++w) s += sum[w][i / D][i % D];
    a.part[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[t][d] = sum over n partials [n][2][D]: 16 columns per workgroup, 64 threads per column with up to 16 loads each in
// flight (1024 partials are one round trip to memory).
constexpr int WT = 1024, WR = WT / 16, WL = 16;
__global__ __launch_bounds__(WT) void k_qk_weight_grad(const float* __restrict__ part, int n, int D, float* dwq,
                                                       float* dwk) {
  __shared__ float sum[WR][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.0f;
  for (int i0 = r; i0 < n; i0 += WR * WL) {
    float v[WL];
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      const int i = i0 + j * WR;
      v[j] = i < n ? part[(int64_t)i * 2 * D + col] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < WL; ++j) s += v[j];
  }
  sum[r][c] = s;
  __syncthreads();
  // wave w: column w
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  s = sum[lane][w];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off, 64);
  const int out_col = blockIdx.x * 16 + w;
  float* out = out_col < D ? dwq : dwk;
  if (out && lane == 0) out[out_col < D ? out_col : out_col - D] = s;
}

int head_groups(int32_t q_heads, int32_t k_heads, int D) {
  const int hp = 64 / (D / 16);
  return (q_heads + hp - 1) / hp + (k_heads + hp - 1) / hp;
}

// Wave items per row: one, unless the rows are too few to give each CU 8 waves.
int slices_for(int64_t rows, int groups) {
  int64_t s = (2048 + rows - 1) / rows;
  return (int)(s < groups ? s : groups);
}

}  // namespace

// K<D / 16, interleaved> launched for the run-time D and pairing
#define QK_LAUNCH(K, g, ...)                                                              \
  do {                                                                                    \
    const dim3 t_(QT);                                                                    \
    if (D == 64 && inter) hipLaunchKernelGGL((K<4, true>), g, t_, 0, s, __VA_ARGS__);     \
    else if (D == 64) hipLaunchKernelGGL((K<4, false>), g, t_, 0, s, __VA_ARGS__);        \
    else if (D == 128 && inter) hipLaunchKernelGGL((K<8, true>), g, t_, 0, s, __VA_ARGS__); \
    else if (D == 128) hipLaunchKernelGGL((K<8, false>), g, t_, 0, s, __VA_ARGS__);       \
    else if (inter) hipLaunchKernelGGL((K<16, true>), g, t_, 0, s, __VA_ARGS__);          \
    else hipLaunchKernelGGL((K<16, false>), g, t_, 0, s, __VA_ARGS__);                    \
  } while (0)

hipError_t launch_qk(const QkArgs& a0, int D, bool inter, hipStream_t s) {
  QkArgs a = a0;
  a.slices = slices_for(a.rows, head_groups(a.q.n, a.k.n, D));
  const dim3 g((unsigned)((a.rows * a.slices + QW - 1) / QW));
  ProfScope ps("k_qk_norm_rope", s);
  QK_LAUNCH(k_qk_norm_rope, g, a);
  return hipGetLastError();
}

static int bwd_grid(int64_t items) {
  const int64_t g = (items + QW - 1) / QW;
  return (int)(g < 1024 ? g : 1024);
}

int qk_bwd_partials(int64_t rows, int32_t q_heads, int32_t k_heads, int D) {
  return bwd_grid(rows * head_groups(q_heads, k_heads, D));   // a row has as many slices as groups at most
}

hipError_t launch_qk_bwd(const QkArgs& a0, int D, bool inter, float* dwq, float* dwk, hipStream_t s) {
  QkArgs a = a0;
  a.slices = slices_for(a.rows, head_groups(a.q.n, a.k.n, D));
  const int grid = bwd_grid(a.rows * a.slices);
  {
    const dim3 g((unsigned)grid);
    ProfScope ps("k_qk_norm_rope_bwd", s);
    QK_LAUNCH(k_qk_norm_rope_bwd, g, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.part) return hipSuccess;
  ProfScope ps("k_qk_weight_grad", s);
  hipLaunchKernelGGL(k_qk_weight_grad, dim3((unsigned)(2 * D / 16)), dim3(WT), 0, s, a.part, grid, D, dwq, dwk);
  return hipGetLastError();
}

}  // namespace qlora
