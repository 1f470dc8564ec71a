// The gated feed-forward block beside its products: the epilogue of the few-token forward, and the backward of activation
// and product.  (The products: k_fwd_nf4_gemm and k_gated_nf4_gemv.)
//
//   H = act(G) U;   dG = dH U act'(G),  dU = dH act(G)
#include "gated.h"
#include "gemm_core.h"
#include "kernels.h"

namespace qlora {

namespace {

using gemm::ld16;
using gemm::make_rsrc;
using gemm::rsrc_t;

struct EpiArgs {
  GatedSide side[2];   // gate, up
  int splits, asplits;
  size_t tpart;        // float offset of the adapter partials
  int64_t M, N, npad, rp, r;
  float scale;
  int act;
  uint16_t* H;
};

// Both sides' sums as k_gemv_epilogue forms them (partial sums in slice order, T = its partials in slice order, Ts = bf16(s T),
// plus Ts B), then the activation and the product.  64 columns of one 16-token group per workgroup; thread t takes
// column t % 64 for tokens t / 64 + 4 q.  The first 4 slices' loads of both sides are issued before any is used.  The ranks
// go through LDS 128 at a time: [2][16][ranks] floats of Ts, [2][ranks][64] bf16 of B.
constexpr int RANKS = 128;
__global__ __launch_bounds__(256) void k_gated_epilogue(EpiArgs a) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int t = threadIdx.x, rp = (int)a.rp, rl = min(rp, RANKS);
  float* const sTs = lds;
  uint16_t* const sB = reinterpret_cast<uint16_t*>(lds + 2 * 16 * rl);
  const int64_t n0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * 16;
  const int c = t & 63, mq = t >> 6;
  const int64_t n = n0 + c, nc = n < a.N ? n : a.N - 1;   // clamped column: every load stays inside the partials
  const int Mg = (int)min<int64_t>(16, a.M - m0), mcap = Mg - 1;
  constexpr int S0 = 4;
  float v[2][S0][4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* const part = a.side[k].partial + m0 * a.npad;
#pragma unroll
    for (int u = 0; u < S0; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[k][u][q] = part[((int64_t)min(u, a.splits - 1) * a.M + min(mq + 4 * q, mcap)) * a.npad + nc];
  }
  const uint32_t bend = (uint32_t)(a.r * a.N * 2);
  const rsrc_t rB[2] = {make_rsrc(a.side[0].B, bend), make_rsrc(a.side[1].B, bend)};
  float lora[2][4] = {};
  for (int j0 = 0; j0 < rp; j0 += RANKS) {
    const int jn = min(rp - j0, RANKS);   // 64 or 128
    // rows j0 .. of B for the 64 columns: jn * 8 chunks of 16 bytes a side (outside B: past its end, zero)
    uint4 bv[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int idx = t + 256 * u, jj = j0 + (idx >> 3), q = idx & 7;
        const bool ok = idx < jn * 8 && jj < a.r && n0 + q * 8 < a.N;
        bv[k][u] = ld16(rB[k], ok ? (uint32_t)((jj * a.N + n0 + q * 8) * 2) : bend);
      }
    if (j0) __syncthreads();   // (the last ranks are done with)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* const tp = a.side[k].partial + a.tpart + m0 * a.rp;
      uint16_t* const save = a.side[k].T_save && blockIdx.x == 0 ? a.side[k].T_save + m0 * a.r : nullptr;
      for (int e0 = t; e0 < Mg * jn; e0 += 4 * 256) {
        float ts[4] = {0.f, 0.f, 0.f, 0.f};
        int at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int idx = min(e0 + e * 256, Mg * jn - 1), m = idx / jn;
          at[e] = m * rp + j0 + idx - m * jn;
        }
        for (int s0 = 0; s0 < a.asplits; s0 += 4) {
          float tv[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) tv[u][e] = tp[(int64_t)min(s0 + u, a.asplits - 1) * a.M * a.rp + at[e]];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (s0 + u < a.asplits) ts[e] = __fadd_rn(ts[e], tv[u][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int idx = e0 + e * 256;
          if (idx >= Mg * jn) continue;
          const int m = idx / jn, jl = idx - m * jn, jj = j0 + jl;
          sTs[(k * 16 + m) * rl + jl] = jj < a.r ? bf16_to_f32(f32_to_bf16_bits(__fmul_rn(a.scale, ts[e]))) : 0.0f;
          if (save && jj < a.r) save[m * a.r + jj] = (uint16_t)f32_to_bf16_bits(ts[e]);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int idx = t + 256 * u;
        if (idx < jn * 8) *reinterpret_cast<uint4*>(sB + k * rl * 64 + idx * 8) = bv[k][u];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int jj = 0; jj < jn; jj += 4) {
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = bf16_to_f32(sB[k * rl * 64 + (jj + i) * 64 + c]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // (tokens past the group read what the LDS holds; their sums are not stored)
          const float4 tq = *reinterpret_cast<const float4*>(sTs + (k * 16 + mq + 4 * q) * rl + jj);
          lora[k][q] = __builtin_fmaf(tq.x, b[0], lora[k][q]);
          lora[k][q] = __builtin_fmaf(tq.y, b[1], lora[k][q]);
          lora[k][q] = __builtin_fmaf(tq.z, b[2], lora[k][q]);
          lora[k][q] = __builtin_fmaf(tq.w, b[3], lora[k][q]);
        }
      }
  }
  if (n >= a.N) return;
  float out[2][4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* const part = a.side[k].partial + m0 * a.npad;
    float acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[q] = v[k][0][q];
#pragma unroll
      for (int u = 1; u < S0; ++u)
        if (u < a.splits) acc[q] = __fadd_rn(acc[q], v[k][u][q]);
    }
    for (int sp = S0; sp < a.splits; ++sp) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        acc[q] = __fadd_rn(acc[q], part[((int64_t)sp * a.M + min(mq + 4 * q, mcap)) * a.npad + n]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) out[k][q] = __fadd_rn(acc[q], lora[k][q]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int m = mq + 4 * q;
    if (m >= Mg) continue;
    const int64_t at = (m0 + m) * a.N + n;
    a.H[at] = (uint16_t)f32_to_bf16_bits(activate(out[0][q], a.act) * out[1][q]);
    if (a.side[0].out) {
      a.side[0].out[at] = (uint16_t)f32_to_bf16_bits(out[0][q]);
      a.side[1].out[at] = (uint16_t)f32_to_bf16_bits(out[1][q]);
    }
  }
}

// Bound by HBM: 6 B read and 4 or 6 B written per element.  8 elements a thread.
template <bool H_OUT>
__global__ __launch_bounds__(256) void k_gated_bwd(const uint4* dH, const uint4* G, const uint4* U, int64_t n8, int act,
                                                   uint4* dG, uint4* dU, uint4* H) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {
    const uint4 dv = dH[i], gv = G[i], uv = U[i];
    const uint32_t d4[4] = {dv.x, dv.y, dv.z, dv.w}, g4[4] = {gv.x, gv.y, gv.z, gv.w}, u4[4] = {uv.x, uv.y, uv.z, uv.w};
    uint32_t og[4], ou[4], oh[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g[2], u[2], h[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto half = [&](uint32_t w) { return __uint_as_float(k ? w & 0xFFFF0000u : w << 16); };
        const float d = half(d4[j]), uu = half(u4[j]);
        float slope;
        const float act_g = activate(half(g4[j]), act, slope);
        g[k] = d * uu * slope;
        u[k] = d * act_g;
        h[k] = act_g * uu;
      }
      og[j] = pack_bf16x2(g[0], g[1]);
      ou[j] = pack_bf16x2(u[0], u[1]);
      oh[j] = pack_bf16x2(h[0], h[1]);
    }
    dG[i] = make_uint4(og[0], og[1], og[2], og[3]);
    dU[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    if (H_OUT) H[i] = make_uint4(oh[0], oh[1], oh[2], oh[3]);
  }
}

}  // namespace

hipError_t launch_gated_epilogue(const GatedSide& gate, const GatedSide& up, const GemvPlan& pl, int64_t M, int64_t N,
                                 int64_t r, float scale, int act, uint16_t* H, hipStream_t s) {
  const int64_t rp = (r + 63) / 64 * 64;
  const EpiArgs a{{gate, up}, pl.splits, pl.asplits, pl.tpart, M, N, pl.npad, rp, r, scale, act, H};
  const size_t lds = (size_t)(rp < RANKS ? rp : RANKS) * (2 * 16 * 4 + 2 * 64 * 2);
  ProfScope ps("k_gated_epilogue", s);
  hipLaunchKernelGGL(k_gated_epilogue, dim3((unsigned)((N + 63) / 64), (unsigned)pl.ngr), dim3(256), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const uint16_t* dH, const uint16_t* G, const uint16_t* U, int64_t n, int act, uint16_t* dG,
                            uint16_t* dU, uint16_t* H, hipStream_t s) {
  const int64_t n8 = n / 8, wgs = (n8 + 255) / 256;
  const dim3 g((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20)), b(256);
  ProfScope ps("k_gated_bwd", s);
  const auto in = [](const uint16_t* p) { return reinterpret_cast<const uint4*>(p); };
  const auto out = [](uint16_t* p) { return reinterpret_cast<uint4*>(p); };
  if (H) hipLaunchKernelGGL((k_gated_bwd<true>), g, b, 0, s, in(dH), in(G), in(U), n8, act, out(dG), out(dU), out(H));
  else hipLaunchKernelGGL((k_gated_bwd<false>), g, b, 0, s, in(dH), in(G), in(U), n8, act, out(dG), out(dU), out(H));
  return hipGetLastError();
}

}  // namespace qlora
