// The gated feed-forward block beside its products: the epilogue of the few-token forward, and the backward of activation
// and product.  (The products: k_fwd_nf4_gemm and k_gated_nf4_gemv.)
//
//   H = act(G) U;   dG = dH U act'(G),  dU = dH act(G)
#include "gated.h"
#include "gemm_core.h"
#include "kernels.h"

namespace qlora {

namespace {

using gemm::i16x4;
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

// Natural [ranks][64] tile of B: row j = 128 bytes of eight 16-byte chunks, chunk q at q ^ 2 f(j), which keeps the
// transposing reads (4 rows x 32 bytes per 16 lanes, two such row quads 8 apart per 32 lanes) free of conflicts.
__device__ __forceinline__ int bpos(int j, int q) {
  const int f = ((j >> 1) & 1) | ((j >> 2) & 2);
  return j * 64 + ((q ^ (f << 1)) << 3);
}

// Both sides' sums (partial sums in slice order, T = its partials in slice order, Ts = bf16(s T), plus Ts B by matrix
// instructions: these take bf16, and it is what the linear layer does.  Half a step of s T: G, U and H differ by 5e-4 to 1e-3 of their norms
// from those of an fp32 T, by flips of their own last rounding, and are as far from the exact ones, 0.0017), then the activation and the product.  64 features of one 16-token group per workgroup, 16 to a wave; lane l
// holds features 4 (l / 16) .. + 3 of token l % 16, as the matrix instruction leaves them.  Bound by latency: the first 4
// slices' loads and B's are issued before any is used.  The ranks go through LDS 128 at a time.
// (16 tokens, 22016 features, rank 64, 4 slices: 6.8 us, where the partial sums are 11.3 MB; with Ts B by fp32 multiply-adds out of
// LDS 11.2.  256 tokens, 5504 features, 2 slices: 12.4 us; with loads of as many slices and ranks at all times 15.1, with two blocks
// of features to a workgroup 16.9.)
constexpr int RANKS = 128, TPAD = 8, S0 = 4;
__global__ __launch_bounds__(256) void k_gated_epilogue(EpiArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int rp = (int)a.rp, rl = min(rp, RANKS), ts_ld = rl + TPAD;
  uint16_t* const sT = lds;                          // [2][16][ts_ld] of Ts
  uint16_t* const sB = lds + 2 * 16 * ts_ld;         // [2][rl][64]
  const int64_t n0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * 16;
  const int tok = lane & 15, g = lane >> 4;
  const int Mg = (int)min<int64_t>(16, a.M - m0);
  const int64_t n = n0 + wave * 16 + 4 * g;          // this lane's features
  const int64_t at = (m0 + min(tok, Mg - 1)) * a.npad + min(n, a.npad - 4), slice = a.M * a.npad;
  f32x4 v[2][S0];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int u = 0; u < S0; ++u)
      if (u < a.splits) v[k][u] = *reinterpret_cast<const f32x4*>(a.side[k].partial + u * slice + at);
  const uint32_t bend = (uint32_t)(a.r * a.N * 2);
  const rsrc_t rB[2] = {make_rsrc(a.side[0].B, bend), make_rsrc(a.side[1].B, bend)};
  f32x4 lora[2] = {};
  for (int j0 = 0; j0 < rp; j0 += RANKS) {
    const int jn = min(rp - j0, RANKS);   // 64 or 128
    // rows j0 .. of B for the 64 features: jn * 8 chunks of 16 bytes a side (outside B: past its end, zero)
    uint4 bv[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int idx = t + 256 * u, jj = j0 + (idx >> 3), q = idx & 7;
        const bool ok = jj < a.r && n0 + q * 8 < a.N;
        if (256 * u < jn * 8) bv[k][u] = ld16(rB[k], ok ? (uint32_t)((jj * a.N + n0 + q * 8) * 2) : bend);
      }
    if (j0) __syncthreads();   // (the last ranks are done with)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* const tp = a.side[k].partial + a.tpart + m0 * a.rp;
      uint16_t* const save = a.side[k].T_save && blockIdx.x == 0 ? a.side[k].T_save + m0 * a.r : nullptr;
      for (int e = t; e < Mg * (jn >> 2); e += 256) {
        const int m = e / (jn >> 2), jl = (e - m * (jn >> 2)) * 4, jj = j0 + jl;
        const float* const p = tp + m * rp + jj;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < a.asplits; s0 += 4) {
          f32x4 tv[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) tv[u] = *reinterpret_cast<const f32x4*>(p + (int64_t)min(s0 + u, a.asplits - 1) * a.M * a.rp);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (s0 + u < a.asplits)
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] = __fadd_rn(sum[i], tv[u][i]);
        }
        uint32_t ts[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (r is a multiple of 8: the four ranks are all below it or none)
          ts[i] = jj < a.r ? f32_to_bf16_bits(__fmul_rn(a.scale, sum[i])) : 0u;
          if (save && jj < a.r) save[m * a.r + jj + i] = (uint16_t)f32_to_bf16_bits(sum[i]);
        }
        *reinterpret_cast<uint2*>(sT + (k * 16 + m) * ts_ld + jl) = make_uint2(ts[0] | ts[1] << 16, ts[2] | ts[3] << 16);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int idx = t + 256 * u;
        if (idx < jn * 8) *reinterpret_cast<uint4*>(sB + k * rl * 64 + bpos(idx >> 3, idx & 7)) = bv[k][u];
      }
    }
    __syncthreads();
    const int j = lane & 15, jc = wave * 16 + (j & 3) * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int ks = 0; ks < jn; ks += 32) {
        const uint16_t* const b = sB + k * rl * 64;
        const int kr = ks + g * 8 + (j >> 2);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(b + bpos(kr, jc >> 3) + (jc & 7)));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(b + bpos(kr + 4, jc >> 3) + (jc & 7)));
        const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
        const u32x4 wa = {x.x, x.y, y.x, y.y};
        // (rows of tokens past the group hold whatever the LDS does; their sums are not stored)
        const u32x4 tb = *reinterpret_cast<const u32x4*>(sT + (k * 16 + tok) * ts_ld + ks + g * 8);
        lora[k] = mfma16(wa, tb, lora[k]);
      }
  }
  if (n >= a.N || tok >= Mg) return;
  f32x4 out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    f32x4 acc = v[k][0];
#pragma unroll
    for (int u = 1; u < S0; ++u)
      if (u < a.splits)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __fadd_rn(acc[i], v[k][u][i]);
    for (int s0 = S0; s0 < a.splits; s0 += S0) {
      f32x4 w[S0];
#pragma unroll
      for (int u = 0; u < S0; ++u) w[u] = *reinterpret_cast<const f32x4*>(a.side[k].partial + min(s0 + u, a.splits - 1) * slice + at);
#pragma unroll
      for (int u = 0; u < S0; ++u)
        if (s0 + u < a.splits)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = __fadd_rn(acc[i], w[u][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) out[k][i] = __fadd_rn(acc[i], lora[k][i]);
  }
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = activate(out[0][i], a.act) * out[1][i];
  const auto put = [&](uint16_t* p, float a0, float a1, float a2, float a3) {
    *reinterpret_cast<uint2*>(p + (m0 + tok) * a.N + n) = make_uint2(pack_bf16x2(a0, a1), pack_bf16x2(a2, a3));
  };
  put(a.H, h[0], h[1], h[2], h[3]);
  if (a.side[0].out) {
    put(a.side[0].out, out[0][0], out[0][1], out[0][2], out[0][3]);
    put(a.side[1].out, out[1][0], out[1][1], out[1][2], out[1][3]);
  }
}

// The tiles that the large forward left in slices: their sums in slice order, then activation and product.  4 features a
// thread; bound by memory (8 B read per slice and output, mostly from the caches, where they have just been written).
__global__ __launch_bounds__(256) void k_gated_finish(const float* gate, const float* up, int slices, int64_t npad, int64_t rows,
                                                      int64_t N, int64_t m0, int64_t n0, int act, uint16_t* H, uint16_t* G,
                                                      uint16_t* U) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = npad / 4;
  const int64_t m = i / per_row, c = (i - m * per_row) * 4, n = n0 + c;
  if (m >= rows || n >= N) return;
  const int64_t slice = 256 * npad, at = m * npad + c;
  f32x4 v[2][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t o = min(u, slices - 1) * slice + at;
    v[0][u] = *reinterpret_cast<const f32x4*>(gate + o);
    v[1][u] = *reinterpret_cast<const f32x4*>(up + o);
  }
#pragma unroll
  for (int u = 1; u < 4; ++u)
    if (u < slices) {
      v[0][0] += v[0][u];
      v[1][0] += v[1][u];
    }
  float h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = activate(v[0][0][j], act) * v[1][0][j];
  const int64_t o = (m0 + m) * N + n;
  *reinterpret_cast<uint2*>(H + o) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
  if (G) {
    *reinterpret_cast<uint2*>(G + o) = make_uint2(pack_bf16x2(v[0][0][0], v[0][0][1]), pack_bf16x2(v[0][0][2], v[0][0][3]));
    *reinterpret_cast<uint2*>(U + o) = make_uint2(pack_bf16x2(v[1][0][0], v[1][0][1]), pack_bf16x2(v[1][0][2], v[1][0][3]));
  }
}

// Bound by HBM: 6 B read and 4 or 6 B written per element.  8 elements a thread.  2048 x 11008 with H: 41 us = 6.5 TB/s where part
// of it is cached, 50 us = 5.4 TB/s where not (a copy: 5.1).
// GRAD: dG and dU (else H alone, from 4 B read).
template <bool GRAD, bool H_OUT>
__global__ __launch_bounds__(256) void k_gated_bwd(const uint4* dH, const uint4* G, const uint4* U, int64_t n8, int act,
                                                   uint4* dG, uint4* dU, uint4* H) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {
    const uint4 dv = GRAD ? dH[i] : make_uint4(0, 0, 0, 0), gv = G[i], uv = U[i];
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
    if (GRAD) {
      dG[i] = make_uint4(og[0], og[1], og[2], og[3]);
      dU[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
    if (H_OUT) H[i] = make_uint4(oh[0], oh[1], oh[2], oh[3]);
  }
}

}  // namespace

hipError_t launch_gated_epilogue(const GatedSide& gate, const GatedSide& up, const GemvPlan& pl, int64_t M, int64_t N,
                                 int64_t r, float scale, int act, uint16_t* H, hipStream_t s) {
  const int64_t rp = (r + 63) / 64 * 64;
  const EpiArgs a{{gate, up}, pl.splits, pl.asplits, pl.tpart, M, N, pl.npad, rp, r, scale, act, H};
  const int64_t rl = rp < RANKS ? rp : RANKS;
  const size_t lds = (size_t)(2 * 16 * (rl + TPAD) + 2 * rl * 64) * 2;   // at most 41 KB
  ProfScope ps("k_gated_epilogue", s);
  hipLaunchKernelGGL(k_gated_epilogue, dim3((unsigned)((N + 63) / 64), (unsigned)pl.ngr), dim3(256), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_gated_finish(const float* gate_partial, const float* up_partial, const GatedTail& tail, int64_t M, int64_t N,
                               int64_t m0, int64_t n0, int act, uint16_t* H, uint16_t* G, uint16_t* U, hipStream_t s) {
  const int64_t rows = M - m0, wgs = (rows * (tail.npad / 4) + 255) / 256;
  ProfScope ps("k_gated_finish", s);
  hipLaunchKernelGGL(k_gated_finish, dim3((unsigned)wgs), dim3(256), 0, s, gate_partial, up_partial, tail.slices, tail.npad, rows,
                     N, m0, n0, act, H, G, U);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const uint16_t* dH, const uint16_t* G, const uint16_t* U, int64_t n, int act, uint16_t* dG,
                            uint16_t* dU, uint16_t* H, hipStream_t s) {
  const int64_t n8 = n / 8, wgs = (n8 + 255) / 256;
  const dim3 g((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20)), b(256);
  ProfScope ps("k_gated_bwd", s);
  const auto in = [](const uint16_t* p) { return reinterpret_cast<const uint4*>(p); };
  const auto out = [](uint16_t* p) { return reinterpret_cast<uint4*>(p); };
  if (!dH) hipLaunchKernelGGL((k_gated_bwd<false, true>), g, b, 0, s, in(dH), in(G), in(U), n8, act, out(dG), out(dU), out(H));
  else if (H) hipLaunchKernelGGL((k_gated_bwd<true, true>), g, b, 0, s, in(dH), in(G), in(U), n8, act, out(dG), out(dU), out(H));
  else hipLaunchKernelGGL((k_gated_bwd<true, false>), g, b, 0, s, in(dH), in(G), in(U), n8, act, out(dG), out(dU), out(H));
  return hipGetLastError();
}

}  // namespace qlora
