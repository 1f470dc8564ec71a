// What the few-token forward's kernels share with the K-sliced products: its parameters and the workgroups that form the
// partial sums of X A.
#pragma once

#include "common.h"
#include "gemm_core.h"
#include "kernels.h"

namespace qlora {
namespace gemv {

using gemm::i16x4;
using gemm::ld16;
using gemm::make_rsrc;
using gemm::rsrc_t;

constexpr int GT = 512;           // threads per workgroup (8 waves)
constexpr int GROWS = 64;         // adapter columns per adapter workgroup
constexpr int ACH = 64;           // rows of A per LDS chunk (8 KiB)
constexpr int XAS = 72;           // X chunk row stride in the adapter workgroups (64 + 8 padding)
constexpr size_t kLdsAdapter = 2 * ACH * 64 * 2 + 2 * 16 * XAS * 2 + 4 * 64 * 16;

struct GemvParams {
  const uint16_t* X;
  int64_t M, K, N;
  NF4View w;
  uint64_t codes_bytes, absmax_bytes, c1_bytes;
  const uint16_t* A;
  int64_t r;
  float* partial;       // weight partials [splits][M][npad]
  float* tpartial;      // adapter partials [asplits][M][rp]
  int64_t npad;         // rgroups * 16
  int64_t rp;
  int splits;           // weight slices of SLB blocks
  int64_t rgroups;      // 16-row groups
  int64_t rranges;      // weight workgroups per slice (contiguous ranges of row groups)
  int64_t agroups;      // adapter workgroups per adapter slice
  int asplits;
  int ka;               // rows of A per adapter slice (a multiple of 64)
  int ngr;              // 16-token groups
  NF4Table tab;
};

// Gated: what the up projection's half of the launch takes in place of the gate's
struct GemvSide {
  const uint8_t* codes;
  const void* absmax;
  const float* c1;
  const float* mu;
  const uint16_t* A;
  float* partial;
  float* tpartial;
};

// Natural [ACH][64] tile of A: row k = 128 bytes of eight 16-byte chunks; chunk q of row
// k sits at q ^ 2 f(k), f(k) = ((k >> 1) & 1) | ((k >> 2) & 2), which keeps the
// transposing reads (4 rows x 32 bytes per 16 lanes, two such row quads 8 apart per 32
// lanes) and the row stores (2 rows x 8 chunks per 16 lanes) conflict-free.
__device__ __forceinline__ int apos(int k, int q) {
  const int f = ((k >> 1) & 1) | ((k >> 2) & 2);
  return k * 64 + ((q ^ (f << 1)) << 3);
}

// ---- adapter workgroup: columns j0.. of A over a slice of ka rows; A is [K][r], columns
// past r read zero.  Loads run in groups of 4 chunks (of 64 rows), one group ahead; each
// chunk of A and of X is stored to LDS (two buffers) and taken by waves 0..3 (first 32 rows)
// and 4..7 (the rest).
__device__ __forceinline__ void adapter_group(const GemvParams& p, int bid, uint8_t* lds) {
  uint16_t* const sAb = reinterpret_cast<uint16_t*>(lds);      // [2][ACH * 64]
  uint16_t* const sXa = sAb + 2 * ACH * 64;                    // [2][16][XAS]
  float4* const sAcc = reinterpret_cast<float4*>(sXa + 2 * 16 * XAS);   // [4][64]
  const int nsp = p.asplits;
  const int tgi = bid % p.ngr;                                 // this workgroup's 16-token group
  const int rest = bid / p.ngr;
  const int grp = rest / nsp;
  const int split = rest - grp * nsp;
  const int m0 = tgi * 16;
  const int kb_beg = split * (p.ka / 64);
  const int nkb = (int)(p.K / 64);
  const int nkb_s = min(nkb, kb_beg + p.ka / 64) - kb_beg;      // blocks (64-row chunks) in this slice
  const int M = min((int)p.M - m0, 16);      // tokens of this group
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wq = wave & 3, par = wave >> 2;
  const int row = lane & 15, g = lane >> 4;
  const int xrow = row < M ? row : row % M;   // token rows past the group repeat real rows (outputs unused)
  const rsrc_t rX = make_rsrc(p.X, (uint64_t)p.M * p.K * 2);
  const uint32_t xend = (uint32_t)(p.M * p.K * 2);
  const int j0 = grp * GROWS;
  const rsrc_t rAd = make_rsrc(p.A, (uint64_t)p.K * p.r * 2);
  const uint32_t aend = (uint32_t)(p.K * p.r * 2);
  const int lr = t >> 3, lq = t & 7;                 // A load mapping: row lr, chunk lq
  const bool col_ok = j0 + lq * 8 < p.r;
  const bool xload = t < M * 8;                      // X load mapping: token t / 8, chunk t % 8
  const int xm = t >> 3;
  const int j = lane & 15, jc = wq * 16 + (j & 3) * 4;
  const int kr = par * 32 + g * 8 + (j >> 2);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  // chunks cb .. cb+3 into registers; chunks past the slice read zero (never stored)
  auto load4 = [&](int cb, uint4 (&va)[4], uint4 (&vx)[4]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = cb + u;
      const int k = (kb_beg + c) * 64 + lr;
      va[u] = ld16(rAd, col_ok && c < nkb_s ? (uint32_t)((k * (int)p.r + j0 + lq * 8) * 2) : aend);
      vx[u] = ld16(rX, xload && c < nkb_s ? (uint32_t)(((m0 + xm) * (int)p.K + (kb_beg + c) * 64 + lq * 8) * 2)
                                         : xend);
    }
  };
  auto proc4 = [&](int cb, const uint4 (&va)[4], const uint4 (&vx)[4]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (cb + u < nkb_s) {   // uniform
        const int buf = (cb + u) & 1;
        uint16_t* sAc = sAb + buf * (ACH * 64);
        uint16_t* sXc = sXa + buf * (16 * XAS);
        *reinterpret_cast<uint4*>(sAc + apos(lr, lq)) = va[u];
        *reinterpret_cast<uint4*>(sXc + (xload ? xm * XAS + lq * 8 : 15 * XAS + 64)) = vx[u];
        __syncthreads();
        // operand A: rows = columns jc = 16 (wave % 4) + l % 16 of A, 8 consecutive k per lane group
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(sAc + apos(kr, jc >> 3) + (jc & 7)));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(sAc + apos(kr + 4, jc >> 3) + (jc & 7)));
        const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
        u32x4 wa;
        wa.x = a.x; wa.y = a.y; wa.z = b.x; wa.w = b.y;
        const u32x4 xb = *reinterpret_cast<const u32x4*>(sXc + xrow * XAS + par * 32 + g * 8);
        acc = mfma16(wa, xb, acc);
      }
    }
  };
  // two groups of four chunks in flight: the loads of the next group are issued before the
  // current one is processed
  uint4 a0[4], x0[4], a1[4], x1[4];
  load4(0, a0, x0);
  for (int cb = 0; cb < nkb_s; cb += 8) {
    load4(cb + 4, a1, x1);
    proc4(cb, a0, x0);
    load4(cb + 8, a0, x0);
    proc4(cb + 4, a1, x1);
  }
  // waves 4..7 hand their sums to waves 0..3; acc[v] = C[column 4 g + v of the wave][token l % 16]
  if (par) sAcc[wq * 64 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (!par && row < M) {
    const float4 o = sAcc[wq * 64 + lane];
    const int64_t n = (int64_t)grp * GROWS + wq * 16 + 4 * g;
    float* dst = p.tpartial + ((int64_t)split * p.M + m0 + row) * p.rp + n;
    *reinterpret_cast<float4*>(dst) = make_float4(__fadd_rn(acc[0], o.x), __fadd_rn(acc[1], o.y),
                                                  __fadd_rn(acc[2], o.z), __fadd_rn(acc[3], o.w));
  }
}

// Parameters of a launch over the plan's slices (gemv.hip).
GemvParams gemv_params(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& w, const uint16_t* A, int64_t r,
                       const GemvPlan& pl, float* partial);

}  // namespace gemv
}  // namespace qlora
