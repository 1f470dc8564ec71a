// Internal launch interface of the operators on whole rows: the residual norm and the log
// probabilities.  Launchers validate nothing: rows_api.cpp has already.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "qlora.h"

namespace qlora {

// bf16 [rows][dim], rows `stride` elements apart
struct RowsView {
  uint16_t* data;
  int64_t stride;
};

#ifdef __HIPCC__
// Sums, maxima and prefix sums of a wave by data-parallel moves (shifts by 1, 2, 4, 8 within rows of 16 lanes, then the last
// lane of a row to the next one, and of the first half to the second): a few cycles a step where an exchange through LDS takes
// over a hundred.  The order is fixed.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or(uint32_t none, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false);
}
#define QL_WAVE_SCAN(STEP) STEP(0x111, 0xF) STEP(0x112, 0xF) STEP(0x114, 0xF) STEP(0x118, 0xF) STEP(0x142, 0xA) STEP(0x143, 0xC)
__device__ __forceinline__ float wave_sum(float v) {
#define QL_STEP(C, R) v += __uint_as_float(dpp_or<C, R>(0u, __float_as_uint(v)));
  QL_WAVE_SCAN(QL_STEP)
#undef QL_STEP
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {   // (NaN are passed over)
#define QL_STEP(C, R) v = fmaxf(v, __uint_as_float(dpp_or<C, R>(0xFF800000u, __float_as_uint(v))));
  QL_WAVE_SCAN(QL_STEP)
#undef QL_STEP
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define QL_STEP(C, R) v = max(v, dpp_or<C, R>(0u, v));
  QL_WAVE_SCAN(QL_STEP)
#undef QL_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ int wave_prefix(int v) {   // the sum up to and with this lane
#define QL_STEP(C, R) v += (int)dpp_or<C, R>(0u, (uint32_t)v);
  QL_WAVE_SCAN(QL_STEP)
#undef QL_STEP
  return v;
}
#undef QL_WAVE_SCAN
#endif

// ---- residual addition and norm (rms_norm.hip) ------------------------------------------------
struct NormArgs {
  RowsView x, res;    // forward: input and residual (or none); backward: dy and the forward's sum
  RowsView dh;        // backward: gradient of the sum besides (or none)
  RowsView y, sum;    // forward: outputs; backward: dx in y
  const uint16_t* w;  // or NULL
  int64_t rows;
  int32_t dim;
  float eps, inv_dim;
  float* part;        // backward: partial weight gradients [groups][dim], or NULL
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
// grows with the rows
size_t norm_part_floats(int64_t rows, int32_t dim);
hipError_t launch_rms_norm_bwd(const NormArgs& a, float* dw, hipStream_t s);

// ---- log probabilities of given tokens (logprob.hip) --------------------------------------------
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxSegs = 32;       // parts of a row at most
constexpr int64_t kLpMaxVocab = int64_t(1) << 20;
// One part of a row, of x in units of LpArgs::unit: the largest, the sum of exponentials from it, and that of each times its distance.
struct LpPart {
  float m, z, s;
  uint32_t pad_;
};
struct LpArgs {
  const void* x;              // bf16 or fp32 [rows][vocab]
  int64_t stride;             // elements between rows
  int64_t rows;
  int32_t vocab;
  int32_t fp32;
  float scale;
  float unit;                 // what the sums' logits are yet to be multiplied with: the scale, or 1 where it is applied first
  int32_t top;
  const int64_t* token;       // or NULL
  float* logprob;             // or NULL
  float* stats;               // [rows][2]
  float* entropy;             // or NULL
  float* top_lp;              // [rows][top]
  int64_t* top_index;
  LpPart* part;               // several parts: [rows][segs]
  unsigned long long* cand;   // and [rows][segs][top] candidates (order, then index)
  int32_t segs;
};
int lp_segments(int64_t rows, int64_t vocab, bool fp32);
hipError_t launch_logprob(const LpArgs& a, hipStream_t s);

struct LpBwdArgs {
  const void* x;
  void* dx;
  int64_t stride, dx_stride;
  int64_t rows;
  int32_t vocab;
  int32_t fp32;
  float scale;
  const int64_t* token;
  const float* stats;
  const float* dlp;       // or NULL
  const float* entropy;   // with dent
  const float* dent;      // or NULL
};
hipError_t launch_logprob_bwd(const LpBwdArgs& a, hipStream_t s);

}  // namespace qlora
