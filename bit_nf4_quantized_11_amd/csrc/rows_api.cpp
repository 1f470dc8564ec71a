// Entry points of the operators on whole rows: the residual norm and the log probabilities of given tokens
// (include/qlora.h).  Validates every argument on the host, then launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "host.h"
#include "kernels.h"
#include "qlora.h"
#include "rows.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 22;       // workgroups times threads of a launch stay below 2^32
constexpr int64_t kMaxLogits = int64_t(1) << 35;
constexpr int64_t kMaxStride = int64_t(1) << 36;
constexpr int32_t kMaxDim = 32768;

qlora_status check_norm(int64_t rows, int32_t dim, const uint16_t* w, float eps) {
  if (rows < 0 || rows >= kMaxRows || dim < 8 || dim > kMaxDim || dim % 8 != 0) return QLORA_ERR_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return QLORA_ERR_UNSUPPORTED;
  if (!aligned16(w)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// Rows of bf16.  `out`: they must not overlap.
qlora_status check_rows(const uint16_t* p, int64_t stride, int64_t rows, int32_t dim, bool out) {
  if (rows == 0) return QLORA_OK;
  if (!p) return QLORA_ERR_NULL;
  if (!aligned16(p)) return QLORA_ERR_ALIGN;
  if (rows == 1) return QLORA_OK;
  if (stride < 0 || stride >= kMaxStride || (out && stride < dim)) return QLORA_ERR_SHAPE;
  return stride % 8 == 0 ? QLORA_OK : QLORA_ERR_ALIGN;
}

// Output rows that begin where input rows do are those rows: with another stride they would overlap others.
bool in_place_ok(const void* out, int64_t out_stride, const void* in, int64_t in_stride, int64_t rows) {
  return out != in || out_stride == in_stride || rows <= 1;
}

RowsView view(const uint16_t* p, int64_t stride) { return RowsView{const_cast<uint16_t*>(p), stride}; }

bool dtype_ok(int32_t d) { return d == QLORA_BF16 || d == QLORA_FP32; }
bool aligned_for(const void* p, int32_t dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == QLORA_FP32 ? 3u : 1u)) == 0; }

qlora_status check_logits(const void* x, int64_t stride, int64_t rows, int64_t vocab, int32_t dtype, float scale, bool out) {
  if (rows < 0 || rows >= kMaxRows || vocab < 1 || vocab > kLpMaxVocab || rows * vocab >= kMaxLogits) return QLORA_ERR_SHAPE;
  if (!dtype_ok(dtype)) return QLORA_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return QLORA_ERR_UNSUPPORTED;
  if (rows == 0) return QLORA_OK;
  if (!x) return QLORA_ERR_NULL;
  if (!aligned_for(x, dtype)) return QLORA_ERR_ALIGN;
  if (rows > 1 && (stride < 0 || stride >= kMaxStride || (out && stride < vocab))) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

struct LpWs {
  LpPart* part;
  unsigned long long* cand;
  size_t bytes;
};
LpWs lp_layout(void* base, int64_t rows, int64_t segs, int32_t top) {
  Carve c(base);
  LpWs w;
  w.part = c.take<LpPart>((size_t)rows * segs);
  w.cand = c.take<unsigned long long>((size_t)rows * segs * top);
  w.bytes = round_up(c.off, 256);
  return w;
}
// Parts of a call with at most these rows and logits: a row is cut into pieces of 16384 logits at least, or smaller ones while
// all rows together have fewer than 128, so into no more than 256 in all then.  0 where every row is whole.
int64_t lp_most_parts(int64_t rows, int64_t vocab) {
  if (vocab <= (rows < 128 ? 32768 : 16384)) return 0;
  const int64_t per_row = (vocab + 16383) / 16384;
  return std::max<int64_t>(256, per_row > 1 ? rows * per_row : 0);
}
int64_t lp_parts(int64_t rows, int64_t vocab, int32_t dtype) { return lp_segments(rows, vocab, dtype == QLORA_FP32); }

}  // namespace

extern "C" {

qlora_status qlora_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, int64_t residual_stride,
                            int64_t rows, int32_t dim, const uint16_t* weight, float eps, uint16_t* y, int64_t y_stride,
                            uint16_t* sum, int64_t sum_stride, hipStream_t stream) {
  qlora_status st = check_norm(rows, dim, weight, eps);
  if (st != QLORA_OK) return st;
  if ((residual == nullptr) != (sum == nullptr) && rows > 0) return QLORA_ERR_NULL;
  if ((st = check_rows(x, x_stride, rows, dim, false)) != QLORA_OK) return st;
  if ((st = check_rows(y, y_stride, rows, dim, true)) != QLORA_OK) return st;
  if (residual) {
    if ((st = check_rows(residual, residual_stride, rows, dim, false)) != QLORA_OK) return st;
    if ((st = check_rows(sum, sum_stride, rows, dim, true)) != QLORA_OK) return st;
    if (rows > 0 && y == sum) return QLORA_ERR_SHAPE;
    if (!in_place_ok(y, y_stride, residual, residual_stride, rows) || !in_place_ok(sum, sum_stride, x, x_stride, rows) ||
        !in_place_ok(sum, sum_stride, residual, residual_stride, rows))
      return QLORA_ERR_SHAPE;
  }
  if (!in_place_ok(y, y_stride, x, x_stride, rows)) return QLORA_ERR_SHAPE;
  if (rows == 0) return QLORA_OK;
  NormArgs a{};
  a.x = view(x, x_stride);
  a.res = view(residual, residual_stride);
  a.y = view(y, y_stride);
  a.sum = view(sum, sum_stride);
  a.w = weight;
  a.rows = rows;
  a.dim = dim;
  a.eps = eps;
  a.inv_dim = 1.0f / (float)dim;
  QL_HIP(launch_rms_norm(a, stream));
  return QLORA_OK;
}

size_t qlora_rms_norm_bwd_workspace(int64_t rows, int32_t dim) {
  if (check_norm(rows, dim, nullptr, 0.0f) != QLORA_OK) return 0;
  return round_up(norm_part_floats(std::max<int64_t>(rows, 1), dim) * sizeof(float), 256);
}

qlora_status qlora_rms_norm_bwd(const uint16_t* dy, int64_t dy_stride, const uint16_t* h, int64_t h_stride,
                                const uint16_t* dh, int64_t dh_stride, int64_t rows, int32_t dim, const uint16_t* weight,
                                float eps, uint16_t* dx, int64_t dx_stride, float* dweight, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  qlora_status st = check_norm(rows, dim, weight, eps);
  if (st != QLORA_OK) return st;
  if (dweight && !weight) return QLORA_ERR_NULL;
  if (!aligned4(dweight)) return QLORA_ERR_ALIGN;
  if ((st = check_rows(dy, dy_stride, rows, dim, false)) != QLORA_OK) return st;
  if ((st = check_rows(h, h_stride, rows, dim, false)) != QLORA_OK) return st;
  if (dh && (st = check_rows(dh, dh_stride, rows, dim, false)) != QLORA_OK) return st;
  if ((st = check_rows(dx, dx_stride, rows, dim, true)) != QLORA_OK) return st;
  if (!in_place_ok(dx, dx_stride, dy, dy_stride, rows) || !in_place_ok(dx, dx_stride, h, h_stride, rows) ||
      !in_place_ok(dx, dx_stride, dh, dh_stride, rows))
    return QLORA_ERR_SHAPE;
  if (dweight) {
    if (!ws || ws_bytes < qlora_rms_norm_bwd_workspace(rows, dim)) return QLORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  }
  if (rows == 0) {
    if (dweight) QL_HIP(launch_fill_u32(reinterpret_cast<uint32_t*>(dweight), dim, 0u, stream));
    return QLORA_OK;
  }
  NormArgs a{};
  a.x = view(dy, dy_stride);
  a.res = view(h, h_stride);
  a.dh = view(dh, dh_stride);
  a.y = view(dx, dx_stride);
  a.w = weight;
  a.rows = rows;
  a.dim = dim;
  a.eps = eps;
  a.inv_dim = 1.0f / (float)dim;
  a.part = dweight ? static_cast<float*>(ws) : nullptr;
  QL_HIP(launch_rms_norm_bwd(a, dweight, stream));
  return QLORA_OK;
}

size_t qlora_token_logprob_workspace(int64_t rows, int64_t vocab, int32_t top) {
  if (rows < 0 || rows >= kMaxRows || vocab < 1 || vocab > kLpMaxVocab || rows * vocab >= kMaxLogits || top < 0 ||
      top > kLpMaxTop)
    return 0;
  return lp_layout(nullptr, 1, lp_most_parts(rows, vocab), top).bytes;
}

qlora_status qlora_token_logprob(const void* logits, int64_t stride, int64_t rows, int64_t vocab, int32_t dtype,
                                 const int64_t* token, float scale, int32_t top, float* logprob, float* stats,
                                 float* entropy, float* top_logprob, int64_t* top_index, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  const qlora_status st = check_logits(logits, stride, rows, vocab, dtype, scale, false);
  if (st != QLORA_OK) return st;
  if (top < 0 || top > kLpMaxTop || top > vocab) return QLORA_ERR_SHAPE;
  if (rows == 0) return QLORA_OK;
  if (!stats || (logprob && !token) || (top > 0 && (!top_logprob || !top_index))) return QLORA_ERR_NULL;
  if (!aligned8(token) || !aligned4(logprob) || !aligned4(stats) || !aligned4(entropy) || !aligned4(top_logprob) ||
      !aligned8(top_index))
    return QLORA_ERR_ALIGN;
  const int64_t segs = lp_parts(rows, vocab, dtype);
  const LpWs w = lp_layout(ws, rows, segs, top);
  if (segs > 1 && (!ws || ws_bytes < w.bytes)) return QLORA_ERR_WORKSPACE;   // (rows in one part need none)
  if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  LpArgs a{};
  a.x = logits;
  a.stride = stride;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.fp32 = dtype == QLORA_FP32;
  a.scale = scale;
  // The scale last is an instruction a logit less (4096 x 32000 of bf16: 43.6 us, first 45.8).  First where differences of logits could
  // overflow before they are scaled, or the scale with the factor of its exponent does.
  a.unit = scale >= 0x1p-64f && scale <= 0x1p64f ? scale : 1.0f;
  a.top = top;
  a.token = token;
  a.logprob = logprob;
  a.stats = stats;
  a.entropy = entropy;
  a.top_lp = top_logprob;
  a.top_index = top_index;
  a.part = w.part;
  a.cand = w.cand;
  a.segs = (int32_t)segs;
  QL_HIP(launch_logprob(a, stream));
  return QLORA_OK;
}

qlora_status qlora_token_logprob_bwd(const void* logits, int64_t stride, int64_t rows, int64_t vocab, int32_t dtype,
                                     const int64_t* token, float scale, const float* stats, const float* dlogprob,
                                     const float* entropy, const float* dentropy, void* dlogits, int64_t dlogits_stride,
                                     hipStream_t stream) {
  qlora_status st = check_logits(logits, stride, rows, vocab, dtype, scale, false);
  if (st != QLORA_OK) return st;
  if ((st = check_logits(dlogits, dlogits_stride, rows, vocab, dtype, scale, true)) != QLORA_OK) return st;
  if (!in_place_ok(dlogits, dlogits_stride, logits, stride, rows)) return QLORA_ERR_SHAPE;
  if (rows == 0) return QLORA_OK;
  if (!stats || (dlogprob && !token) || (dentropy && !entropy) || (!dlogprob && !dentropy)) return QLORA_ERR_NULL;
  if (!aligned8(token) || !aligned4(stats) || !aligned4(dlogprob) || !aligned4(entropy) || !aligned4(dentropy))
    return QLORA_ERR_ALIGN;
  LpBwdArgs a{};
  a.x = logits;
  a.dx = dlogits;
  a.stride = stride;
  a.dx_stride = dlogits_stride;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.fp32 = dtype == QLORA_FP32;
  a.scale = scale;
  a.token = dlogprob ? token : nullptr;
  a.stats = stats;
  a.dlp = dlogprob;
  a.entropy = entropy;
  a.dent = dentropy;
  QL_HIP(launch_logprob_bwd(a, stream));
  return QLORA_OK;
}

}  // extern "C"
