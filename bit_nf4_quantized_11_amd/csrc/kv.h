// Device views of the head tensors, the 4-bit key/value cache and the batch description
// (qlora_heads, qlora_kv_cache, qlora_kv_batch), and the internal launch interface of the kernels
// behind them.  Launchers validate nothing: kv_api.cpp has already.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "qlora.h"

namespace qlora {

// bf16 [rows][heads][head_dim]
struct Heads {
  uint16_t* data;
  int64_t rs, hs;   // row and head strides in elements
  int32_t n;        // heads
};

struct KvView {
  uint8_t* kc;
  uint16_t* ks;
  uint8_t* vc;
  uint16_t* vs;
  int64_t pages;
  int32_t heads;
  int32_t pshift;   // log2 of the page size
  int32_t cb;
};

struct BatchView {
  const int32_t* start;
  const int32_t* length;
  const int32_t* table;
  int32_t* fault;
  int64_t rows;
  int32_t batch;
  int32_t max_pages;
  int32_t max_len;   // max_pages << pshift
};

enum : int32_t { kFaultStart = 1, kFaultLength = 2, kFaultPage = 4 };
constexpr uint32_t kBf16NaN = 0x7FC0u;

#ifdef __HIPCC__
__device__ __forceinline__ void raise_fault(const BatchView& b, int bit) {
  if (b.fault) atomicOr(b.fault, bit);
}

// Dword position of dword e (elements 8e..8e+7) in a key row of D elements: e = 4k + g of its
// section of 32 n elements sits at n g + k.
template <int D>
__device__ __forceinline__ int key_dword(int e) {
  constexpr int N = D == 64 ? 2 : 4;
  const int r = e & (4 * N - 1);
  return (e & ~(4 * N - 1)) + (r & 3) * N + (r >> 2);
}

// the larger of a lane's value and that of the lane that the DPP control names
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
#endif

// ---- head norms and rotation (qk_rope.hip) --------------------------------------------------
struct QkArgs {
  Heads q, k, qo, ko;             // inputs and outputs (backward: the gradients of the outputs and of the inputs)
  Heads xq, xk;                   // backward: the forward's inputs
  const uint16_t* wq;
  const uint16_t* wk;
  const int64_t* pos;
  const float* freq;
  int64_t rows;
  float eps;
  int32_t rot;
  int32_t slices;                 // wave items per row
  float* part;                    // backward: weight gradient partials [workgroup][2][D]
};
hipError_t launch_qk(const QkArgs& a, int D, bool interleaved, hipStream_t s);
// partial sums of each weight gradient (workgroups of the backward) in a call with at most these rows: grows with them, as
// the workgroups do not (fewer rows can be cut into more slices)
int qk_bwd_partials(int64_t rows, int32_t q_heads, int32_t k_heads, int D);
hipError_t launch_qk_bwd(const QkArgs& a, int D, bool interleaved, float* dwq, float* dwk, hipStream_t s);

// ---- cache write and read (kv_cache.hip) ------------------------------------------------------
hipError_t launch_kv_write(const Heads& k, const Heads& v, const KvView& c, const BatchView& b, int D, int block,
                           hipStream_t s);
hipError_t launch_kv_read(const Heads& k, const Heads& v, const KvView& c, const BatchView& b, int D, int block,
                          hipStream_t s);

// ---- attention over the cache (kv_attn.hip) -----------------------------------------------------
struct AttnArgs {
  Heads q, o;
  float* lse;                     // [rows][q.n] or NULL
  KvView c;
  BatchView b;
  int32_t group;                  // query heads per cache head, and n / group = n group_mul >> group_shift
  uint32_t group_mul;
  int32_t group_shift;
  float scale;
  int32_t causal, window;
  int32_t ushift;                 // log2 of the unit of work in steps of every wave
  int32_t few;                    // rows per cache head up to which a sequence is the first kernel's
  float* part;                    // partial sums of ranges that end inside an item
  int32_t* meta;                  // [workgroups][kMetaInts] (second kernel: [1 + tiles])
};
// Sizes of a launch, from what the host knows.
struct AttnPlan {
  int tile;                       // query rows per tile (row = token and query head of one cache head)
  int ushift, few;                // as in AttnArgs; few = INT32_MAX: the first kernel alone, 0: the second alone
  int64_t wgs;                    // workgroups of the first kernel's ranges
  int64_t many_wgs;               // workgroups of the second kernel, its tiles x cache heads at most
  int64_t many_split;             // how many of these it may cut into parts: 0 (no join), or up to kSplitWgs / 2
  int split_tokens;               // tokens of a part at least; 0: none is cut
  bool sparse;                    // a quarter of its tiles' rows or more are empty
  size_t part_floats, meta_ints;  // workspace: the most that a call with at most these rows, sequences and tokens uses
};
AttnPlan attn_plan(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t batch, int64_t max_len, int D);
hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s);
// sequences with many rows (kv_attn_many.hip)
struct CodePlanes;
CodePlanes code_planes(int codebook);
hipError_t launch_kv_attn_many(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s);

}  // namespace qlora
