// Log probabilities of given tokens, the distribution's entropy and its most likely alternatives; and the gradient.
//
// With x a row's logits times `scale`, m the largest, d = x - m, z = sum e^d:
//   log p_v = d_v - ln z,   entropy = -sum p ln p = ln z - (sum e^d d) / z
//   dx_v = scale (dlp (1[v = token] - p_v) - dent p_v (ln p_v + entropy))
//
// Bound by HBM: the forward reads the logits once (a workgroup holds its part of a row in registers, so the sums are
// taken from the row's own maximum without a second look at memory), the backward reads and writes them once.
// Long rows, and few ones, are cut into parts that a second kernel joins.
//
// The k largest: a wave's k-th largest of its lanes' maxima is a bound that at least k of its elements reach; with the
// largest bound of all waves few elements remain (about 1.5 k a wave).  They are listed in LDS as 64-bit numbers
// (order of the value, then the lower index) and each counts those above it: its rank, whatever the order of the list.
// Rows with more candidates than the list holds (many equal logits) or with a NaN take k rounds of a maximum instead.
#include "kernels.h"
#include "rows.h"

namespace qlora {

namespace {

constexpr int NT = 512;       // threads of a part
constexpr int NW = NT / 64;
constexpr int CAP = 1024;     // candidates that the list holds
constexpr float kLog2e = 1.4426950408889634f;

typedef unsigned long long u64;

// E elements of a row in 16 bytes
template <bool F32>
struct Elem;
template <>
struct Elem<true> {
  typedef float T;
  static constexpr int E = 4;
  __device__ static void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static float value(const float* p) { return *p; }
  __device__ static void store(float* p, float v) { *p = v; }
};
template <>
struct Elem<false> {
  typedef uint16_t T;
  static constexpr int E = 8;
  __device__ static void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
  __device__ static float value(const uint16_t* p) { return bf16_to_f32(*p); }
  __device__ static void store(uint16_t* p, float v) { *p = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
};

// 16 bytes at any element's address (rows of an odd length start anywhere)
__device__ __forceinline__ uint4 load_any(const void* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store_any(void* p, const uint4& v) { __builtin_memcpy(p, &v, 16); }

// Elements col .. col + E - 1 of a row of n; -infinity behind its end.
template <bool F32>
__device__ __forceinline__ uint4 load_chunk(const typename Elem<F32>::T* row, int col, int n) {
  typedef Elem<F32> X;
  if (col + X::E <= n) return load_any(row + col);
  float f[X::E];
#pragma unroll
  for (int j = 0; j < X::E; ++j) f[j] = col + j < n ? X::value(row + col + j) : -INFINITY;
  return X::pack(f);
}

// Larger numbers for larger values; NaN above all, both zeros the same.  Never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = x == 0.0f ? 0u : __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 entry_of(float x, int col) { return (u64)order_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)col); }
__device__ __forceinline__ float value_of(u64 e) {
  const uint32_t k = (uint32_t)(e >> 32);
  if (k == 0xFFFFFFFFu) return NAN;
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ int col_of(u64 e) { return (int)(0xFFFFFFFFu - (uint32_t)e); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// What the forward leaves of a row, from its whole sums.
struct RowEnd {
  float m, logz;
  bool empty;   // no logit above -infinity
};
template <bool F32>
__device__ __forceinline__ RowEnd finish_row(const LpArgs& a, int64_t row, float m, float z, float s, bool write) {
  typedef Elem<F32> X;
  RowEnd r;
  r.m = m;
  r.empty = z == 0.0f;
  r.logz = logf(z);
  if (!write) return r;
  a.stats[2 * row] = m;
  a.stats[2 * row + 1] = z;
  if (a.entropy) a.entropy[row] = r.empty ? 0.0f : r.logz - s / z;
  if (a.logprob) {
    const int64_t t = a.token[row];
    float lp = 0.0f;
    if (t >= a.vocab) {
      lp = NAN;
    } else if (t >= 0) {
      const float x = X::value(static_cast<const typename X::T*>(a.x) + row * a.stride + t) * a.scale;
      lp = r.empty ? -INFINITY : (x - m) - r.logz;
    }
    a.logprob[row] = lp;
  }
  return r;
}
__device__ __forceinline__ void write_top(const LpArgs& a, int64_t row, int rank, u64 e, const RowEnd& r) {
  a.top_lp[row * a.top + rank] = r.empty ? -INFINITY : (value_of(e) * a.scale - r.m) - r.logz;
  a.top_index[row * a.top + rank] = col_of(e);
}

// One part of one row.  C: 16-byte loads of a thread.
template <bool F32, int C, bool TOP>
__global__ __launch_bounds__(NT) void k_token_logprob(LpArgs a) {
  typedef Elem<F32> X;
  constexpr int E = X::E;
  __shared__ float red[3][NW];
  __shared__ u64 list[TOP ? CAP : 1];
  __shared__ uint32_t bound[NW];
  __shared__ int count;
  const int64_t row = blockIdx.x / (unsigned)a.segs;
  const int seg = (int)(blockIdx.x - row * a.segs);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const auto* const x = static_cast<const typename X::T*>(a.x) + row * a.stride;
  const int col0 = (seg * C * NT + t) * E;
  uint4 v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = load_chunk<F32>(x, col0 + i * NT * E, a.vocab);
  float top = -INFINITY;   // (NaN are passed over)
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float f[E];
    X::unpack(v[i], f);
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, f[j]);
  }
  {
    const float w = wave_max(top);
    if (lane == 0) red[0][wave] = w;
  }
  if (TOP) {
    // the wave's k-th largest lane maximum, by the upper half of its order (a lower bound is as good)
    const uint32_t mine = order_of(top) >> 16;
    uint32_t b = 0;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t next = b | 1u << bit;
      if (__popcll(__ballot(mine >= next)) >= a.top) b = next;
    }
    if (lane == 0) bound[wave] = b << 16;
    if (t == 0) count = 0;
  }
  __syncthreads();
  float m = red[0][0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = fmaxf(m, red[0][w]);
  m *= a.scale;
  const float from = m == -INFINITY ? 0.0f : m;
  float z = 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float f[E];
    X::unpack(v[i], f);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = f[j] * a.scale - from;
      const float e = __builtin_amdgcn_exp2f(d * kLog2e);
      z += e;
      s = __builtin_fmaf(e, fmaxf(d, -1e30f), s);   // (nothing of a logit of -infinity)
    }
  }
  z = wave_sum(z);
  s = wave_sum(s);
  if (lane == 0) red[1][wave] = z, red[2][wave] = s;
  if (TOP) {
    uint32_t b = bound[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) b = max(b, bound[w]);
    const float least = b <= 0x007FFFFFu ? -INFINITY : value_of((u64)b << 32);
    if (top >= least) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float f[E];
        X::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const int col = col0 + i * NT * E + j;
          if (f[j] >= least && col < a.vocab) {
            const int n = atomicAdd(&count, 1);
            if (n < CAP) list[n] = entry_of(f[j], col);
          }
        }
      }
    }
  }
  __syncthreads();
  z = red[1][0], s = red[2][0];
#pragma unroll
  for (int w = 1; w < NW; ++w) z += red[1][w], s += red[2][w];
  const bool whole = a.segs == 1;
  RowEnd end{};
  if (whole) {
    end = finish_row<F32>(a, row, m, z, s, t == 0);
  } else if (t == 0) {
    a.part[row * a.segs + seg] = LpPart{m, z, s, 0};
  }
  if (!TOP) return;
  u64* const cand = whole ? nullptr : a.cand + (row * a.segs + seg) * a.top;
  const int n = count;
  if (n <= CAP && z == z) {
    for (int i = t; i < n; i += NT) {
      const u64 e = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += list[j] > e;
      if (rank >= a.top) continue;
      if (whole) write_top(a, row, rank, e, end);
      else cand[rank] = e;
    }
    if (!whole)
      for (int i = n + t; i < a.top; i += NT) cand[i] = 0;
    return;
  }
  u64 last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    u64 best = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float f[E];
      X::unpack(v[i], f);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int col = col0 + i * NT * E + j;
        const u64 e = entry_of(f[j], col);
        if (e < last && e > best && col < a.vocab) best = e;
      }
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) {
      const u64 o = __shfl_xor(best, off, 64);
      best = o > best ? o : best;
    }
    __syncthreads();   // (the list, and the last round's, is done with)
    if (lane == 0) list[wave] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) best = list[w] > best ? list[w] : best;
    if (t == 0) {
      if (!whole) cand[k] = best;
      else write_top(a, row, k, best, end);   // (a whole row has k elements)
    }
    last = best;   // 0 where the part has no more: then nothing is below it
  }
}

// The parts of a row joined: one workgroup per row.
constexpr int JT = 256;
template <bool F32, bool TOP>
__global__ __launch_bounds__(JT) void k_logprob_join(LpArgs a) {
  __shared__ u64 list[TOP ? kLpMaxSegs * kLpMaxTop : 1];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63;
  // every wave joins the sums (a part to a lane)
  float m = -INFINITY, z = 0.0f, s = 0.0f;
  if (lane < a.segs) {
    const LpPart p = a.part[row * a.segs + lane];
    m = p.m, z = p.z, s = p.s;
  }
  const int n = a.segs * a.top;
  if (TOP)
    for (int i = t; i < n; i += JT) list[i] = a.cand[row * n + i];
  const float mm = wave_max(m);
  const float d = m == -INFINITY ? 0.0f : m - mm;
  const float e = __builtin_amdgcn_exp2f(d * kLog2e);
  s = e * __builtin_fmaf(z, d, s);
  z = e * z;
  z = wave_sum(z);
  s = wave_sum(s);
  const RowEnd end = finish_row<F32>(a, row, mm, z, s, t == 0);
  if (!TOP) return;
  __syncthreads();
  for (int i = t; i < n; i += JT) {
    const u64 x = list[i];
    if (x == 0) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > x;
    if (rank < a.top) write_top(a, row, rank, x, end);
  }
}

// Gradient: BC 16-byte pieces of a row to a thread.
constexpr int BT = 256, BC = 4;
template <bool F32>
__global__ __launch_bounds__(BT) void k_token_logprob_bwd(LpBwdArgs a, unsigned segs) {
  typedef Elem<F32> X;
  constexpr int E = X::E;
  const int64_t row = blockIdx.x / segs;
  const int seg = (int)(blockIdx.x - row * segs);
  const auto* const x = static_cast<const typename X::T*>(a.x) + row * a.stride;
  auto* const dx = static_cast<typename X::T*>(a.dx) + row * a.dx_stride;
  const int col0 = (seg * BC * BT + (int)threadIdx.x) * E;
  uint4 v[BC];
#pragma unroll
  for (int i = 0; i < BC; ++i) v[i] = load_chunk<F32>(x, min(col0 + i * BT * E, a.vocab), a.vocab);
  const int64_t token = a.token ? a.token[row] : -1;
  const float m = a.stats[2 * row], z = a.stats[2 * row + 1];
  const bool empty = z == 0.0f;
  const float dlp = token >= a.vocab ? NAN : token >= 0 && a.dlp ? a.dlp[row] : 0.0f;
  const float dent = a.dent ? a.dent[row] : 0.0f;
  const float rz = empty ? 0.0f : 1.0f / z, logz = empty ? 0.0f : logf(z);
  const float from = empty ? 0.0f : m;
  // -p (dlp + dent (ln p + entropy)) = -p (c + dent d),  c = dlp + dent (entropy - ln z)
  const float c = a.dent ? __builtin_fmaf(dent, a.entropy[row] - logz, dlp) : dlp;
#pragma unroll
  for (int i = 0; i < BC; ++i) {
    const int col = col0 + i * BT * E;
    if (col >= a.vocab) break;
    float f[E];
    X::unpack(v[i], f);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = f[j] * a.scale - from;
      const float p = __builtin_amdgcn_exp2f(d * kLog2e) * rz;
      float g = -p * __builtin_fmaf(dent, fmaxf(d, -1e30f), c);
      if (col + j == token && !empty) g += dlp;
      f[j] = g * a.scale;
    }
    if (col + E <= a.vocab) {
      store_any(dx + col, X::pack(f));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (col + j < a.vocab) X::store(dx + col + j, f[j]);
    }
  }
}

int64_t pieces(int64_t vocab, bool fp32) { return (vocab + (fp32 ? 3 : 7)) / (fp32 ? 4 : 8); }

// 16-byte loads of a thread: the fewest that hold a row in one part, or 32 K elements (64 registers of fp32); fewer where
// the rows alone would leave CUs without work.
int loads_for(int64_t rows, int64_t vocab, bool fp32) {
  const int64_t n = pieces(vocab, fp32);
  const int most = fp32 ? 16 : 8;
  int c = 1;
  while (c < most && (int64_t)c * NT < n) c *= 2;
  while (c > 1 && rows * ((n + c * NT - 1) / (c * NT)) < 128 && (n + c / 2 * NT - 1) / (c / 2 * NT) <= kLpMaxSegs) c /= 2;
  return c;
}

template <bool F32, bool TOP>
hipError_t launch_parts(const LpArgs& a, int c, hipStream_t s) {
  const dim3 g((unsigned)(a.rows * a.segs)), b(NT);
  {
    ProfScope ps("k_token_logprob", s);
    if (c == 1) hipLaunchKernelGGL((k_token_logprob<F32, 1, TOP>), g, b, 0, s, a);
    else if (c == 2) hipLaunchKernelGGL((k_token_logprob<F32, 2, TOP>), g, b, 0, s, a);
    else if (c == 4) hipLaunchKernelGGL((k_token_logprob<F32, 4, TOP>), g, b, 0, s, a);
    else if (c == 8 || !F32) hipLaunchKernelGGL((k_token_logprob<F32, 8, TOP>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_token_logprob<F32, F32 ? 16 : 8, TOP>), g, b, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.segs == 1) return e;
  }
  ProfScope ps("k_logprob_join", s);
  hipLaunchKernelGGL((k_logprob_join<F32, TOP>), dim3((unsigned)a.rows), dim3(JT), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int lp_segments(int64_t rows, int64_t vocab, bool fp32) {
  const int64_t per = (int64_t)loads_for(rows, vocab, fp32) * NT;
  return (int)((pieces(vocab, fp32) + per - 1) / per);
}

hipError_t launch_logprob(const LpArgs& a, hipStream_t s) {
  const int c = loads_for(a.rows, a.vocab, a.fp32);
  if (a.fp32) return a.top ? launch_parts<true, true>(a, c, s) : launch_parts<true, false>(a, c, s);
  return a.top ? launch_parts<false, true>(a, c, s) : launch_parts<false, false>(a, c, s);
}

hipError_t launch_logprob_bwd(const LpBwdArgs& a, hipStream_t s) {
  const int64_t segs = (pieces(a.vocab, a.fp32) + BC * BT - 1) / (BC * BT);
  const dim3 g((unsigned)(a.rows * segs)), b(BT);
  ProfScope ps("k_token_logprob_bwd", s);
  if (a.fp32) hipLaunchKernelGGL((k_token_logprob_bwd<true>), g, b, 0, s, a, (unsigned)segs);
  else hipLaunchKernelGGL((k_token_logprob_bwd<false>), g, b, 0, s, a, (unsigned)segs);
  return hipGetLastError();
}

}  // namespace qlora
