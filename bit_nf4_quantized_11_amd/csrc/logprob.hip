// Log probabilities of given tokens, the distribution's entropy and its most likely alternatives; and the gradient.
//
// With x a row's logits times `scale`, m the largest, d = x - m, z = sum e^d:
//   log p_v = d_v - ln z,   entropy = -sum p ln p = ln z - (sum e^d d) / z
//   dx_v = scale (dlp (1[v = token] - p_v) - dent p_v (ln p_v + entropy))
//
// Bound by HBM: the forward reads the logits once (a wave holds its share of a part of a row in registers, so its sums are
// taken from its own maximum without a second look at memory), the backward reads and writes them once.
// Rows of several parts, and few long ones, are joined by a second kernel.  4096 x 32000 logits of bf16: forward 41 us = 6.4
// TB/s and 4.7 for the join, backward 97 us = 5.4 TB/s; of fp32 forward 87 us = 6.0 TB/s.  With the waves of a row waiting for one
// maximum it was 65 us.  8 x 32000: 5.3 us, 8.2 to 8.7 with 20 alternatives (latency).
//
// The k largest: a wave's k-th largest of its lanes' maxima is a bound that at least k of its elements reach; so is the least of
// all waves' ceil(k / waves)-th largest, which leaves fewer where the large ones are spread (k = 20 over 8 waves: about 46 of a
// row of 32000, with the first kind alone 130; the higher of the two is taken).  What remains is listed in LDS as 64-bit numbers
// (order of the value, then the lower index) and each counts those above it: its rank, whatever the order of the list.
// Where a mask leaves no such bound, all above -infinity are, and of the others the first (8 x 32000, 3 of them allowed: 8 us).
// With more candidates than the list holds (equal logits) the bound is taken in full and only the first k of
// each wave's elements that equal it are listed; rows with still more, or with a NaN, take k rounds of a maximum instead.
#include <cfloat>

#include "kernels.h"
#include "rows.h"

namespace qlora {

namespace {

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

// Elements col .. col + E - 1 of a row of n, one by one; -infinity behind its end.
template <bool F32>
__device__ __forceinline__ uint4 load_edge(const typename Elem<F32>::T* row, int col, int n) {
  typedef Elem<F32> X;
  float f[X::E];
#pragma unroll
  for (int j = 0; j < X::E; ++j) f[j] = col + j < n ? X::value(row + col + j) : -INFINITY;
  return X::pack(f);
}
template <bool F32>
__device__ __forceinline__ uint4 load_piece(const typename Elem<F32>::T* row, int col, int n) {
  if (col + Elem<F32>::E <= n) return load_any(row + col);
  return load_edge<F32>(row, col, n);
}
// C such pieces, `step` elements apart.  All are loaded first, without a branch between the loads (behind the row's end,
// its last piece); then those at the end again.
template <bool F32, int C>
__device__ __forceinline__ void load_pieces(uint4 (&v)[C], const typename Elem<F32>::T* row, int col, int step, int n) {
  constexpr int E = Elem<F32>::E;
  if (n >= E) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = load_any(row + min(col + i * step, n - E));
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (col + i * step + E > n) v[i] = load_edge<F32>(row, col + i * step, n);
}

// Larger numbers for larger values; NaN above all (+infinity is 0xFF800000), both zeros the same.  Never 0, nor all ones, which
// with the inverted index 0 would make an entry that none is below.
constexpr uint32_t kNanOrder = 0xFFFFFFFEu;
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return kNanOrder;
  const uint32_t b = x == 0.0f ? 0u : __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 entry_of(float x, int col) { return (u64)order_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)col); }
__device__ __forceinline__ float value_of(u64 e) {
  const uint32_t k = (uint32_t)(e >> 32);
  if (k == kNanOrder) return NAN;
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ int col_of(u64 e) { return (int)(0xFFFFFFFFu - (uint32_t)e); }

// The given token of a row and its logit, asked for early.
template <bool F32>
struct Given {
  int64_t token;
  float x;
  __device__ Given(const LpArgs& a, int64_t row, int64_t token) : token(token), x(0.0f) {
    typedef Elem<F32> X;
    if (token >= 0 && token < a.vocab) x = X::value(static_cast<const typename X::T*>(a.x) + row * a.stride + token);
  }
};

// What the forward leaves of a row, from its whole sums (of `unit` times these).
struct RowEnd {
  float m, logz;
  bool empty;   // no logit above -infinity
};
template <bool F32>
__device__ __forceinline__ RowEnd finish_row(const LpArgs& a, int64_t row, const Given<F32>& g, float top, float z, float s,
                                             bool write) {
  RowEnd r;
  r.m = top * a.unit;
  // (a finite logit whose product with the scale is infinite counts as that infinity; a NaN, which the maximum passes over, stays in z)
  if (r.m == -INFINITY && z == z) z = 0.0f;
  if (r.m == INFINITY) z = NAN;
  r.empty = z == 0.0f;
  r.logz = logf(z);
  if (!write) return r;
  a.stats[2 * row] = r.m;
  a.stats[2 * row + 1] = z;
  if (a.entropy) a.entropy[row] = r.empty ? 0.0f : r.logz - s * (a.unit / z);
  if (a.logprob)
    a.logprob[row] = g.token >= a.vocab ? NAN : g.token < 0 ? 0.0f : r.empty ? -INFINITY : (g.x * a.scale - r.m) - r.logz;
  return r;
}
__device__ __forceinline__ void write_top(const LpArgs& a, int64_t row, int rank, u64 e, const RowEnd& r) {
  a.top_lp[row * a.top + rank] = r.empty ? -INFINITY : (value_of(e) * a.scale - r.m) - r.logz;
  a.top_index[row * a.top + rank] = col_of(e);
}

// The k-th largest of a wave's lanes' orders, or a lower bound of it with the lower half zero.
template <int LOW>
__device__ __forceinline__ uint32_t kth_largest(uint32_t mine, int k) {
  uint32_t b = 0;
#pragma unroll
  for (int bit = 31; bit >= LOW; --bit) {
    const uint32_t next = b | 1u << bit;
    if (__popcll(__ballot(mine >= next)) >= k) b = next;
  }
  return b;
}

// Both of two such numbers at once: their rounds' chains of scalar instructions run beside each other.
template <int LOW>
__device__ __forceinline__ void kth_largest(uint32_t mine, int k0, int k1, uint32_t& b0, uint32_t& b1) {
  b0 = b1 = 0;
#pragma unroll
  for (int bit = 31; bit >= LOW; --bit) {
    const uint32_t next0 = b0 | 1u << bit, next1 = b1 | 1u << bit;
    if (__popcll(__ballot(mine >= next0)) >= k0) b0 = next0;
    if (__popcll(__ballot(mine >= next1)) >= k1) b1 = next1;
  }
}

// Where this lane's `mine` places begin in a list that all waves share.
__device__ __forceinline__ int places(int mine, int* count) {
  if (!__ballot(mine > 0)) return 0;
  const int incl = wave_prefix(mine);
  int base = 0;
  if ((threadIdx.x & 63) == 63) base = atomicAdd(count, incl);
  return __builtin_amdgcn_readlane(base, 63) + incl - mine;
}

// Each of the n entries of an LDS list with its rank, `out(rank, entry)`, for ranks below k; T threads, all of which call.
// 8 neighbouring lanes share the comparisons of an entry, 8 of which are read at a time: the list ends in zeros
// (kPad places behind n).
constexpr int kLanes = 8, kPad = 8 * kLanes;
template <int T, class F>
__device__ __forceinline__ void rank_list(u64* list, int n, int k, F out) {
  if (threadIdx.x < kPad) list[n + threadIdx.x] = 0;
  __syncthreads();
  const int sub = threadIdx.x & (kLanes - 1);
  for (int i0 = 0; i0 < n; i0 += T / kLanes) {
    const int i = i0 + threadIdx.x / kLanes;
    const u64 e = list[min(i, n - 1)];
    int rank = 0;
    for (int j = sub; j < n; j += kPad) {
      u64 o[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) o[u] = list[j + u * kLanes];
#pragma unroll
      for (int u = 0; u < 8; ++u) rank += o[u] > e;
    }
    // the lanes' sum: neighbours, pairs, and the other half of 8
    rank += (int)dpp_or<0xB1, 0xF>(0u, (uint32_t)rank);
    rank += (int)dpp_or<0x4E, 0xF>(0u, (uint32_t)rank);
    rank += (int)dpp_or<0x141, 0xF>(0u, (uint32_t)rank);
    if (i < n && sub == 0 && rank < k) out(rank, e);
  }
}

// One part of one row.  C: 16-byte loads of each of the NT threads.  Every wave sums from its own maximum, so that none waits for
// another's loads; the waves' sums are joined at the end.
template <bool F32, int C, bool TOP, int NT>
__global__ __launch_bounds__(NT) void k_token_logprob(LpArgs a) {
  typedef Elem<F32> X;
  constexpr int E = X::E, NW = NT / 64;
  __shared__ float red[3][NW];
  __shared__ u64 list[TOP ? CAP + kPad : 1];
  __shared__ uint32_t bound[2][NW];
  __shared__ int count;
  const bool whole = a.segs == 1;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t row = blockIdx.x / (unsigned)a.segs;
  const int seg = (int)(blockIdx.x - row * a.segs);
  const int col0 = (seg * C * NT + t) * E;
  const int64_t token = whole && a.logprob ? a.token[row] : -1;
  const auto* const x = static_cast<const typename X::T*>(a.x) + row * a.stride;
  uint4 v[C];
  load_pieces<F32, C>(v, x, col0, NT * E, a.vocab);
  const Given<F32> given(a, row, token);
  float top = -INFINITY;   // (NaN are passed over)
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float f[E];
    X::unpack(v[i], f);
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, f[j]);
  }
  const bool far = a.unit != a.scale;
  const float mine_m = wave_max(top) * (far ? a.scale : 1.0f);
  const float from = mine_m == -INFINITY ? 0.0f : mine_m, by = a.unit * kLog2e;
  float z = 0.0f, s = 0.0f;
  const auto sums = [&](float first) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float f[E];
      X::unpack(v[i], f);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        // (the difference before the scale: equal ones give 0)
        const float d = f[j] * first - from;
        const float e = __builtin_amdgcn_exp2f(d * by);
        z += e;
        s = __builtin_fmaf(e, fmaxf(d, -1e30f), s);   // (nothing of a logit of -infinity)
      }
    }
  };
  if (far) sums(a.scale);
  else sums(1.0f);
  z = wave_sum(z);
  s = wave_sum(s);
  if (lane == 0) red[0][wave] = mine_m, red[1][wave] = z, red[2][wave] = s;
  bool nothing = false;
  if (TOP) {
    // the wave's k-th largest lane maximum, and its share of k, by the upper halves of their orders (lower bounds are as good)
    uint32_t own, share;
    kth_largest<16>(order_of(top), a.top, (a.top + NW - 1) / NW, own, share);
    if (lane == 0) bound[0][wave] = own, bound[1][wave] = share;
    if (t == 0) count = 0;
    __syncthreads();
    uint32_t b = bound[0][0], all = bound[1][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) b = max(b, bound[0][w]), all = min(all, bound[1][w]);
    b = max(b, all);
    // (where the bound is -infinity, all above that)
    nothing = b <= 0x007FFFFFu;
    const float least = nothing ? -FLT_MAX : value_of((u64)b << 32);
    // A bit for each of the thread's elements, the first one highest; those that are listed are read again (the row is in the caches;
    // a branch on each in its register is 5 KB of instructions to fetch: 8 x 32000 9.9 us against 8.0).
    static_assert(C * E <= 64, "bits of a thread's elements");
    constexpr int B = C * E < 32 ? C * E : 32;
    uint32_t hit[C * E / B] = {};
    if (top >= least) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float f[E];
        X::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          uint32_t& h = hit[(i * E + j) / B];
          h = h + h + (f[j] >= least ? 1u : 0u);
        }
      }
    }
    int above = 0;
#pragma unroll
    for (int k = 0; k < C * E / B; ++k) above += __popc(hit[k]);
    int at = places(above, &count);
    if (at + above <= CAP) {
#pragma unroll
      for (int k = 0; k < C * E / B; ++k)
        for (uint32_t h = hit[k]; h; ++at) {
          const int b = 31 - __clz(h), e = k * B + B - 1 - b, col = col0 + e / E * (NT * E) + e % E;
          h ^= 1u << b;
          list[at] = entry_of(X::value(x + col), col);
        }
    }
  }
  __syncthreads();
  float m = red[0][0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = fmaxf(m, red[0][w]);
  z = s = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float mw = red[0][w], d = mw == -INFINITY ? 0.0f : mw - m, e = __builtin_amdgcn_exp2f(d * by);
    z += e * red[1][w];
    s += e * __builtin_fmaf(red[1][w], fmaxf(d, -1e30f), red[2][w]);
  }
  RowEnd end{};
  if (whole) {
    end = finish_row<F32>(a, row, given, m, z, s, t == 0);
  } else if (t == 0) {
    a.part[row * a.segs + seg] = LpPart{m, z, s, 0};
  }
  if (!TOP) return;
  u64* const cand = whole ? nullptr : a.cand + (row * a.segs + seg) * a.top;
  const auto put = [&](int rank, u64 e) {
    if (whole) write_top(a, row, rank, e, end);
    else cand[rank] = e;
  };
  int n = count;
  if (n > CAP && z == z) {
    // Many equal logits (or nearly so): the bound in full, all elements above it, and of those that equal it the first k
    // of each wave.
    const uint32_t mine = order_of(top), b = kth_largest<0>(mine, a.top);
    __syncthreads();
    if (lane == 0) bound[0][wave] = b;
    if (t == 0) count = 0;
    __syncthreads();
    uint32_t order = bound[0][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) order = max(order, bound[0][w]);
    const float least = value_of((u64)order << 32);
    // (read again, a few loads at a time: this path is to cost the common one no registers)
    const bool larger = __ballot(top > least) != 0;   // (in this wave)
    constexpr int U = C < 4 ? C : 4;
    int have = 0;   // equal ones of this wave
#pragma unroll 1
    for (int i0 = 0; i0 < C && (larger || have < a.top); i0 += U) {
      uint4 again[U];
#pragma unroll
      for (int u = 0; u < U; ++u) again[u] = load_piece<F32>(x, col0 + (i0 + u) * NT * E, a.vocab);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[E];
        X::unpack(again[u], f);
        const int col = col0 + (i0 + u) * NT * E;
        uint32_t above = 0, equal = 0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          above |= (f[j] > least ? 1u : 0u) << j;
          equal |= (f[j] == least && col + j < a.vocab ? 1u : 0u) << j;
        }
        if (!__ballot((above | (have < a.top ? equal : 0u)) != 0)) continue;
        const int ties = __popc(equal), incl = wave_prefix(ties), before = have + incl - ties;
        int mine = min(max(a.top - before, 0), ties);
        int to = places(__popc(above) + mine, &count);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const bool tie = equal >> j & 1 && mine > 0;
          mine -= tie;
          if ((above >> j & 1 || tie) && to < CAP) list[to++] = entry_of(f[j], col + j);
        }
        have += __builtin_amdgcn_readlane(incl, 63);
      }
    }
    __syncthreads();
    n = count;
  }
  if (nothing && n < a.top) {
    // Masked rows: with fewer than k elements above -infinity there are enough of those that equal it among the part's first k.
    __syncthreads();
    const int col = seg * C * NT * E + t;
    if (t < a.top && col < a.vocab && X::value(x + col) == -INFINITY) list[atomicAdd(&count, 1)] = entry_of(-INFINITY, col);
    __syncthreads();
    n = count;
  }
  if (n <= CAP && z == z) {
    rank_list<NT>(list, n, a.top, put);
    if (!whole)
      for (int i = n + t; i < a.top; i += NT) cand[i] = 0;
    return;
  }
  // k rounds of a maximum
  u64 last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    u64 best = 0;
#pragma unroll 1
    for (int i = 0; i < C; ++i) {
      float f[E];
      X::unpack(load_piece<F32>(x, col0 + i * NT * E, a.vocab), f);
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
    if (t == 0) put(k, best);   // 0 where the part has no more (a whole row has k elements); then nothing is below it
    last = best;
  }
}

// The parts of a row joined by a wave, a part to a lane.  The parts' candidates are in descending order each, so the
// largest of all is the largest of their first ones; parts ascend with the tokens, so of equal ones it is the first
// lane's.  JW waves to a workgroup, which share nothing.
constexpr int JW = 4;
template <bool F32, bool TOP>
__global__ __launch_bounds__(64 * JW) void k_logprob_join(LpArgs a) {
  extern __shared__ u64 lists[];   // [JW][segs][top]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * JW + wave;
  if (row >= a.rows) return;
  const Given<F32> given(a, row, a.logprob ? a.token[row] : -1);
  float m = -INFINITY, z = 0.0f, s = 0.0f;
  if (lane < a.segs) {
    const LpPart p = a.part[row * a.segs + lane];
    m = p.m, z = p.z, s = p.s;
  }
  const int n = a.segs * a.top;
  u64* const list = lists + wave * n;
  if (TOP) {
    constexpr int U = 8;   // loads in flight
    for (int i0 = lane; i0 < n; i0 += 64 * U) {
      u64 c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = a.cand[row * n + min(i0 + 64 * u, n - 1)];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + 64 * u < n) list[i0 + 64 * u] = c[u];
    }
  }
  const float mm = wave_max(m);
  const float d = m == -INFINITY ? 0.0f : m - mm;
  const float e = __builtin_amdgcn_exp2f(d * (a.unit * kLog2e));
  s = e * __builtin_fmaf(z, fmaxf(d, -1e30f), s);
  z = wave_sum(e * z);
  s = wave_sum(s);
  const RowEnd end = finish_row<F32>(a, row, given, mm, z, s, lane == 0);
  if (!TOP) return;
  // (written and read by one wave, whose LDS accesses keep their order) a lane's first candidate, and its next one loaded ahead; 0 where there are none
  const int stop = lane < a.segs ? (lane + 1) * a.top : 0;
  int at = lane * a.top;
  u64 head = at < stop ? list[at] : 0, next = at + 1 < stop ? list[at + 1] : 0, kept = 0;
  for (int k = 0; k < a.top; ++k) {
    const uint32_t mine = (uint32_t)(head >> 32), best = wave_max(mine);
    const int from = __ffsll(__ballot(mine == best)) - 1;
    const uint32_t low = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)head, from);
    if (lane == k) kept = (u64)best << 32 | low;
    if (lane == from) {
      ++at;
      head = next;
      next = at + 1 < stop ? list[at + 1] : 0;
    }
  }
  if (lane < a.top) write_top(a, row, lane, kept, end);
}

// Gradient: BC 16-byte pieces of a row to a thread, 4 B (bf16) or 8 B of traffic an element.
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
  load_pieces<F32, BC>(v, x, col0, BT * E, a.vocab);
  const int64_t token = a.token ? a.token[row] : -1;
  const float m = a.stats[2 * row], z = a.stats[2 * row + 1];
  const float dlp = token >= a.vocab ? NAN : token >= 0 && a.dlp ? a.dlp[row] : 0.0f;
  const float dent = a.dent ? a.dent[row] : 0.0f;
  // rows whose gradient is 0 whatever their logits (padding may hold NaN) and the gradients are: without a token, and empty ones
  const bool none = (token < 0 && !a.dent) || (z == 0.0f && token < a.vocab);
  const float rz = 1.0f / z, logz = logf(z);
  const float rest = a.dent ? a.entropy[row] - logz : 0.0f;   // ln p + entropy = d + rest
#pragma unroll
  for (int i = 0; i < BC; ++i) {
    const int col = col0 + i * BT * E;
    if (col >= a.vocab) break;
    float f[E] = {};
    if (!none) {
      X::unpack(v[i], f);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float d = f[j] * a.scale - m;
        const float p = __builtin_amdgcn_exp2f(d * kLog2e) * rz;
        // (p first: a gradient of the entropy times ln p alone can be infinite where p is 0.  Nothing of a logit of -infinity)
        float g = -__builtin_fmaf(dent, p * (fmaxf(d, -1e30f) + rest), p * dlp);
        if (col + j == token) g += dlp;
        f[j] = g * a.scale;
      }
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

// Threads of a part and 16-byte loads of each.
struct Part {
  int t, c;
};
// By what the rows alone say, not by the outputs that a call asks for, so that the sums do not depend on these.
//   A row of up to 32 K logits is one part, held by as few threads as its length allows (1000 logits by a wave: 4096 rows 6 us, by
// 512 threads 12).
//   Of bf16 and 128 rows or more, parts have 16 K logits at most: 4096 rows of 32000 take 41 + 5 us with the join (62 + 9 with 20
// alternatives), whole ones 51 (fp32, as many: 87 whole, 87 + 5); 8 rows are faster whole (8 us with 20 alternatives).
//   Longer rows have parts of that size, and smaller ones while all rows together have fewer than 128.
Part part_for(int64_t rows, int64_t vocab, bool fp32) {
  const int64_t n = pieces(vocab, fp32);
  if (n <= 64) return {64, 1};
  if (n <= 256) return {64, 4};
  if (n <= 512) return {256, 2};
  if (n <= 1024) return {256, 4};
  if (n <= 2048) return {256, 8};
  const auto parts = [&](int64_t per) { return (n + per - 1) / per; };
  const Part most = fp32 ? Part{512, 16} : Part{512, 8};
  int64_t per = (int64_t)most.t * most.c;
  if (!fp32 && rows >= 128 && parts(2048) <= kLpMaxSegs) return {256, 8};
  if (n <= 4096) return {512, 8};
  if (per >= n) return most;
  while (per > 512 && rows * parts(per) < 128 && parts(per / 2) <= kLpMaxSegs) per /= 2;
  return per == 512 ? Part{512, 1} : per == 1024 ? Part{512, 2} : per == 2048 ? Part{512, 4} : per == 4096 ? Part{512, 8} : most;
}

template <bool F32, bool TOP>
hipError_t launch_parts(const LpArgs& a, Part p, hipStream_t s) {
  const int64_t items = a.rows * a.segs;
  const dim3 g((unsigned)items), b(p.t);
  {
    ProfScope ps("k_token_logprob", s);
#define LP_LAUNCH(T, C) hipLaunchKernelGGL((k_token_logprob<F32, C, TOP, T>), g, b, 0, s, a)
    if (p.t == 64 && p.c == 1) LP_LAUNCH(64, 1);
    else if (p.t == 64) LP_LAUNCH(64, 4);
    else if (p.t == 256 && p.c == 2) LP_LAUNCH(256, 2);
    else if (p.t == 256 && p.c == 4) LP_LAUNCH(256, 4);
    else if (p.t == 256) LP_LAUNCH(256, 8);
    else if (p.c == 1) LP_LAUNCH(512, 1);
    else if (p.c == 2) LP_LAUNCH(512, 2);
    else if (p.c == 4) LP_LAUNCH(512, 4);
    else if (p.c == 8) LP_LAUNCH(512, 8);
    else if constexpr (F32) LP_LAUNCH(512, 16);   // (of fp32 alone)
#undef LP_LAUNCH
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.segs == 1) return e;
  }
  ProfScope ps("k_logprob_join", s);
  const size_t lds = (size_t)JW * a.segs * a.top * sizeof(u64);   // at most 32 KB
  hipLaunchKernelGGL((k_logprob_join<F32, TOP>), dim3((unsigned)((a.rows + JW - 1) / JW)), dim3(64 * JW), lds, s, a);
  return hipGetLastError();
}

}  // namespace

int lp_segments(int64_t rows, int64_t vocab, bool fp32) {
  const Part p = part_for(rows, vocab, fp32);
  const int64_t per = (int64_t)p.t * p.c;
  return (int)((pieces(vocab, fp32) + per - 1) / per);
}

hipError_t launch_logprob(const LpArgs& a, hipStream_t s) {
  const Part p = part_for(a.rows, a.vocab, a.fp32);
  if (a.fp32) return a.top ? launch_parts<true, true>(a, p, s) : launch_parts<true, false>(a, p, s);
  return a.top ? launch_parts<false, true>(a, p, s) : launch_parts<false, false>(a, p, s);
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
