// What the two attention kernels share: decoding of 4-bit codes to fp16, a batch's sequences, the tiles of their rows, and
// the sum of a tile's parts.
#pragma once

#include "kernels.h"
#include "kv.h"

namespace qlora {

constexpr int kMetaInts = 8;   // per part or range in the workspace: what the join has to know of its tile
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// The 16 levels times c in fp16, in the two forms that codes are decoded by.
//   pair: a byte of codes is looked up in a table of 256 pairs in LDS (one dword: its low nibble's level, its
//     high nibble's): 1 VALU and 1 LDS instruction for 2 elements.
//   planes: byte permutes.  v_perm_b32 picks 4 bytes out of 8 by selectors 0..7; its selectors 8..15 give constants
//     (the sign of byte 1, 3, 5 or 7 for 8..11, then 0, 0xFF, 0xFF, 0xFF).  So the low 8 entries of a byte plane
//     looked up by the code and the high 8 by the code ^ 8 each give, for the codes that are not theirs, a constant
//     of the code, which is xored into the tables beforehand: 2 permutes and a xor per plane of 4 codes, and 2 permutes
//     to interleave the planes: 21 VALU for 8 elements.
struct CodePlanes {
  uint32_t lo[4], hi[4];   // [0..1] entries 0..7, [2..3] entries 8..15 of the low and the high bytes
  float inv;               // 1 / c
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x4 mfma16h(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// two fp32 -> fp16, round to nearest even
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) * __builtin_bit_cast(f16x2, b));
}
__device__ __forceinline__ u32x4 decode_planes(const CodePlanes& p, uint32_t w) {
  u32x4 o;
#pragma unroll
  for (int half = 0; half < 2; ++half) {   // elements 0..3 in the low nibbles, 4..7 in the high ones
    const uint32_t a = (half ? w >> 4 : w) & 0x0F0F0F0Fu, b = a ^ 0x08080808u;
    const uint32_t lo = __builtin_amdgcn_perm(p.lo[1], p.lo[0], a) ^ __builtin_amdgcn_perm(p.lo[3], p.lo[2], b);
    const uint32_t hi = __builtin_amdgcn_perm(p.hi[1], p.hi[0], a) ^ __builtin_amdgcn_perm(p.hi[3], p.hi[2], b);
    o[2 * half] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
    o[2 * half + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  }
  return o;
}
// elements in the order 0, 4, 1, 5, 2, 6, 3, 7 (byte i holds i and i + 4)
__device__ __forceinline__ u32x4 decode_pairs(const uint32_t* pair, uint32_t w) {
  return u32x4{pair[w & 0xFFu], pair[(w >> 8) & 0xFFu], pair[(w >> 16) & 0xFFu], pair[w >> 24]};
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127
// exponent of a bf16 magnitude, kept where its power of two and the inverse are ordinary numbers
__device__ __forceinline__ int exponent_of(uint32_t mag) { return min(max((int)(mag >> 7) - 127, -100), 126); }
// What a row of q is multiplied with: 2^-e, or NaN where it holds an infinity (or a NaN): its logits have no softmax, but
// where all of them are -inf they would pass for those of masked tokens.
__device__ __forceinline__ float row_unit(uint32_t mag, int e) { return mag < 0x7F80u ? pow2(-e) : __builtin_nanf(""); }

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v = dpp_max<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  v = dpp_max<0x141>(v);   // row_half_mirror
  v = dpp_max<0x140>(v);   // row_mirror
  auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max(a[0], a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return __builtin_amdgcn_readfirstlane(max(b[0], b[1]));
}

// Sequence b as a call sees it.
struct Seq {
  int64_t row0;   // first row
  int32_t n;      // rows (tokens of this call); 0 if its start entries are wrong
  int32_t len;    // tokens in the cache; -1 if the entry is wrong
};

__device__ __forceinline__ Seq seq_of(const BatchView& b, int i) {
  Seq s;
  const int64_t s0 = b.start[i], s1 = b.start[i + 1];
  const int len = b.length[i];
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= b.rows;
  s.row0 = ok ? s0 : 0;
  s.n = ok ? (int)(s1 - s0) : 0;
  s.len = (len < 0 || len > b.max_len) ? -1 : len;
  return s;
}

// The same value, but what is computed from it is not moved to before this point: addresses of code outside a loop,
// formed ahead of it, would be held in registers all through it (50 of them, here).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// T sequences from c0 on: what the kernels need of them, and the sum of count(sequence) before each.
template <int T>
struct SeqTable {
  int32_t pre[T + 1];
  int32_t row0[T], n[T], len[T];
  int32_t wave_tot[T / 64];
  // entry i, as scalars
  __device__ __forceinline__ Seq seq(int i) const {
    return Seq{__builtin_amdgcn_readfirstlane(row0[i]), __builtin_amdgcn_readfirstlane(n[i]),
               __builtin_amdgcn_readfirstlane(len[i])};
  }
};
template <int T, class F>
__device__ __forceinline__ void scan_seqs(const BatchView& b, int c0, int base, SeqTable<T>& q, F count) {
  const int t = opaque(threadIdx.x), i = c0 + t, lane = t & 63, w = t >> 6;
  // Each count and, for entries in order, their sum is at most 2^30.  Entries out of order can give the same rows to
  // many sequences: the sums stop at 2^30 then, and what lies past it is left out.
  auto add = [](int x, int y) { return (int)min((uint32_t)x + (uint32_t)y, 1u << 30); };
  int u = 0;
  if (i < b.batch) {
    const Seq s = seq_of(b, i);
    u = count(s);
    q.row0[t] = (int)s.row0;
    q.n[t] = s.n;
    q.len[t] = s.len;
  }
  int inc = u;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(inc, off, 64);
    if (lane >= off) inc = add(inc, o);
  }
  if (lane == 63) q.wave_tot[w] = inc;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < T / 64 - 1; ++k)
    if (k < w) inc = add(inc, q.wave_tot[k]);
  q.pre[t + 1] = add(base, inc);
  if (t == 0) q.pre[0] = base;
  __syncthreads();
}

// One workgroup's check of all entries of the batch (the kernels leave out what is wrong; this reports it).
template <int T>
__device__ __forceinline__ void check_batch_entries(const BatchView& b) {
  for (int i = threadIdx.x; i < b.batch; i += T) {
    const int64_t s0 = b.start[i], s1 = b.start[i + 1];
    if (s0 < 0 || s1 < s0 || s1 > b.rows) raise_fault(b, kFaultStart);
    const int len = b.length[i];
    if (len < 0 || len > b.max_len) raise_fault(b, kFaultLength);
  }
}

// The tile of a segment, in registers that are the same in every lane.
struct Tile {
  Seq s;
  int32_t b, h, rho0, nval;      // sequence, cache head, first row of the tile and rows it has
  int32_t base, hi, hi_min, lo_max;   // tokens base .. hi - 1 hold what its rows see, lo_max .. hi_min - 1 are seen by all
  int32_t skip;                       // how many tokens from base on, fewer than 64, no row sees
};

// n / a.group for 0 <= n < 2^31 (a product and a shift: a division is 30 dependent instructions)
__device__ __forceinline__ int div_group(const AttnArgs& a, int n) {
  return (int)((uint64_t)(uint32_t)n * a.group_mul >> a.group_shift);
}

template <int TR>
__device__ __forceinline__ Tile tile_of(const AttnArgs& a, const Seq& s, int b, int h, int rt) {
  Tile t;
  t.s = s;
  t.b = b;
  t.h = h;
  t.rho0 = rt * TR;
  const int left = (int)((int64_t)s.n * a.group - t.rho0);
  t.nval = left < TR ? left : TR;
  const int len = s.len < 0 ? 0 : s.len;
  const int p0 = len - s.n + div_group(a, t.rho0), p1 = len - s.n + div_group(a, t.rho0 + t.nval - 1);
  t.hi = a.causal ? max(p1 + 1, 0) : len;
  t.hi_min = a.causal ? p0 + 1 : len;
  const int lo = a.window ? max(p0 + 1 - a.window, 0) : 0;
  t.lo_max = a.window ? max(p1 + 1 - a.window, 0) : 0;
  t.base = lo & ~63;
  t.skip = lo & 63;
  return t;
}

// Row rr of a tile from its n parts, by one wave.  part(k): part k, [rows][D] sums, then [rows] maxima (log2), then
// [rows] sums of probabilities; element(d): the element at position d of a row.  mt: the tile's entry.  Eight parts are
// read at a time, so that their loads are in flight together.
template <int D, class P, class E>
__device__ __forceinline__ void join_row(const AttnArgs& a, int n, int rows, int rr, const int32_t* mt, P part, E element) {
  constexpr int C = D / 64;   // columns of a lane
  typedef float vec __attribute__((ext_vector_type(C)));
  const int lane = threadIdx.x & 63;
  float m = neg_inf(), l = 0.0f;
  vec o = 0.0f;
  for (int k0 = 0; k0 < n; k0 += 8) {
    float pm[8], pl[8];
    vec po[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* p = part(min(k0 + i, n - 1));
      pm[i] = p[rows * D + rr];
      pl[i] = p[rows * D + rows + rr];
      po[i] = *reinterpret_cast<const vec*>(p + rr * D + lane * C);
    }
    float mx = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k0 + i >= n) pm[i] = neg_inf(), pl[i] = 0.0f, po[i] = 0.0f;
      mx = fmaxf(mx, pm[i]);
    }
    const float mu = mx == neg_inf() ? 0.0f : mx;
    const float f0 = __builtin_amdgcn_exp2f(m - mu);
    m = mx;
    l *= f0;
    o *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = __builtin_amdgcn_exp2f(pm[i] - mu);
      l = __builtin_fmaf(pl[i], f, l);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = __builtin_fmaf(po[i][c], f, o[c]);
    }
  }
  const int rho = mt[2] + rr, i = div_group(a, rho), qh = mt[4] * a.group + (rho - i * a.group);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = a.o.data + (mt[1] + i) * a.o.rs + qh * a.o.hs;
#pragma unroll
  for (int c = 0; c < C; ++c) out[element(lane * C + c)] = (uint16_t)(pack_bf16x2(o[c] * inv, 0.0f) & 0xFFFFu);
  if (a.lse && lane == 0)
    a.lse[(mt[1] + i) * (int64_t)a.q.n + qh] = l == 0.0f ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// The kernel for many rows cuts the tokens of its tiles into as many parts as kSplitWgs workgroups, one per CU, are enough
// for, of at least this many tokens.  A part's sums cost 130 KB written and read where all 256 rows of its tile are there
// (8 cache heads of 128, 1024 rows of 1024 tokens: parts of 256 50 us, of 1024, so uncut, 48; D = 64 45 and 36; 512
// rows of 4096 62 and 63, of 2048 94), little where few are (32 rows of 4096: D = 128 24 us with parts of 256, 28 of 512; D = 256,
// whose tiles are half as large, 41 and 53).
constexpr int kSplitWgs = 256;
constexpr int split_tokens_of(int D, bool sparse) { return sparse || D == 256 ? 256 : 1024; }

// Threads of a workgroup of the kernel for many rows: 32 rows of a tile to a wave, 8 waves where the registers allow two
// waves per SIMD, 4 otherwise.
constexpr int many_threads(int D) { return D == 256 ? 256 : 512; }

}  // namespace qlora
