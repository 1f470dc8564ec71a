// Attention over the 4-bit cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),  k_j = level[c] s,  v_j = level[c] s
//
// One pass over the cache with a running maximum and sum.  A tile is TR rows of q, a row being one
// (token, query head) of one cache head, so that all query heads of a group use a key once it is decoded; the
// work of a tile is cut into units of 256 tokens, and all units of the call, laid end to end, are
// cut into equal ranges, one per workgroup, by the kernel itself from the device's lengths.  A ragged batch
// is so balanced without the host knowing it, and one long sequence uses the whole GPU.  A range that
// holds all of a tile's units writes its output; otherwise it writes its sums to the workspace (a range has
// at most two such tiles, its first and its last), and k_kv_attn_join adds them in the order of the tokens.
//
// A wave takes 64 tokens at a time, on its own (no barrier until the end of a tile):
//   S^T = K Q^T (16x16x32 MFMA, K as the row operand): a lane holds the codes of one token's 32
//     elements in one 16-byte load (the key rows' dword order), decodes them to bf16 by byte
//     permutes of a constant table, and the block's scale is applied to the accumulators, 4 tokens per lane,
//     instead of to 32 elements;
//   P^T falls out of that in the layout that the next product's column operand has: which token is which
//     row of the S^T tiles is chosen so that lane group g holds tokens 16g .. 16g + 15;
//   O^T = V^T P^T: the value codes go through LDS as they are and come back transposed by nibbles
//     (ds_read_b64_tr_b4: a lane gets 16 tokens of one element), so 4 bits per element cross LDS instead
//     of 16; the scale of a value depends on the token, the reduction index here, so it is multiplied
//     into P, once per block.
// The tables hold level * kLevelScale: FP4 (x 6) and Int4 (x 7) levels are then exact in bf16, NF4's
// (x 1.43675) off by 2^-10.2 rms instead of 2^-9.5.
#include "kernels.h"
#include "kv.h"

namespace qlora {

namespace {

constexpr int AT = 256, AW = AT / 64;
constexpr int kStep = 64;              // tokens per wave step
constexpr int kUnit = kStep * AW;      // tokens per unit of work
constexpr int kMetaInts = 8;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct CodePlanes {
  uint32_t lo[4], hi[4];   // as Planes: bytes of bf16(level * kLevelScale)
  float inv;               // 1 / kLevelScale
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// maximum over the four lane groups (lanes l % 16 + 16 g)
__device__ __forceinline__ float group_max(float v) {
  uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  u = __float_as_uint(m);
  auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float v) {
  uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  u = __float_as_uint(m);
  auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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

// Units of every tile of a sequence: enough for the tile that sees the most tokens.
template <int TR>
__device__ __forceinline__ int units_of(const AttnArgs& a, const Seq& s) {
  int64_t span = s.len < 0 ? 0 : s.len;
  if (a.window) {
    const int64_t tokens = (TR + a.group - 1) / a.group + 1;   // tokens a tile's rows can belong to
    const int64_t w = (int64_t)a.window + tokens + kStep;
    if (w < span) span = w;
  }
  const int u = (int)((span + kUnit - 1) / kUnit);
  return u > 0 ? u : 1;
}
template <int TR>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Seq& s) {
  return (int)(((int64_t)s.n * a.group + TR - 1) / TR);
}

// Prefix sums of the units of 256 sequences from c0 on: pre[i] = units before sequence c0 + i.
template <int TR>
__device__ void scan_units(const AttnArgs& a, int c0, int64_t base, int64_t* pre, int64_t* wave_tot) {
  const int t = threadIdx.x, i = c0 + t, lane = t & 63, w = t >> 6;
  int64_t u = 0;
  if (i < a.b.batch) {
    const Seq s = seq_of(a.b, i);
    u = (int64_t)tiles_of<TR>(a, s) * units_of<TR>(a, s) * a.c.heads;
  }
  int64_t inc = u;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(inc, off, 64);
    if (lane >= off) inc += o;
  }
  if (lane == 63) wave_tot[w] = inc;
  __syncthreads();
  for (int k = 0; k < w; ++k) inc += wave_tot[k];
  pre[t + 1] = base + inc;
  if (t == 0) pre[0] = base;
  __syncthreads();
}

// The tile of a segment, in registers that are the same in every lane.
struct Tile {
  Seq s;
  int32_t b, h, rho0, nval;      // sequence, cache head, first row of the tile and rows it has
  int32_t base, hi, hi_min, lo_max;   // tokens base .. hi - 1 are seen by some row, lo_max .. hi_min - 1 by all
};

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
  const int p0 = len - s.n + t.rho0 / a.group, p1 = len - s.n + (t.rho0 + t.nval - 1) / a.group;
  t.hi = a.causal ? max(p1 + 1, 0) : len;
  t.hi_min = a.causal ? p0 + 1 : len;
  const int lo = a.window ? max(p0 + 1 - a.window, 0) : 0;
  t.lo_max = a.window ? max(p1 + 1 - a.window, 0) : 0;
  t.base = lo & ~(kStep - 1);
  return t;
}

// Registers of one step's loads.
template <int D, int NB>
struct StepLoads {
  static constexpr int KW = D == 64 ? 1 : D / 128;   // 16-byte (D = 64: 8-byte) loads per token tile
  static constexpr int VL = D / 32;                  // 16-byte loads of the values
  u32x4 k[4][KW];
  u32x4 v[VL];
  uint32_t ks[(NB + 1) / 2], vs[(NB + 1) / 2];       // this lane's token's scales
};

template <int D, int NB, int NR>
__global__ __launch_bounds__(AT, 2) void k_kv_attn(AttnArgs a, CodePlanes cp) {
  constexpr int TR = 16 * NR, B = D / NB, KK = D / 32, UN = D / 16;
  constexpr int RB = D / 2;                // bytes of a cache row
  constexpr int CH = RB / 16;              // 16-byte chunks of a row
  constexpr int kVBytes = kStep * RB;      // a wave's value codes
  constexpr int kScaleFloats = 2 * NB * kStep;
  constexpr int kWaveBytes = kVBytes + kScaleFloats * 4;
  constexpr int kMergeBytes = 2 * TR * (D + 4) * 4;
  constexpr int kShared = AW * kWaveBytes > kMergeBytes ? AW * kWaveBytes : kMergeBytes;
  __shared__ __attribute__((aligned(16))) unsigned char smem[kShared];
  __shared__ float ml[AW][2][TR];
  __shared__ int64_t pre[AT + 1];
  __shared__ int64_t wave_tot[AW];
  __shared__ int found;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  unsigned char* const vbuf = smem + wave * kWaveBytes;
  float* const kscale = reinterpret_cast<float*>(vbuf + kVBytes);
  float* const vscale = kscale + NB * kStep;
  Planes P;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    P.lo[i] = cp.lo[i];
    P.hi[i] = cp.hi[i];
  }
  const float kmul = a.scale * kLog2e * cp.inv, vmul = cp.inv;

  // this workgroup's range of units
  scan_units<TR>(a, 0, 0, pre, wave_tot);
  int c0 = 0;
  int64_t total = pre[AT];
  for (int c = AT; c < a.b.batch; c += AT) {   // more than 256 sequences: the total first, then back to the front
    __syncthreads();
    scan_units<TR>(a, c, total, pre, wave_tot);
    total = pre[AT];
    c0 = c;
  }
  const int64_t W = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x, w = blockIdx.x;   // no empty ranges below W
  const int64_t lo = w < W ? total * w / W : 0, hi = w < W ? total * (w + 1) / W : 0;
  if (threadIdx.x == 0) a.meta[w * kMetaInts] = -1;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.b.batch; i += AT) {
      const int64_t s0 = a.b.start[i], s1 = a.b.start[i + 1];
      if (s0 < 0 || s1 < s0 || s1 > a.b.rows) raise_fault(a.b, kFaultStart);
      const int len = a.b.length[i];
      if (len < 0 || len > a.b.max_len) raise_fault(a.b, kFaultLength);
    }
  if (lo >= hi) return;
  if (c0 != 0) {
    int64_t base = 0;
    for (c0 = 0;; c0 += AT) {
      __syncthreads();
      scan_units<TR>(a, c0, base, pre, wave_tot);
      if (pre[AT] > lo) break;
      base = pre[AT];
    }
  }

  for (int64_t cur = lo; cur < hi;) {
    // the sequence that holds unit `cur`
    while (pre[AT] <= cur) {
      const int64_t base = pre[AT];
      __syncthreads();
      c0 += AT;
      scan_units<TR>(a, c0, base, pre, wave_tot);
    }
    if (pre[threadIdx.x] <= cur && cur < pre[threadIdx.x + 1]) found = threadIdx.x;
    __syncthreads();
    const int bi = __builtin_amdgcn_readfirstlane(found);
    const Seq s = seq_of(a.b, c0 + bi);
    const int units = units_of<TR>(a, s), tiles = tiles_of<TR>(a, s);
    const int64_t rem = cur - pre[bi];
    const int64_t tile_id = rem / units;      // (head, tile) of the sequence
    const int u0 = (int)(rem - tile_id * units);
    const int u1 = (int)(hi - cur < units - u0 ? u0 + (hi - cur) : units);
    const int h = (int)(tile_id / tiles), rt = (int)(tile_id - (int64_t)h * tiles);
    const Tile t = tile_of<TR>(a, s, c0 + bi, h, rt);
    const int64_t item0 = cur - u0;           // the tile's first unit
    const bool whole = u0 == 0 && u1 == units;

    // rows of this lane: row r * 16 + l16 of the tile
    u32x4 qf[NR][KK];
    int32_t r_lo[NR], r_hi[NR];               // tokens it sees
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int rr = r * 16 + l16;
      const bool ok = rr < t.nval;
      const int rho = t.rho0 + (ok ? rr : 0);
      const int i = rho / a.group, qh = t.h * a.group + (rho - i * a.group);
      const int len = s.len < 0 ? 0 : s.len;
      const int p = len - s.n + i;
      r_hi[r] = !ok ? 0 : a.causal ? p + 1 : len;
      r_lo[r] = a.window ? p + 1 - a.window : 0;
      const uint16_t* qp = a.q.data + (s.row0 + i) * a.q.rs + qh * a.q.hs;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        qf[r][k] = *reinterpret_cast<const u32x4*>(qp + 32 * k + 8 * g);
        if (!ok) qf[r][k] = u32x4{0, 0, 0, 0};
      }
    }

    f32x4 O[NR][UN];
    float m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = neg_inf();
      l[r] = 0.0f;
#pragma unroll
      for (int u = 0; u < UN; ++u) O[r][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int steps = t.hi > t.base ? (t.hi - t.base + kStep - 1) / kStep : 0;
    const int st_end = min(u1 * AW, steps);

    // page of this lane group's 16 tokens of a step: -1 past the last token, -2 where the entry is wrong
    auto page_at = [&](int st) -> int {
      const int tok = t.base + st * kStep + 16 * g;
      if (st >= st_end || tok >= t.hi) return -1;
      const int pid = a.b.table[(int64_t)t.b * a.b.max_pages + (tok >> a.c.pshift)];
      if (pid < 0 || pid >= a.c.pages) {
        if (l16 == 0) raise_fault(a.b, kFaultPage);
        return -2;
      }
      return pid;
    };
    auto row_of = [&](int pid, int tok) -> int64_t {   // row of the cache's buffers (row 0 where there is none)
      return pid < 0 ? 0 : (((int64_t)pid * a.c.heads + t.h) << a.c.pshift) + (tok & ((1 << a.c.pshift) - 1));
    };
    auto load = [&](StepLoads<D, NB>& L, int st, int pid) {
      const int tok0 = t.base + st * kStep;
      // keys: row 4a + i of token tile tt is token 16a + 4tt + i
      const int ka = l16 >> 2;
      const int kp = __shfl(pid, 16 * ka, 64);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const uint8_t* p = a.c.kc + row_of(kp, tok0 + 16 * ka + 4 * tt + (l16 & 3)) * RB;
        if constexpr (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(p + 8 * g);
          L.k[tt][0] = u32x4{x.x, x.y, 0, 0};
        } else {
#pragma unroll
          for (int k = 0; k < StepLoads<D, NB>::KW; ++k)
            L.k[tt][k] = *reinterpret_cast<const u32x4*>(p + 64 * k + 16 * g);
        }
      }
      // values: CH lanes per token
#pragma unroll
      for (int i = 0; i < StepLoads<D, NB>::VL; ++i) {
        const int tk = i * (64 / CH) + lane / CH;
        const int vp = __shfl(pid, tk & ~15, 64);
        L.v[i] = *reinterpret_cast<const u32x4*>(a.c.vc + row_of(vp, tok0 + tk) * RB + 16 * (lane & (CH - 1)));
      }
      // scales of token `lane`
      const int64_t row = row_of(pid, tok0 + lane) * NB;
      if constexpr (NB == 1) {
        L.ks[0] = a.c.ks[row];
        L.vs[0] = a.c.vs[row];
      } else {
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
          L.ks[k] = reinterpret_cast<const uint32_t*>(a.c.ks + row)[k];
          L.vs[k] = reinterpret_cast<const uint32_t*>(a.c.vs + row)[k];
        }
      }
      // no token: scale 0; no page: NaN
      const bool none = tok0 + lane >= t.hi;
#pragma unroll
      for (int k = 0; k < (NB + 1) / 2; ++k) {
        if (pid == -2) L.ks[k] = L.vs[k] = kBf16NaN * 0x10001u;
        if (none) L.ks[k] = L.vs[k] = 0;
      }
    };

    int st = u0 * AW + wave;
    StepLoads<D, NB> L;
    int pid = page_at(st);
    int pid_next = page_at(st + AW);
    if (st < st_end) load(L, st, pid);
    for (; st < st_end; st += AW) {
      const int tok0 = t.base + st * kStep;
      // value codes and scales to LDS, this wave's own part of it (a wave's LDS accesses stay in order)
#pragma unroll
      for (int i = 0; i < StepLoads<D, NB>::VL; ++i) {
        const int tk = i * (64 / CH) + lane / CH, c = lane & (CH - 1);
        // chunks turned by the token, so that 16 tokens' pieces of one column lie in different banks
        constexpr int SH = D == 64 ? 3 : D == 128 ? 2 : 1;
        *reinterpret_cast<u32x4*>(vbuf + tk * RB + 16 * (c ^ ((tk >> SH) & (CH - 1)))) = L.v[i];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t kw = b & 1 ? L.ks[b / 2] >> 16 : L.ks[b / 2] & 0xFFFFu;
        const uint32_t vw = b & 1 ? L.vs[b / 2] >> 16 : L.vs[b / 2] & 0xFFFFu;
        kscale[b * kStep + lane] = bf16_to_f32(kw) * kmul;
        vscale[b * kStep + lane] = bf16_to_f32(vw) * vmul;
      }
      u32x4 kc[4][StepLoads<D, NB>::KW];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int k = 0; k < StepLoads<D, NB>::KW; ++k) kc[tt][k] = L.k[tt][k];
      // the next step's loads run under this step's work
      if (st + AW < st_end) {
        load(L, st + AW, pid_next);
        pid_next = page_at(st + 2 * AW);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

      // S^T: rows = tokens, columns = rows of q
      f32x4 S[NR][4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          f32x4 acc[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = b * (B / 32); k < (b + 1) * (B / 32); ++k) {
            const u32x4 kf = dequant8(P, kc[tt][k / 4][k % 4]);
#pragma unroll
            for (int r = 0; r < NR; ++r) acc[r] = mfma16(kf, qf[r][k], acc[r]);
          }
          const f32x4 sk = *reinterpret_cast<const f32x4*>(kscale + b * kStep + 16 * g + 4 * tt);
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              S[r][tt][i] = b == 0 ? acc[r][i] * sk[i] : __builtin_fmaf(acc[r][i], sk[i], S[r][tt][i]);
        }
      }

      const bool edge = tok0 < t.lo_max || tok0 + kStep > t.hi_min;
      uint32_t vis[NR];   // bit 4tt + i: the lane's row sees that token
#pragma unroll
      for (int r = 0; r < NR; ++r) vis[r] = 0xFFFFu;
      if (edge) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          vis[r] = 0;
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = tok0 + 16 * g + 4 * tt + i;
              const bool see = tok >= r_lo[r] && tok < r_hi[r];
              if (!see) S[r][tt][i] = neg_inf();
              vis[r] |= see ? 1u << (4 * tt + i) : 0u;
            }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float mx = S[r][0][0];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, S[r][tt][i]);
        mx = fmaxf(group_max(mx), m[r]);
        const float mu = mx == neg_inf() ? 0.0f : mx;
        if (__any(mx > m[r])) {
          const float alpha = __builtin_amdgcn_exp2f(m[r] - mu);
          l[r] *= alpha;
#pragma unroll
          for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[r][u][i] *= alpha;
        }
        m[r] = mx;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            S[r][tt][i] = __builtin_amdgcn_exp2f(S[r][tt][i] - mu);
            l[r] += S[r][tt][i];
          }
      }

      // O^T += V^T (P s)^T, one block of elements at a time
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 pf[NR][2];   // tokens 16g + 0..7 and + 8..15
        f32x4 sv[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) sv[tt] = *reinterpret_cast<const f32x4*>(vscale + b * kStep + 16 * g + 4 * tt);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              float x = S[r][tt][i] * sv[tt][i], y = S[r][tt][i + 1] * sv[tt][i + 1];
              // a scale can be NaN: what the row does not see is left out, not multiplied by zero
              if (!(vis[r] >> (4 * tt + i) & 1u)) x = 0.0f;
              if (!(vis[r] >> (4 * tt + i + 1) & 1u)) y = 0.0f;
              pf[r][tt / 2][2 * (tt & 1) + i / 2] = pack_bf16x2(x, y);
            }
#pragma unroll
        for (int u = b * (B / 16); u < (b + 1) * (B / 16); ++u) {
          // row of lane n of the 16: token 8 (n / 8) + (n % 8) / 2 + 4 (n % 2), so that the dword of 8 tokens
          // decodes in token order
          const int tk = 16 * g + (l16 & 8) + ((l16 & 7) >> 1) + 4 * (l16 & 1);
          constexpr int SH = D == 64 ? 3 : D == 128 ? 2 : 1;
          const int off = tk * RB + 16 * ((u >> 1) ^ ((tk >> SH) & (CH - 1))) + 8 * (u & 1);
          typedef int v2i __attribute__((ext_vector_type(2)));
          const v2i w2 =
              __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) v2i*)(vbuf + off));
          const u32x4 v0 = dequant8(P, (uint32_t)w2[0]), v1 = dequant8(P, (uint32_t)w2[1]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            O[r][u] = mfma16(v0, pf[r][0], O[r][u]);
            O[r][u] = mfma16(v1, pf[r][1], O[r][u]);
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

    // the four waves' sums, two by two
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] = group_sum(l[r]);
      if (g == 0) {
        ml[wave][0][r * 16 + l16] = m[r];
        ml[wave][1][r * 16 + l16] = l[r];
      }
    }
    __syncthreads();   // also: every wave is done with its value buffer
    float mt[NR], lt[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      mt[r] = neg_inf();
#pragma unroll
      for (int k = 0; k < AW; ++k) mt[r] = fmaxf(mt[r], ml[k][0][r * 16 + l16]);
      const float mu = mt[r] == neg_inf() ? 0.0f : mt[r];
      lt[r] = 0.0f;
#pragma unroll
      for (int k = 0; k < AW; ++k)
        lt[r] += ml[k][1][r * 16 + l16] * __builtin_amdgcn_exp2f(ml[k][0][r * 16 + l16] - mu);
      const float f = __builtin_amdgcn_exp2f(m[r] - mu);
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[r][u][i] *= f;
    }
    float* const mg = reinterpret_cast<float*>(smem);
    constexpr int LDO = D + 4;
#pragma unroll
    for (int round = 2; round >= 1; round >>= 1) {
      if (wave >= round && wave < 2 * round) {
        float* d = mg + (wave - round) * TR * LDO;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int u = 0; u < UN; ++u) *reinterpret_cast<f32x4*>(d + (r * 16 + l16) * LDO + u * 16 + 4 * g) = O[r][u];
      }
      __syncthreads();
      if (wave < round) {
        const float* d = mg + wave * TR * LDO;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(d + (r * 16 + l16) * LDO + u * 16 + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) O[r][u][i] += x[i];
          }
      }
      __syncthreads();
    }

    if (wave == 0) {
      if (whole) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int rr = r * 16 + l16;
          if (rr >= t.nval) continue;
          const int rho = t.rho0 + rr, i = rho / a.group, qh = t.h * a.group + (rho - i * a.group);
          float inv = lt[r] == 0.0f ? 0.0f : 1.0f / lt[r];
          if (s.len < 0) inv = __builtin_nanf("");
          uint16_t* op = a.o.data + (s.row0 + i) * a.o.rs + qh * a.o.hs;
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            // rows 4g + i of the tile: elements d, d + 4, d + 1, d + 5
            uint32_t* d = reinterpret_cast<uint32_t*>(op + 16 * u + 8 * (g >> 1) + 2 * (g & 1));
            d[0] = pack_bf16x2(O[r][u][0] * inv, O[r][u][2] * inv);
            d[2] = pack_bf16x2(O[r][u][1] * inv, O[r][u][3] * inv);
          }
          if (a.lse && g == 0)
            a.lse[(s.row0 + i) * a.q.n + qh] =
                s.len < 0 ? __builtin_nanf("") : lt[r] == 0.0f ? neg_inf() : (mt[r] + __builtin_amdgcn_logf(lt[r])) * kLn2;
        }
      } else {
        // slot 0: the range's first tile, begun in an earlier range; slot 1: its last, ending in a later one
        float* d = a.part + (2 * w + (u0 == 0 ? 1 : 0)) * (int64_t)(TR * (D + 2));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int rr = r * 16 + l16;
#pragma unroll
          for (int u = 0; u < UN; ++u)
            *reinterpret_cast<f32x4*>(d + rr * D + u * 16 + 4 * g) = O[r][u];
          if (g == 0) {
            d[TR * D + rr] = mt[r];
            d[TR * D + TR + rr] = lt[r];
          }
        }
        if (u0 != 0 && u1 == units && lane == 0) {
          // this range ends the tile: the join of its partial sums is noted here
          int32_t* mt_ = a.meta + w * kMetaInts;
          mt_[0] = (int32_t)(((item0 + 1) * W - 1) / total);   // the workgroup whose range holds its first unit
          mt_[1] = (int32_t)s.row0;
          mt_[2] = t.rho0;
          mt_[3] = t.nval;
          mt_[4] = t.h;
        }
      }
    }
    cur += u1 - u0;
    __syncthreads();
  }
}

// Adds the partial sums of a tile that was cut: workgroup (w, y) the tile that ends in range w, if any,
// rows y, y + gridDim.y, ...  The parts lie in slot 1 of the first range and slot 0 of the others.
template <int D, int TR>
__global__ __launch_bounds__(D) void k_kv_attn_join(AttnArgs a) {
  const int64_t w = blockIdx.x;
  const int32_t* mt = a.meta + w * kMetaInts;
  const int64_t w0 = mt[0];
  if (w0 < 0) return;
  const int d = threadIdx.x;
  constexpr int64_t P = TR * (D + 2);
  for (int rr = blockIdx.y; rr < mt[3]; rr += gridDim.y) {
    float m = neg_inf();
    for (int64_t k = w0; k <= w; ++k) m = fmaxf(m, a.part[(2 * k + (k == w0)) * P + TR * D + rr]);
    const float mu = m == neg_inf() ? 0.0f : m;
    float l = 0.0f, o = 0.0f;
    for (int64_t k = w0; k <= w; ++k) {
      const float* p = a.part + (2 * k + (k == w0)) * P;
      const float f = __builtin_amdgcn_exp2f(p[TR * D + rr] - mu);
      l = __builtin_fmaf(p[TR * D + TR + rr], f, l);
      o = __builtin_fmaf(p[rr * D + d], f, o);
    }
    const int rho = mt[2] + rr, i = rho / a.group, qh = mt[4] * a.group + (rho - i * a.group);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    // position d of a partial row: row d % 16 of column tile d / 16
    const int e = (d & ~15) + (d & 8) + ((d & 7) >> 1) + 4 * (d & 1);
    a.o.data[(mt[1] + i) * a.o.rs + qh * a.o.hs + e] = (uint16_t)(pack_bf16x2(o * inv, 0.0f) & 0xFFFFu);
    if (a.lse && d == 0)
      a.lse[(mt[1] + i) * (int64_t)a.q.n + qh] = l == 0.0f ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

uint16_t bf16_host(float f) {
  uint32_t b;
  __builtin_memcpy(&b, &f, 4);
  return (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

CodePlanes planes_host(int cb) {
  CodePlanes p{};
  const float c = cb == QLORA_CODEBOOK_FP4 ? 6.0f : cb == QLORA_CODEBOOK_INT4 ? 7.0f : 1.43675f;
  const float* lv = codebook_levels_host(cb);
  for (int i = 0; i < 16; ++i) {
    const uint16_t h = bf16_host(lv[i] * c);
    p.lo[i / 4] |= (uint32_t)(h & 0xFF) << (8 * (i % 4));
    p.hi[i / 4] |= (uint32_t)(h >> 8) << (8 * (i % 4));
  }
  p.inv = 1.0f / c;
  return p;
}

}  // namespace

AttnPlan attn_plan(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t batch, int64_t max_len, int D) {
  AttnPlan p;
  const int64_t group = q_heads / kv_heads;
  p.tile = 16;
  const int64_t tiles = ((rows * group + p.tile - 1) / p.tile + batch) * kv_heads;
  const int64_t units = (max_len + kUnit - 1) / kUnit + 1;
  p.wgs = 768;
  if (tiles < p.wgs && tiles * units < p.wgs) p.wgs = tiles * units;
  p.part_floats = (size_t)p.wgs * 2 * p.tile * (D + 2);
  p.meta_ints = (size_t)p.wgs * kMetaInts;
  return p;
}

template <int D, int NB>
static hipError_t launch_attn(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  {
    ProfScope ps("k_kv_attn", s);
    hipLaunchKernelGGL((k_kv_attn<D, NB, 1>), dim3((unsigned)pl.wgs), dim3(AT), 0, s, a, planes_host(a.c.cb));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ProfScope ps("k_kv_attn_join", s);
  hipLaunchKernelGGL((k_kv_attn_join<D, 16>), dim3((unsigned)pl.wgs, 4), dim3(D), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s) {
  const int nb = D / block;
  if (D == 64) return nb == 1 ? launch_attn<64, 1>(a, pl, s) : launch_attn<64, 2>(a, pl, s);
  if (D == 128)
    return nb == 1 ? launch_attn<128, 1>(a, pl, s) : nb == 2 ? launch_attn<128, 2>(a, pl, s) : launch_attn<128, 4>(a, pl, s);
  return nb == 2 ? launch_attn<256, 2>(a, pl, s) : nb == 4 ? launch_attn<256, 4>(a, pl, s) : launch_attn<256, 8>(a, pl, s);
}

}  // namespace qlora
