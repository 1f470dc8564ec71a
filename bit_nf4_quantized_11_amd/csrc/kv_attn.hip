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
//     elements in one 16-byte load (the key rows' dword order), decodes them to fp16 by lookups of
//     pairs of codes in LDS, and the block's scale is applied to the accumulators, 4 tokens per lane,
//     instead of to 32 elements;
//   P^T falls out of that in the layout that the next product's column operand has: which token is which
//     row of the S^T tiles is chosen so that lane group g holds tokens 16g .. 16g + 15;
//   O^T = V^T P^T: the value codes go through LDS as they are and come back transposed by nibbles
//     (ds_read_b64_tr_b4: a lane gets 16 tokens of one element), so 4 bits per element cross LDS instead
//     of 16, and are decoded by byte permutes (the keys' lookups leave LDS no time for theirs); the scale of a
//     value depends on the token, the reduction index here, so it is multiplied into P, once per block.
// The products are in fp16, not bf16: its 11 bits bring the level tables (times 6 for FP4 and 7 for Int4, which
// makes them exact) and the probabilities 8 times closer, and the output's error down to little more than
// its own rounding to bf16 (with bf16 operands it was twice that).  What fp16 lacks is range, so every operand is
// brought to about 1 by a power of two first: a row of q by its own largest element (all 8 bits of elements down to
// 2^-17 of it stay), the scaled probabilities of a step by the largest scale so far of that
// block of elements (a running exponent, like the running maximum, that all rows share).
//
// Measured: 16 sequences of up to 32768 tokens (311 k in all, 338 MB), 64 query on 8 cache heads of 128: 84 us a pass =
// 4.0 TB/s, where a large copy reaches 4.8 (in a trace 81 to 94 of this kernel and 5 of the join, where an empty kernel has
// 2.5 to 4): the steps are bound by HBM (a step's 18.9 MB in 4 us when all 2048 waves are in theirs), VALU issue close behind.
// A tile of a single step takes about 10500 cycles of one workgroup: 1200 to find it, 2400 for table, queries and codes, 6000
// for the step, 1000 for the waves' sums; two workgroups to a CU overlap half of that: 1000 sequences of one token 84 us, 512
// of 128 tokens 51 (17 at copy rate), 16 of 4096 23 (15), one of 777 tokens 9.
#include <algorithm>

#include "kv_attn.h"

namespace qlora {

namespace {

constexpr int AT = 256, AW = AT / 64;
constexpr int kStep = 64;              // tokens per wave step
constexpr int kUnitShift = 8;          // log2 of the tokens per unit of work: one step of every wave
static_assert(kStep * AW == 1 << kUnitShift, "a unit is one step of every wave");
// Waves per SIMD, and the workgroups of a launch: as many as are resident then.  The registers of a step's loads,
// operands and sums decide: D = 64 fits three without spilling (16 sequences of 16 k tokens, 8 cache heads: 45 us, 48
// with two waves), 128 and 256 two (82 and 153 us; 84 and 348 with three and the spills, 98 and 184 with one).
constexpr int waves_of(int D, int NR) { return D == 64 && NR == 1 ? 3 : 2; }
constexpr int64_t kCUs = 256;

// Probabilities are held times 2^13 (with a scale, up to twice its power of two, below fp16's 65504), so that ones
// down to 2^-27 of the largest keep all their bits and ones below 2^-38 of it are lost.
constexpr float kPBits = 13.0f;
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

// Units of every tile of a sequence: enough for the tile that sees the most tokens.
template <int TR>
__device__ __forceinline__ int units_of(const AttnArgs& a, const Seq& s) {
  int64_t span = s.len < 0 ? 0 : s.len;
  if (a.window) {
    const int64_t tokens = (TR + a.group - 1) / a.group + 1;   // tokens a tile's rows can belong to
    const int64_t w = (int64_t)a.window + tokens + kStep;
    if (w < span) span = w;
  }
  const int shift = kUnitShift + a.ushift;
  const int u = (int)((span + (int64_t(1) << shift) - 1) >> shift);
  return u > 0 ? u : 1;
}
template <int TR>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Seq& s) {
  const int64_t rows = (int64_t)s.n * a.group;
  return rows > a.few ? 0 : (int)((rows + TR - 1) / TR);   // many rows: the other kernel's
}

// Units 0 .. total - 1 in W <= total ranges as even as can be, the first total % W of them one longer.
struct Ranges {
  uint32_t len, more;
  __device__ __forceinline__ Ranges(uint32_t total, uint32_t W) : len(total / W), more(total - total / W * W) {}
  __device__ __forceinline__ uint32_t first(uint32_t w) const { return w * len + min(w, more); }
  __device__ __forceinline__ uint32_t of(uint32_t unit) const {   // the range that holds a unit
    const uint32_t border = more * (len + 1);
    return unit < border ? unit / (len + 1) : more + (unit - border) / len;
  }
};

// A step's four page entries (16 tokens each) as scalars.
struct Pages {
  int p[4];
};
__device__ __forceinline__ Pages pages_of(int pid) {
  return Pages{{__builtin_amdgcn_readlane(pid, 0), __builtin_amdgcn_readlane(pid, 16), __builtin_amdgcn_readlane(pid, 32),
                __builtin_amdgcn_readlane(pid, 48)}};
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
__global__ __launch_bounds__(AT, waves_of(D, NR)) void k_kv_attn(AttnArgs a, CodePlanes cp) {
  constexpr int TR = 16 * NR, B = D / NB, KK = D / 32, UN = D / 16;
  constexpr int RB = D / 2;                // bytes of a cache row
  constexpr int CH = RB / 16;              // 16-byte chunks of a row
  constexpr int LB = RB + 16;              // a row in LDS: 16 rows' pieces of one column lie in different banks
  constexpr int kVBytes = kStep * LB;      // a wave's value codes
  constexpr int kStepBytes = kVBytes + NB * kStep * 6;   // value codes, fp32 key scales, fp16 value scales
  constexpr int LDO = D + 4;               // floats of a row of sums
  constexpr int kWaveBytes = kStepBytes > TR * LDO * 4 ? kStepBytes : TR * LDO * 4;
  __shared__ __attribute__((aligned(16))) unsigned char smem[AW * kWaveBytes];
  __shared__ uint32_t pair[256];
  __shared__ float ml[AW][2][TR];          // maxima (log2) and sums of each wave's rows
  __shared__ int vexp[AW][NB];             // units of its output sums
  __shared__ SeqTable<AT> seqs;
  __shared__ int found;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  unsigned char* const vbuf = smem + wave * kWaveBytes;
  float* const kscale = reinterpret_cast<float*>(vbuf + kVBytes);
  uint16_t* const vscale = reinterpret_cast<uint16_t*>(kscale + NB * kStep);
  {
    const u32x4 w = decode_planes(cp, threadIdx.x);   // elements 0 and 4: the low and the high nibble of byte 0
    pair[threadIdx.x] = (w[0] & 0xFFFFu) | w[2] << 16;
  }
  const float kmul = a.scale * kLog2e * cp.inv;

  // this workgroup's range of units
  auto count = [&](const Seq& s) -> int { return tiles_of<TR>(a, s) * units_of<TR>(a, s) * a.c.heads; };
  scan_seqs(a.b, 0, 0, seqs, count);
  int c0 = 0;
  int total = seqs.pre[AT];
  for (int c = AT; c < a.b.batch; c += AT) {   // more than 256 sequences: the total first, then back to the front
    __syncthreads();
    scan_seqs(a.b, c, total, seqs, count);
    total = seqs.pre[AT];
    c0 = c;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  int w = blockIdx.x;
  if (blockIdx.x == 0) check_batch_entries<AT>(a.b);
  // workgroups are dealt out to the 8 XCDs in turn: neighbouring ranges, which can share a sequence's tokens, go to one
  const int grid = gridDim.x;
  if (total >= grid && (grid & 7) == 0) w = (w & 7) * (grid >> 3) + (w >> 3);
  if (threadIdx.x == 0) a.meta[w * kMetaInts] = -1;   // (of the range: another workgroup's would come too late)
  const int W = min(total, grid);
  if (w >= W) return;
  const Ranges ranges(total, W);
  const int lo = ranges.first(w), hi = ranges.first(w + 1);
  if (c0 != 0) {
    int base = 0;
    for (c0 = 0;; c0 += AT) {
      __syncthreads();
      scan_seqs(a.b, c0, base, seqs, count);
      if (seqs.pre[AT] > lo) break;
      base = seqs.pre[AT];
    }
  }

  int seq_first = 0, seq_end = 0, bi = 0, units = 1, tiles = 1;   // the sequence at hand: its units, as numbered here
  Seq s{};
  for (int cur = lo; cur < hi;) {
    if (cur >= seq_end) {
      // the sequence that holds unit `cur`
      while (seqs.pre[AT] <= cur) {
        const int base = seqs.pre[AT];
        __syncthreads();
        c0 += AT;
        scan_seqs(a.b, c0, base, seqs, count);
      }
      const int tx = opaque(threadIdx.x);
      if (seqs.pre[tx] <= cur && cur < seqs.pre[tx + 1]) found = tx;
      __syncthreads();
      bi = __builtin_amdgcn_readfirstlane(found);
      s = seqs.seq(bi);
      units = units_of<TR>(a, s);
      tiles = tiles_of<TR>(a, s);
      seq_first = __builtin_amdgcn_readfirstlane(seqs.pre[bi]);
      seq_end = __builtin_amdgcn_readfirstlane(seqs.pre[bi + 1]);
    }
    const uint32_t rem = cur - seq_first;
    // (head, tile) of the sequence; most sequences of a decoding step have one tile, short ones one unit
    const int tile_id = units == 1 ? (int)rem : __builtin_amdgcn_readfirstlane(rem / (uint32_t)units);
    const int u0 = (int)rem - tile_id * units, u1 = min(u0 + hi - cur, units);
    const int h = tiles == 1 ? tile_id : __builtin_amdgcn_readfirstlane((uint32_t)tile_id / (uint32_t)tiles), rt = tile_id - h * tiles;
    const Tile t = tile_of<TR>(a, s, c0 + bi, h, rt);
    const bool whole = u0 == 0 && u1 == units;

    // rows of this lane: row r * 16 + l16 of the tile
    u32x4 qf[NR][KK];
    int32_t r_lo[NR], r_hi[NR];               // tokens it sees
    float rs[NR];                             // logit (in log2) of one unit of its products
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int rr = r * 16 + l16;
      const bool ok = rr < t.nval;
      const int rho = t.rho0 + (ok ? rr : 0);
      const int i = div_group(a, rho), qh = t.h * a.group + (rho - i * a.group);
      const int len = s.len < 0 ? 0 : s.len;
      const int p = len - s.n + i;
      r_hi[r] = !ok ? 0 : a.causal ? p + 1 : len;
      r_lo[r] = a.window ? p + 1 - a.window : 0;
      const uint16_t* qp = a.q.data + (s.row0 + i) * a.q.rs + qh * a.q.hs;
      uint32_t mag = 0;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        qf[r][k] = *reinterpret_cast<const u32x4*>(qp + 32 * k + 8 * g);
        if (!ok) qf[r][k] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < 4; ++x) mag = max(mag, max(qf[r][k][x] & 0x7FFFu, (qf[r][k][x] >> 16) & 0x7FFFu));
      }
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 16, 64));
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 32, 64));
      const int e = exponent_of(mag);
      const float f = row_unit(mag, e);
      // not 0, which a masked token's -inf would turn into NaN, and finite, so that products of 0 stay 0
      rs[r] = fminf(fmaxf(kmul * pow2(e), 0x1p-149f), 0x1.fffffep127f);
      // in the order that pairs decode to: 0, 4, 1, 5, 2, 6, 3, 7
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        const u32x4 w = qf[r][k];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          qf[r][k][2 * x] = pack_f16x2(__uint_as_float(w[x] << 16) * f, __uint_as_float(w[x + 2] << 16) * f);
          qf[r][k][2 * x + 1] =
              pack_f16x2(__uint_as_float(w[x] & 0xFFFF0000u) * f, __uint_as_float(w[x + 2] & 0xFFFF0000u) * f);
        }
      }
    }

    f32x4 O[NR][UN];
    float m[NR], l[NR];                       // running maximum (in products' units) and this lane's part of the sum
    int ve[NB];                               // O is in units of 2^ve of each block
#pragma unroll
    for (int b = 0; b < NB; ++b) ve[b] = -100;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = neg_inf();
      l[r] = 0.0f;
#pragma unroll
      for (int u = 0; u < UN; ++u) O[r][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int steps = t.hi > t.base ? (t.hi - t.base + kStep - 1) / kStep : 0;
    const int st_end = min((u1 << a.ushift) * AW, steps);

    // the table's entry for this lane group's 16 tokens of a step (its first entry past the last token): loaded two steps
    // ahead, and looked at only when it is used, so that no wait for it waits for the loads behind it
    const int32_t* const table = a.b.table + (int64_t)t.b * a.b.max_pages;
    const int pshift = a.c.pshift;
    auto page_at = [&](int st) -> int {
      const int tok = t.base + st * kStep + 16 * g;
      return table[tok < t.hi ? tok >> pshift : 0];
    };
    const uint32_t pages = (uint32_t)a.c.pages;
    // this head's rows of page 0, and the row of a token from there (of page 0 where the entry is wrong: read, not used)
    const int64_t head_row = (int64_t)t.h << a.c.pshift;
    const uint8_t* const kc = a.c.kc + head_row * RB;
    const uint8_t* const vc = a.c.vc + head_row * RB;
    const uint16_t* const ksc = a.c.ks + head_row * NB;
    const uint16_t* const vsc = a.c.vs + head_row * NB;
    const uint32_t page_rows = (uint32_t)a.c.heads << a.c.pshift, slot_mask = (1u << a.c.pshift) - 1;
    auto row_of = [&](int pid, int tok) -> uint64_t {
      return (uint64_t)((uint32_t)pid < pages ? (uint32_t)pid : 0u) * page_rows + ((uint32_t)tok & slot_mask);
    };
    auto load_k = [&](StepLoads<D, NB>& L, int st, int pid, Pages pg) {
      // row 4a + i of token tile tt is token 16a + 4tt + i: 16 tokens aligned to 16 lie in one page
      const int ka = l16 >> 2;
      int pk = pg.p[0];
      if (ka == 1) pk = pg.p[1];
      if (ka == 2) pk = pg.p[2];
      if (ka == 3) pk = pg.p[3];
      const uint8_t* p = kc + row_of(pk, t.base + st * kStep + 16 * ka + (l16 & 3)) * RB;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        if constexpr (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(p + 4 * tt * RB + 8 * g);
          L.k[tt][0] = u32x4{x.x, x.y, 0, 0};
        } else {
#pragma unroll
          for (int k = 0; k < StepLoads<D, NB>::KW; ++k)
            L.k[tt][k] = *reinterpret_cast<const u32x4*>(p + 4 * tt * RB + 64 * k + 16 * g);
        }
      }
    };
    auto load_v = [&](StepLoads<D, NB>& L, int st, int pid, Pages pg) {
      const int tok0 = t.base + st * kStep;
      // CH lanes per token: a load takes 32 (D = 64), 16 or 8 (D = 256) tokens, so one or half of a page's 16, whose
      // base is the same in all lanes, or two
      const uint32_t own = 16 * lane;
#pragma unroll
      for (int i = 0; i < StepLoads<D, NB>::VL; ++i) {
        const uint8_t* p;
        if constexpr (D == 64) {
          const uint64_t r0 = row_of(pg.p[2 * i], tok0 + 32 * i), r1 = row_of(pg.p[2 * i + 1], tok0 + 32 * i + 16);
          p = vc + (lane < 32 ? r0 : r1) * RB + (own & 511u);
        } else {
          constexpr int T = 64 / CH;
          p = vc + row_of(pg.p[i * T / 16], tok0 + i * T) * RB + own;
        }
        L.v[i] = *reinterpret_cast<const u32x4*>(p);
      }
      // scales of token `lane`
      const uint64_t row = row_of(pid, tok0 + lane) * NB;
      if constexpr (NB == 1) {
        L.ks[0] = ksc[row];
        L.vs[0] = vsc[row];
      } else {
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
          L.ks[k] = reinterpret_cast<const uint32_t*>(ksc + row)[k];
          L.vs[k] = reinterpret_cast<const uint32_t*>(vsc + row)[k];
        }
      }
    };

    int st = (u0 << a.ushift) * AW + wave;
    StepLoads<D, NB> L;
    int pid = page_at(st), pid_next = page_at(st + AW), pid_after;
    if (st < st_end) {
      const Pages pg = pages_of(pid);
      load_v(L, st, pid, pg);
      load_k(L, st, pid, pg);
      // tokens at the front that no row sees (lane 0 has the tile's first row; held ready in the tile, it took 6 registers more)
      const int skip = st == 0 && a.window ? __builtin_amdgcn_readfirstlane(r_lo[0]) - t.base : 0;
      if (skip > 0 && lane < skip) {   // neither their scales nor their pages' entries count
        pid = 0;
#pragma unroll
        for (int x = 0; x < (NB + 1) / 2; ++x) L.ks[x] = L.vs[x] = 0;
      }
    }
    // this lane's token row of the transposing reads: row n of 16 is token 8 (n / 8) + (n % 8) / 2 + 4 (n % 2), so that a
    // dword of what comes back decodes in token order
    unsigned char* const vplanes = vbuf + ((lane & ~7) + ((lane & 7) >> 1) + 4 * (lane & 1)) * LB;
    for (; st < st_end; st += AW) {
      const int tok0 = t.base + st * kStep;
      pid_after = page_at(st + 2 * AW);
      // value codes and scales to LDS, this wave's own part of it (a wave's LDS accesses stay in order)
#pragma unroll
      for (int i = 0; i < StepLoads<D, NB>::VL; ++i) {
        const int tk = i * (64 / CH) + lane / CH, c = lane & (CH - 1);
        *reinterpret_cast<u32x4*>(vbuf + tk * LB + 16 * c) = L.v[i];
      }
      const bool none = tok0 + lane >= t.hi;   // no token: scale 0; no page: NaN
      const bool wrong = (uint32_t)pid >= pages && !none;
      if (__any(wrong) && lane == 0) raise_fault(a.b, kFaultPage);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t kw = b & 1 ? L.ks[b / 2] >> 16 : L.ks[b / 2] & 0xFFFFu;
        uint32_t vw = b & 1 ? L.vs[b / 2] >> 16 : L.vs[b / 2] & 0xFFFFu;
        if (wrong) kw = vw = kBf16NaN;
        if (none) kw = vw = 0;
        kscale[b * kStep + lane] = bf16_to_f32(kw);
        const uint32_t mag = vw & 0x7FFFu, held = (uint32_t)(ve[b] + 128) << 7;   // magnitudes below `held` fit
        if (__any(mag >= held && mag < 0x7F80u)) {
          const int e = exponent_of(wave_max(mag < 0x7F80u ? mag : 0u));
          const float f = pow2(max(ve[b] - e, -126));
          ve[b] = e;
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int u = b * (B / 16); u < (b + 1) * (B / 16); ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) O[r][u][i] *= f;
        }
        vscale[b * kStep + lane] = (uint16_t)(pack_f16x2(bf16_to_f32(vw) * pow2(-ve[b]), 0.0f) & 0xFFFFu);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

      // S^T: rows = tokens, columns = rows of q, in stages of two products (64 elements of a token tile).  The lookups
      // of a stage are issued one stage ahead of its products (left to itself the compiler waits for each pair's own)
      constexpr int ST = KK / 2, SB = B == 32 ? 2 : 1;   // stages of a token tile, blocks that a stage touches
      f32x4 S[NR][4];
      u32x4 kf[2][2];
      f32x4 sk[2][SB];
      auto fetch = [&](int i) {
        const int tt = i / ST, h2 = i % ST;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int k = 2 * h2 + x;
          kf[i & 1][x] = decode_pairs(pair, L.k[tt][k / 4][k % 4]);
        }
#pragma unroll
        for (int x = 0; x < SB; ++x)
          sk[i & 1][x] =
              *reinterpret_cast<const f32x4*>(kscale + (2 * h2 + x) * 32 / B * kStep + 16 * g + 4 * tt);
      };
      fetch(0);
      f32x4 acc[NR];
#pragma unroll
      for (int i = 0; i < 4 * ST; ++i) {
        const int tt = i / ST, h2 = i % ST;
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < 4 * ST) fetch(i + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int k = 2 * h2 + x;
          const bool first = 32 * k % B == 0, last = 32 * (k + 1) % B == 0;   // of its block
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (first) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
            acc[r] = mfma16h(kf[i & 1][x], qf[r][k], acc[r]);
            if (last) {
              const f32x4 f = sk[i & 1][SB == 2 ? x : 0];
#pragma unroll
              for (int j = 0; j < 4; ++j) S[r][tt][j] = k < B / 32 ? acc[r][j] * f[j] : __builtin_fmaf(acc[r][j], f[j], S[r][tt][j]);
            }
          }
        }
        // the scaled products are formed here: left alone, the compiler moves this into the branches below and holds
        // the products of all blocks and all scales until then, 50 registers more
        if (h2 == ST - 1) {
#pragma unroll
          for (int r = 0; r < NR; ++r) asm volatile("" : "+v"(S[r][tt]));
        }
      }
      pid = pid_next;
      pid_next = pid_after;
      // the next step's loads run under the rest of this one
      if (st + AW < st_end) {
        const Pages pg = pages_of(pid);
        load_v(L, st + AW, pid, pg);
        load_k(L, st + AW, pid, pg);
      }

      // value codes, transposed, and scales: the first ones are read now and used after the softmax, the others two
      // column tiles and one block ahead
      typedef int v2i __attribute__((ext_vector_type(2)));
      v2i vw[UN];
      u32x4 sv[NB][2];
      auto read_v = [&](int u) {
        vw[u] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) v2i*)(vplanes + 8 * u));
      };
      auto read_sv = [&](int b) {
#pragma unroll
        for (int x = 0; x < 2; ++x) sv[b][x] = *reinterpret_cast<const u32x4*>(vscale + b * kStep + 16 * g + 8 * x);
      };
      read_sv(0);
      read_v(0);
      read_v(1);
      __builtin_amdgcn_sched_barrier(0);

      // tokens 16g + 4tt + i that the lane's row does not see (only in steps at an end of what some row sees)
      const bool edge = tok0 < t.lo_max || tok0 + kStep > t.hi_min;
      uint32_t vis[NR];   // bit 4tt + i: the lane's row sees that token (used at an edge only)
      if (edge) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int t0 = tok0 + 16 * g;
          const int lo = min(max(r_lo[r] - t0, 0), 16), hi = min(max(r_hi[r] - t0, 0), 16);
          vis[r] = (1u << hi) - (1u << min(lo, hi));
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t m = __builtin_amdgcn_sbfe((int)vis[r], 4 * tt + i, 1);
              S[r][tt][i] = __uint_as_float((__float_as_uint(S[r][tt][i]) & m) | (0xFF800000u & ~m));
            }
        }
      }
      uint32_t pp[NR][4][2];   // probabilities of tokens 16g + 4tt + 0, 1 and 2, 3 in fp16
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
          const float alpha = __builtin_amdgcn_exp2f((m[r] - mu) * rs[r]);
          l[r] *= alpha;
#pragma unroll
          for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[r][u][i] *= alpha;
        }
        m[r] = mx;
        const float off = kPBits - mu * rs[r];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r][tt][2 * i], rs[r], off));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r][tt][2 * i + 1], rs[r], off));
            l[r] += p0;
            l[r] += p1;
            pp[r][tt][i] = pack_f16x2(p0, p1);
          }
      }

      // O^T += V^T (P s)^T, one block of elements at a time
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 pf[NR][2];   // tokens 16g + 0..7 and + 8..15
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            pf[r][x / 4][x % 4] = mul_f16x2(pp[r][x / 2][x % 2], sv[b][x / 4][x % 4]);
        if (edge) {
          // a scale can be NaN: what the row does not see is left out, not multiplied by zero
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            uint32_t see = vis[r];
            asm volatile("" : "+v"(see));   // formed anew for each block: the masks kept from one to the next are 24 registers
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const uint32_t m0 = __builtin_amdgcn_sbfe((int)see, 2 * x, 1), m1 = __builtin_amdgcn_sbfe((int)see, 2 * x + 1, 1);
              pf[r][x / 4][x % 4] &= (m0 & 0xFFFFu) | (m1 & 0xFFFF0000u);
            }
          }
        }
#pragma unroll
        for (int u = b * (B / 16); u < (b + 1) * (B / 16); ++u) {
          __builtin_amdgcn_sched_barrier(0);
          if (u + 2 < UN) read_v(u + 2);
          if (b + 1 < NB && u + 1 == (b + 1) * (B / 16)) read_sv(b + 1);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const u32x4 v = decode_planes(cp, (uint32_t)vw[u][x]);
#pragma unroll
            for (int r = 0; r < NR; ++r) O[r][u] = mfma16h(v, pf[r][x], O[r][u]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

    // The four waves' sums: each leaves its own in LDS, then all threads add them up, a thread 8 neighbouring columns
    // of a row.  (Added two by two, and written by one wave, this took 4200 cycles of the 15000 of a tile with one step.)
    {
      const int el = opaque(lane), e16 = el & 15, eg = el >> 4;
      float* const mg = reinterpret_cast<float*>(vbuf);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        l[r] = group_sum(l[r]);
        if (eg == 0) {
          ml[wave][0][r * 16 + e16] = m[r] * rs[r];
          ml[wave][1][r * 16 + e16] = l[r];
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) *reinterpret_cast<f32x4*>(mg + (r * 16 + e16) * LDO + u * 16 + 4 * eg) = O[r][u];
      }
      if (el == 0)
#pragma unroll
        for (int b = 0; b < NB; ++b) vexp[wave][b] = ve[b];
    }
    __syncthreads();
    constexpr int CT = D / 8;   // threads of a row
#pragma unroll
    for (int i = 0; i < (TR * CT + AT - 1) / AT; ++i) {
      const int item = opaque(threadIdx.x) + i * AT, rr = item / CT, c = item % CT;
      if (rr >= t.nval) continue;
      float mk[AW], mt = neg_inf(), lt = 0.0f;
#pragma unroll
      for (int k = 0; k < AW; ++k) mt = fmaxf(mt, mk[k] = ml[k][0][rr]);
      const float mu = mt == neg_inf() ? 0.0f : mt;
      f32x4 o[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < AW; ++k) {
        const float f = __builtin_amdgcn_exp2f(mk[k] - mu) * pow2(-(int)kPBits);
        const float fo = f * pow2(vexp[k][8 * c / B]) * cp.inv;
        lt = __builtin_fmaf(ml[k][1][rr], f, lt);
        const f32x4* const p = reinterpret_cast<const f32x4*>(smem + k * kWaveBytes) + (rr * LDO + 8 * c) / 4;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const f32x4 w = p[x];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[x][j] = __builtin_fmaf(w[j], fo, o[x][j]);
        }
      }
      if (whole) {
        const int rho = t.rho0 + rr, row = div_group(a, rho), qh = t.h * a.group + (rho - row * a.group);
        float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
        if (s.len < 0) inv = __builtin_nanf("");
        // the columns hold elements 0, 4, 1, 5, 2, 6, 3, 7 of their eight
        *reinterpret_cast<uint4*>(a.o.data + (s.row0 + row) * a.o.rs + qh * a.o.hs + 8 * c) =
            make_uint4(pack_bf16x2(o[0][0] * inv, o[0][2] * inv), pack_bf16x2(o[1][0] * inv, o[1][2] * inv),
                       pack_bf16x2(o[0][1] * inv, o[0][3] * inv), pack_bf16x2(o[1][1] * inv, o[1][3] * inv));
        if (a.lse && c == 0)
          a.lse[(s.row0 + row) * a.q.n + qh] =
              s.len < 0 ? __builtin_nanf("") : lt == 0.0f ? neg_inf() : (mt + __builtin_amdgcn_logf(lt)) * kLn2;
      } else {
        // slot 0: the range's first tile, begun in an earlier range; slot 1: its last, ending in a later one
        float* d = a.part + (2 * (int64_t)w + (u0 == 0 ? 1 : 0)) * (TR * (D + 2));
#pragma unroll
        for (int x = 0; x < 2; ++x) *reinterpret_cast<f32x4*>(d + rr * D + 8 * c + 4 * x) = o[x];
        if (c == 0) {
          d[TR * D + rr] = mt;
          d[TR * D + TR + rr] = lt;
        }
      }
    }
    if (!whole && u0 != 0 && u1 == units && threadIdx.x == 0) {
      // this range ends the tile: the join of its partial sums is noted here
      int32_t* mt_ = a.meta + w * kMetaInts;
      mt_[0] = (int32_t)ranges.of(cur - u0);   // the range that holds its first unit
      mt_[1] = (int32_t)s.row0;
      mt_[2] = t.rho0;
      mt_[3] = t.nval;
      mt_[4] = t.h;
    }
    cur += u1 - u0;
    __syncthreads();
  }
}

// Adds the partial sums of a tile that was cut: workgroup (w, y) the tile that ends in range w, if any, wave v row
// 4y + v.  The parts lie in slot 1 of the first range and slot 0 of the others.
template <int D, int TR>
__global__ __launch_bounds__(256) void k_kv_attn_join(AttnArgs a) {
  constexpr int64_t P = TR * (D + 2);
  const int w = blockIdx.x;
  const int32_t* mt = a.meta + w * kMetaInts;
  const int w0 = mt[0], rr = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w0 < 0 || rr >= mt[3]) return;
  join_row<D>(
      a, w - w0 + 1, TR, rr, mt, [&](int k) { return a.part + (2 * (int64_t)(w0 + k) + (k == 0)) * P; },
      // position d of a partial row: row d % 16 of column tile d / 16
      [](int d) { return (d & ~15) + (d & 8) + ((d & 7) >> 1) + 4 * (d & 1); });
}

// Byte tables of v_perm_b32 lookups by the code and by the code ^ 8 whose xor is table[code] (see CodePlanes).
void xor_tables(const uint8_t (&table)[16], uint32_t (&out)[4]) {
  uint8_t t[16];
  for (int i = 0; i < 16; ++i) t[i] = table[i];
  // low entry c (0..7) is xored with what the high table's lookup gives for selector c + 8, high entry c with what the
  // low table's gives; the signs that selectors 8..11 copy are those of entries finished before
  auto sign = [&](int i) { return (uint8_t)(t[i] & 0x80 ? 0xFF : 0); };
  for (int c = 5; c < 8; ++c) t[c] ^= 0xFF, t[8 + c] ^= 0xFF;   // selectors 13..15; 12 gives 0
  t[3] ^= sign(8 + 7), t[8 + 3] ^= sign(7);                     // selector 11: byte 7
  t[1] ^= sign(8 + 3), t[8 + 1] ^= sign(3);                     // selector 9: byte 3
  t[2] ^= sign(8 + 5), t[8 + 2] ^= sign(5);                     // selector 10: byte 5
  t[0] ^= sign(8 + 1), t[8 + 0] ^= sign(1);                     // selector 8: byte 1
  for (int i = 0; i < 4; ++i)
    out[i] = t[4 * i] | (uint32_t)t[4 * i + 1] << 8 | (uint32_t)t[4 * i + 2] << 16 | (uint32_t)t[4 * i + 3] << 24;
}

}  // namespace

CodePlanes code_planes(int cb) {
  CodePlanes p{};
  const float c = cb == QLORA_CODEBOOK_FP4 ? 6.0f : cb == QLORA_CODEBOOK_INT4 ? 7.0f : 1.0f;
  const float* lv = codebook_levels_host(cb);
  uint8_t lo[16], hi[16];
  for (int i = 0; i < 16; ++i) {
    const uint16_t h = __builtin_bit_cast(uint16_t, (_Float16)(lv[i] * c));
    lo[i] = (uint8_t)(h & 0xFF);
    hi[i] = (uint8_t)(h >> 8);
  }
  xor_tables(lo, p.lo);
  xor_tables(hi, p.hi);
  p.inv = 1.0f / c;
  return p;
}

// Sequences with at most this many rows per cache head go to the kernel of this file, those with more to the one for
// many rows.  The host knows the rows and the sequences of a call, not which has how many.  With one sequence it leaves all
// to one kernel; with more, to the first (which is right for any) where the mean is low and no sequence can have more than
// kAlone rows, each of the others having one; otherwise it launches both.
// This kernel and the other one, 16 sequences of 4096 tokens, 32 cache heads: D = 64, 64 rows 101 and 221 us, 128 rows 181 and 219,
// 160 rows 225 and 239; D = 128, 64 rows 176 and 242, 96 rows 248 and 243, 128 rows 329 and 256; D = 256, 64 rows 516 and
// 555, 96 rows 754 and 561.  With one sequence it depends on how long it is, which the host does not know: 8 heads of 64,
// 2048 tokens, 64 rows 12.5 and 17.6 us, 128 rows 16.4 and 19.5; 32768 tokens, 49 and 41, 50 and 43; heads of 128 with 64 rows,
// 15.9 and 20.2, 51 and 44; of 256, 22 and 33, 73 and 86.  So it goes by the same numbers of rows.
constexpr int few_rows(int D) { return D == 64 ? 128 : 64; }
// 32 sequences of 4096, 8 cache heads of 128, one with 520 rows, the others with 4: 76 us by the first kernel, 91 by both; 64 of
// 2000 and one of 8192 with 2048 rows 212 and 155; 300 of 1000 and one of 4096 with 16384 rows 809 and 343; 64 of 4096
// with 32 rows each, where the second finds nothing to do, 100 and 104.
constexpr int64_t kAlone = 1024;

// A workspace made for the largest call serves smaller ones, which may be cut into parts where the large one is not: every
// size at its most for up to these rows, sequences and tokens, so that it grows with each of them.
static void size_workspace(AttnPlan& p, int64_t rows_h, int64_t nseq, int64_t kv_heads, int64_t max_len, int D) {
  const int64_t units = (max_len >> kUnitShift) + 1;
  // ranges of the kernel for few rows, with tiles of 16 rows and, where a call may have those, of 32
  const int wide = D < 256 && rows_h > 16 && nseq * kv_heads * units >= 2 * kCUs * waves_of(D, 2) ? 2 : 1;
  for (int nr = 1; nr <= wide; ++nr) {
    const int tile = 16 * nr;
    const int64_t tiles = ((rows_h + tile - 1) / tile + nseq) * kv_heads;
    const size_t wgs = (size_t)std::min(tiles * units, kCUs * waves_of(D, nr));
    p.part_floats = std::max(p.part_floats, wgs * 2 * tile * (D + 2));
    p.meta_ints = std::max(p.meta_ints, wgs * kMetaInts);
  }
  // parts of the one for many rows, which runs before the other and leaves it the same memory
  if (rows_h > few_rows(D) && max_len >= 2 * split_tokens_of(D, true)) {
    p.part_floats = std::max(p.part_floats, (size_t)kSplitWgs * (many_threads(D) / 2) * (D + 2));
    p.meta_ints = std::max(p.meta_ints, (size_t)(1 + kSplitWgs / 2) * kMetaInts);
  }
}

AttnPlan attn_plan(int64_t rows, int32_t q_heads, int32_t kv_heads, int32_t batch, int64_t max_len, int D) {
  AttnPlan p{};
  const int64_t group = q_heads / kv_heads, rows_h = rows * group, nseq = batch > 1 ? batch : 1;
  const int few = few_rows(D);
  if (rows_h <= few * nseq && rows_h - (nseq - 1) * group <= kAlone) p.few = INT32_MAX;
  else p.few = nseq == 1 ? 0 : few;
  // Tiles of 32 rows decode a token once for twice the rows, but make half the units: they are taken where sequences have more
  // than 16 rows and every workgroup still has two units.  8 cache heads of 128, 32 and 64 rows of each sequence: 16
  // sequences of 4096 40 and 55 us (43 and 67 with tiles of 16), 4 of them 30 and 31 (23 and 28), one 21 and 22 (18 and
  // 22).  Where the mean is that of a prompt, the sequences left for this kernel are taken to have single tokens (64 of them
  // with 4096 tokens and 8 query heads per cache head beside a prompt: 69 us, 86 with tiles of 32).  D = 256 has no
  // registers for it.
  const int64_t units32 = nseq * kv_heads * ((max_len >> kUnitShift) + 1);
  const int nr = D < 256 && rows_h > 16 * nseq && rows_h <= few * nseq && units32 >= 2 * kCUs * waves_of(D, 2) ? 2 : 1;
  p.tile = 16 * nr;
  if (p.few > 0) {
    const int64_t tiles = ((rows_h + p.tile - 1) / p.tile + nseq) * kv_heads;
    // units so large that their number stays below 2^30
    while (tiles * ((max_len >> (kUnitShift + p.ushift)) + 1) >= int64_t(1) << 30 && p.ushift < 22) ++p.ushift;
    const int64_t units = (max_len >> (kUnitShift + p.ushift)) + 1;
    p.wgs = kCUs * waves_of(D, nr);
    if (tiles * units < p.wgs) p.wgs = tiles * units;
    p.part_floats = (size_t)p.wgs * 2 * p.tile * (D + 2);
    p.meta_ints = (size_t)p.wgs * kMetaInts;
  }
  if (p.few != INT32_MAX) {
    const int tr = many_threads(D) / 2;
    const int64_t most = rows_h / ((int64_t)p.few + 1) + 1;   // sequences that can have more than `few` rows
    p.many_wgs = (rows_h / tr + (most < nseq ? most : nseq)) * kv_heads;
    p.sparse = p.many_wgs * tr * 3 >= 4 * rows_h * kv_heads;
    const int64_t least = (rows_h - p.few * nseq) / tr * kv_heads;   // tiles that there are, if all rows are a sequence's
    const int tokens = split_tokens_of(D, p.sparse);
    if (max_len >= 2 * tokens && least <= kSplitWgs / 2) {
      p.many_split = p.many_wgs < kSplitWgs / 2 ? p.many_wgs : kSplitWgs / 2;
      if (p.many_wgs < kSplitWgs) p.many_wgs = kSplitWgs;
      p.split_tokens = tokens;
      p.part_floats = std::max(p.part_floats, (size_t)kSplitWgs * tr * (D + 2));
      p.meta_ints = std::max(p.meta_ints, (size_t)(1 + p.many_split) * kMetaInts);
    }
  }
  size_workspace(p, rows_h, nseq, kv_heads, max_len, D);
  return p;
}

template <int D, int NB, int NR>
static hipError_t launch_attn(const AttnArgs& a0, const AttnPlan& pl, hipStream_t s) {
  AttnArgs a = a0;
  a.ushift = pl.ushift;
  a.few = pl.few;
  {
    ProfScope ps("k_kv_attn", s);
    hipLaunchKernelGGL((k_kv_attn<D, NB, NR>), dim3((unsigned)pl.wgs), dim3(AT), 0, s, a, code_planes(a.c.cb));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ProfScope ps("k_kv_attn_join", s);
  hipLaunchKernelGGL((k_kv_attn_join<D, 16 * NR>), dim3((unsigned)pl.wgs, 4 * NR), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int D, int NB>
static hipError_t launch_tile(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  if constexpr (D < 256) {
    if (pl.tile == 32) return launch_attn<D, NB, 2>(a, pl, s);
  }
  return launch_attn<D, NB, 1>(a, pl, s);
}

static hipError_t launch_few(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s) {
  const int nb = D / block;
  if (D == 64) return nb == 1 ? launch_tile<64, 1>(a, pl, s) : launch_tile<64, 2>(a, pl, s);
  if (D == 128)
    return nb == 1 ? launch_tile<128, 1>(a, pl, s) : nb == 2 ? launch_tile<128, 2>(a, pl, s) : launch_tile<128, 4>(a, pl, s);
  return nb == 2 ? launch_tile<256, 2>(a, pl, s) : nb == 4 ? launch_tile<256, 4>(a, pl, s) : launch_tile<256, 8>(a, pl, s);
}

hipError_t launch_kv_attn(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s) {
  if (pl.few != INT32_MAX) {
    AttnArgs m = a;
    m.few = pl.few;
    const hipError_t e = launch_kv_attn_many(m, pl, D, block, s);
    if (e != hipSuccess || pl.few == 0) return e;
  }
  return launch_few(a, pl, D, block, s);
}

}  // namespace qlora
