// Attention over the 4-bit cache for many rows of a sequence (prompts): tiles of 32 rows per wave, all waves of a
// workgroup on the same tokens.
//
// The same sums as kv_attn.hip; with this many rows the decoding is shared and the matrix products rule.  64 tokens
// at a time are decoded by the whole workgroup into LDS as fp16 (level * scale, each tile brought to about 1 by a power of
// two: the keys' goes into the logits' factor, the values' is a running exponent like the running maximum), one tile
// ahead of the products, from codes loaded another tile ahead.  S^T = K Q^T and O^T = V^T P^T on 32x32x16 MFMA:
// a lane holds 32 logits of one row, so the softmax needs one exchange of two lanes, and P^T is the next
// product's operand as it stands (its token order is the accumulator's; the values are read to match, transposed by
// ds_read_b64_tr_b16).  The maximum is moved only when one grows by more than 2^6, so that the sums are rarely rescaled.
//
// Per 64 tokens and SIMD (D = 128, two waves) the matrix cores take 2048 cycles, about 400 VALU instructions of each
// wave 3700 with the exponentials' 16 each, LDS 2250: of 5800 in all.  Bound by the issue of VALU instructions, which
// the matrix products of the other wave overlap in part.
// Measured: 16384 rows of one sequence, 32 query on 8 cache heads of 128, causal, 2.49 to 2.6 ms = 850 to 884 TFLOP/s
// (a square library product of 8192 reaches 1190); 4 x 4096 rows 0.70 to 0.78 ms, 705 to 780.  Heads of 64: 1.75 ms, 627, and
// 0.51 ms, 545 (twice the exponentials and decoding per product).  Heads of 256: 8.5 ms, 516, and 2.36 ms, 466 (4 waves to a CU
// with 512 registers each: nothing overlaps a wave's waits).  A workgroup's start, its first tile and its end cost 12 to 15 us,
// which is what short sequences pay: 1024 rows 46 us.
//
// One workgroup per tile of a sequence.  Each finds all tiles of the call from the device's lengths; where there are no more
// than half as many as CUs, the tokens of every tile are cut into parts for all of them, whose sums k_kv_attn_many_join adds (2
// sequences of 8192, 512 rows of each, 197 us; 290 with the tiles whole).
// SKIP: waves pass over tokens that none of their rows sees, for tiles with many empty rows: a wave without rows then decodes
// only (64 sequences of 4096, 8 cache heads of 128, 96 rows of each 252 us, 326 without it; 192 rows 331 and 351).  Full tiles do
// better without the second loop body: 256 rows 370 us, 377 with it, 16384 rows of one sequence 2.52 and 2.58 ms.
#include "kv_attn.h"

namespace qlora {

namespace {

constexpr int kTile = 64;                 // tokens of a step
constexpr float kManyBits = 7.0f;         // probabilities are held times 2^7 relative to a maximum up to 2^6 too small
constexpr float kMoveAt = 6.0f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma32h(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// maximum and sum of a lane and the one 32 away
__device__ __forceinline__ float pair_max(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// A thread's share of a tile: 16-byte chunks of codes (32 elements of one token) and their scales.
template <int D, int NB>
struct ManyLoads {
  static constexpr int T = many_threads(D);
  static constexpr int CH = D / 32;                        // chunks of a row
  static constexpr int ITEMS = 2 * kTile * CH / T > 0 ? 2 * kTile * CH / T : 1;
  static constexpr int KN = D == 64 ? 2 : 4;               // 32-element runs that a key chunk touches
  static constexpr int NKS = KN * NB * 32 / D > 0 ? KN * NB * 32 / D : 1;   // and blocks
  uint32_t page[ITEMS];                                    // the table's entries
  u32x4 c[ITEMS];
  uint32_t s[ITEMS][(NKS + 1) / 2];                        // bf16 scales (a value chunk has one)
};

template <int D, int NB, bool SKIP>
__global__ __launch_bounds__(many_threads(D), many_threads(D) / 256) void k_kv_attn_many(AttnArgs a, CodePlanes cp0,
                                                                                        int split, int cuts) {
  using Loads = ManyLoads<D, NB>;
  constexpr int T = Loads::T, MW = T / 64, TR = 32 * MW, B = D / NB, CH = Loads::CH, ITEMS = Loads::ITEMS;
  constexpr int NKS = Loads::NKS, KN = Loads::KN, KK = D / 16, DT = D / 32, RB = D / 2;
  constexpr int KS = 2 * D + 16;          // bytes of a key row in LDS: 16 rows' pieces of 16 bytes lie in different banks
  constexpr int VS = 2 * D + 64;          // of a value row: 4 rows' pieces of 64 bytes do
  __shared__ __attribute__((aligned(16))) unsigned char kt[2][kTile * KS];
  __shared__ __attribute__((aligned(16))) unsigned char vt[2][kTile * VS];
  __shared__ uint32_t pub[2][16];         // per wave the largest finite scale of its key chunks, from 8 on of its value chunks
  __shared__ uint32_t poison[2][2 * NB];  // tokens whose values are NaN, per block
  __shared__ SeqTable<T> seqs;
  __shared__ int found;

  // the tables in vector registers: a byte permute takes one scalar operand at most, and would have the other copied each time
  CodePlanes cp = cp0;
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(cp.lo[i]), "+v"(cp.hi[i]));

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h32 = lane >> 5;

  // All tiles of the call and the longest cache among them: from these, in how many parts each tile is cut.
  auto tiles = [&](const Seq& s) -> int {
    const int64_t rows = (int64_t)s.n * a.group;
    return rows > a.few ? (int)((rows + TR - 1) / TR) : 0;
  };
  if (threadIdx.x == 0) found = 0;
  if (blockIdx.x == 0) check_batch_entries<T>(a.b);
  int c0 = 0, total = 0;
  for (;;) {
    scan_seqs(a.b, c0, total, seqs, tiles);
    total = __builtin_amdgcn_readfirstlane(seqs.pre[T]);
    if (split && c0 + threadIdx.x < a.b.batch && tiles(Seq{0, seqs.n[threadIdx.x], 0})) atomicMax(&found, seqs.len[threadIdx.x]);
    __syncthreads();
    if (c0 + T >= a.b.batch) break;
    c0 += T;
  }
  int splits = 1;
  if (split) {
    const int most = __builtin_amdgcn_readfirstlane(found) / split;
    // (entries out of order can make more tiles than the workspace and the join were sized for: those stay whole)
    if (total <= cuts / a.c.heads) splits = max(min(most, kSplitWgs / max(total * a.c.heads, 1)), 1);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.meta[0] = total;
      a.meta[1] = splits;
    }
  }
  // this workgroup's tile: item = ((tile of the call) * heads + head) * splits + part
  const int item = blockIdx.x / splits, part = blockIdx.x - item * splits;
  const int tile_at = item / a.c.heads, h = item - tile_at * a.c.heads;
  if (tile_at >= total) return;
  if (a.b.batch > T) {
    c0 = 0;
    int base = 0;
    for (;;) {
      __syncthreads();
      scan_seqs(a.b, c0, base, seqs, tiles);
      base = seqs.pre[T];
      if (base > tile_at) break;
      c0 += T;
    }
  }
  __syncthreads();
  if (seqs.pre[threadIdx.x] <= tile_at && tile_at < seqs.pre[threadIdx.x + 1]) found = threadIdx.x;
  __syncthreads();
  const int bi = __builtin_amdgcn_readfirstlane(found);
  const Seq s = seqs.seq(bi);
  // the last tiles of a sequence see the most tokens: they start first
  const int rt = tiles(s) - 1 - (tile_at - __builtin_amdgcn_readfirstlane(seqs.pre[bi]));
  const Tile t = tile_of<TR>(a, s, c0 + bi, h, rt);

  // rows of q: row 32 wave + l32 of the tile
  const int rr = wave * 32 + l32;
  const bool ok = rr < t.nval;
  const int rho = t.rho0 + (ok ? rr : 0), ri = div_group(a, rho), qh = h * a.group + (rho - ri * a.group);
  const int len = s.len < 0 ? 0 : s.len, pos = len - s.n + ri;
  const int r_hi = !ok ? 0 : a.causal ? pos + 1 : len, r_lo = a.window ? pos + 1 - a.window : 0;
  // tokens that some row of this wave sees
  const int w_hi = (int)wave_max((uint32_t)max(r_hi, 0)), w_lo = __builtin_amdgcn_readfirstlane(r_lo);
  u32x4 qf[KK];
  float rs;                               // logit (in log2) of one unit of its products, but for the keys' exponent
  {
    const uint16_t* qp = a.q.data + (s.row0 + ri) * a.q.rs + qh * a.q.hs + 8 * h32;
#pragma unroll
    for (int k = 0; k < KK; ++k) qf[k] = *reinterpret_cast<const u32x4*>(qp + 16 * k);
  }

  // this part's steps
  const int all = t.hi > t.base ? (t.hi - t.base + kTile - 1) / kTile : 0;
  const int per = (all + splits - 1) / splits, st0 = min(part * per, all), st1 = min(st0 + per, all);

  const int pshift = a.c.pshift;
  const uint32_t pages = (uint32_t)a.c.pages;
  const int64_t head_row = (int64_t)h << pshift;
  const uint8_t *const kc = a.c.kc + head_row * RB, *const vc = a.c.vc + head_row * RB;
  const uint16_t *const ksc = a.c.ks + head_row * NB, *const vsc = a.c.vs + head_row * NB;
  const uint32_t page_rows = (uint32_t)a.c.heads << a.c.pshift, slot_mask = (1u << a.c.pshift) - 1;
  const int32_t* const table = a.b.table + (int64_t)t.b * a.b.max_pages;

  // Chunk `i` of this thread: of the keys for the first half of all chunks, then of the values.  (64 chunks of one kind
  // to a wave, so the kind is a scalar.)
  auto is_key = [&](int i) { return wave * 64 + i * T < kTile * CH; };
  auto has = [&](int i) { return 2 * kTile * CH % T == 0 || wave * 64 + i * T < 2 * kTile * CH; };
  auto chunk_of = [&](int i, int& tok, int& c) {
    const int n = ((int)threadIdx.x + i * T) & (kTile * CH - 1);
    tok = n / CH;
    c = n % CH;
  };
  // The table's entries of a tile are loaded a tile ahead of its codes, and neither they nor the scales are looked at
  // before the step in which they are used: a wait for one load would be one for all.
  auto load_pages = [&](uint32_t (&pg)[ITEMS], int st) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      int tk, c;
      chunk_of(i, tk, c);
      const int tok = t.base + st * kTile + tk;
      pg[i] = table[tok < t.hi ? tok >> pshift : 0];
    }
  };
  auto load = [&](Loads& L, const uint32_t (&pg)[ITEMS], int st) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      const bool key = is_key(i);
      int tk, c;
      chunk_of(i, tk, c);
      L.page[i] = pg[i];
      const uint32_t tok = t.base + st * kTile + tk;
      const uint64_t row = (uint64_t)(pg[i] < pages ? pg[i] : 0u) * page_rows + (tok & slot_mask);
      L.c[i] = *reinterpret_cast<const u32x4*>((key ? kc : vc) + row * RB + 16 * c);
      const uint16_t* sp = (key ? ksc : vsc) + row * NB;
      if (key) {
        sp += D == 256 ? (c / 4) * NKS : 0;   // the scales of its section
        if constexpr (NKS == 1) {
          L.s[i][0] = *sp;
        } else {
#pragma unroll
          for (int x = 0; x < NKS / 2; ++x) L.s[i][x] = reinterpret_cast<const uint32_t*>(sp)[x];
        }
      } else {
        L.s[i][0] = sp[32 * c / B];
      }
    }
  };
  auto finite = [](uint32_t h) { return (h & 0x7FFFu) < 0x7F80u ? h & 0x7FFFu : 0u; };
  // Tile st, loaded: scales of tokens past the end become 0, of tokens without a page NaN; then its largest finite scales
  // and (bit 31) whether a value's is not finite, for all waves.
  auto publish = [&](Loads& L, int st) {
    const int par = st & 1;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      int tk, c;
      chunk_of(i, tk, c);
      if (NKS > 1 && !is_key(i)) {   // a value chunk has one scale: in every place
#pragma unroll
        for (int x = 0; x < (NKS + 1) / 2; ++x) L.s[i][x] = (L.s[i][0] & 0xFFFFu) * 0x10001u;
      }
      const bool last = t.base + (st + 1) * kTile > t.hi, in = !last || t.base + st * kTile + tk < t.hi;
      const bool wrong = in && L.page[i] >= pages;
      if (last || __any(wrong)) {
        if (__any(wrong) && lane == 0) raise_fault(a.b, kFaultPage);
#pragma unroll
        for (int x = 0; x < (NKS + 1) / 2; ++x) {
          if (wrong) L.s[i][x] = kBf16NaN * 0x10001u;
          if (!in) L.s[i][x] = 0;
        }
      }
    }
    uint32_t mk = 0, mv = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      if (is_key(i)) {
#pragma unroll
        for (int x = 0; x < (NKS + 1) / 2; ++x) {
          mk = max(mk, finite(L.s[i][x]));
          if (NKS > 1) mk = max(mk, finite(L.s[i][x] >> 16));
        }
      } else {
        mv = max(mv, finite(L.s[i][0]));
        bad |= (L.s[i][0] & 0x7FFFu) >= 0x7F80u;
      }
    }
    if constexpr (ITEMS == 1) {   // a wave's chunks are of one kind
      const bool key = is_key(0);
      const uint32_t m = wave_max(key ? mk : mv);
      mk = key ? m : 0u;
      mv = key ? 0u : m;
    } else {
      mk = wave_max(mk);
      mv = wave_max(mv);
    }
    if (__any(bad)) mv |= 0x80000000u;
    if (lane == 0) {
      pub[par][wave] = mk;
      pub[par][8 + wave] = mv;
    }
  };
  struct TileExp {
    int k, v;        // powers of two that its scales were divided by
    bool bad;        // some value is NaN
  };
  int v_most = -100;   // (the same in all waves)
  auto exps = [&](int par) {
    // lanes 0 .. 7 (of every 16) take the waves' keys, 8 .. 15 their values
    const uint32_t w = (lane & 7) < MW ? pub[par][lane & 15] : 0u;
    TileExp e;
    e.bad = __any(w >> 31);
    uint32_t m = w & 0x7FFFFFFFu;
    m = dpp_max<0xB1>(m);    // quad_perm [1, 0, 3, 2]
    m = dpp_max<0x4E>(m);    // quad_perm [2, 3, 0, 1]
    m = dpp_max<0x141>(m);   // row_half_mirror
    e.k = exponent_of(__builtin_amdgcn_readlane(m, 0));
    // not below 2^-60 of the largest so far: the probabilities that make up for it stay in range
    e.v = max(exponent_of(__builtin_amdgcn_readlane(m, 8)), v_most - 60);
    v_most = max(v_most, e.v);
    return e;
  };
  // The tokens of a tile whose values are NaN, for the rows that see them: in the tile they are zeros (0 * NaN would reach
  // rows that do not).  All waves take this branch or none does.
  auto note_poison = [&](const Loads& L, int par) {
    if (threadIdx.x < 2 * NB) poison[par][threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i) || is_key(i)) continue;
      int tk, c;
      chunk_of(i, tk, c);
      if ((L.s[i][0] & 0x7FFFu) >= 0x7F80u) atomicOr(&poison[par][2 * (32 * c / B) + (tk >> 5)], 1u << (tk & 31));
    }
    __syncthreads();
  };
  // Quarter x of this thread's decoding (8 elements of each chunk), and what it needs of the scales.
  auto scales = [&](const Loads& L, const TileExp& e, uint32_t (&sc)[ITEMS][NKS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      const bool key = is_key(i);
      const float f = pow2(key ? -e.k : -e.v);
#pragma unroll
      for (int x = 0; x < NKS; ++x) {
        const uint32_t w = x & 1 ? L.s[i][x / 2] & 0xFFFF0000u : L.s[i][x / 2] << 16;
        float v = __uint_as_float(w) * f;
        if (!key && (w & 0x7F800000u) == 0x7F800000u) v = 0.0f;
        sc[i][x] = pack_f16x2(v, v);
      }
    }
  };
  auto decode = [&](const Loads& L, int par, const uint32_t (&sc)[ITEMS][NKS], int x) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      const bool key = is_key(i);
      int tk, c;
      chunk_of(i, tk, c);
      u32x4 v = decode_planes(cp, L.c[i][x]);
      // dword 4c + x of the row: of a key row run k, group g of its section
      const int k = D == 64 ? x & 1 : x;
      const uint32_t sx = sc[i][NKS == 1 ? 0 : NKS == KN ? k : k / 2];
#pragma unroll
      for (int y = 0; y < 4; ++y) v[y] = mul_f16x2(v[y], sx);
      const int own = key ? (D == 64 ? 2 * c : (c & ~3) * 4 + (c & 3)) : 4 * c;
      const int at = key ? (D == 64 ? 4 * (x & 1) + (x >> 1) : 4 * x) : x;
      unsigned char* const row = key ? kt[par] + tk * KS : vt[par] + tk * VS;
      *reinterpret_cast<u32x4*>(row + 16 * own + 16 * at) = v;
    }
  };

  f32x16 O[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[d][i] = 0.0f;
  float m = neg_inf(), l = 0.0f;      // the maximum that the sums are relative to (log2), this lane's part of the sum
  int ve = -100;                      // O is in units of 2^ve
  uint32_t nan_blocks = 0;            // blocks in which this row has seen a NaN

  // the first two tiles' loads are in flight while the rows are brought to fp16
  Loads L, L0;
  uint32_t pg[ITEMS], pg0[ITEMS], pg1[ITEMS];
  TileExp cur{0, 0, false}, nxt{0, 0, false};
  if (st0 < st1) {
    load_pages(pg0, st0);
    load_pages(pg1, st0 + 1);
    load_pages(pg, st0 + 2);
    load(L0, pg0, st0);
    load(L, pg1, st0 + 1);
  }
  {
    uint32_t mag = 0;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      if (!ok) qf[k] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 4; ++x) mag = max(mag, max(qf[k][x] & 0x7FFFu, (qf[k][x] >> 16) & 0x7FFFu));
    }
    mag = max(mag, (uint32_t)__shfl_xor((int)mag, 32, 64));
    const int e = exponent_of(mag);
    const float f = row_unit(mag, e);
    rs = a.scale * kLog2e * cp.inv * pow2(e);
#pragma unroll
    for (int k = 0; k < KK; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        qf[k][x] = pack_f16x2(__uint_as_float(qf[k][x] << 16) * f, __uint_as_float(qf[k][x] & 0xFFFF0000u) * f);
  }
  if (st0 < st1) {
    // Tokens at the front that no row sees: neither their scales nor their pages' entries count.  (A scalar: with the bound
    // in a vector register heads of 256 take 1.5% longer, by other registers in the same loop.)
    const int skip = __builtin_amdgcn_readfirstlane(st0 == 0 ? t.skip : 0);
    if (skip) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (!has(i)) continue;
        int tk, c;
        chunk_of(i, tk, c);
        if (tk >= skip) continue;
        L0.page[i] = 0;
#pragma unroll
        for (int x = 0; x < (NKS + 1) / 2; ++x) L0.s[i][x] = 0;
      }
    }
    publish(L0, st0);
    __syncthreads();
    cur = exps(st0 & 1);
    if (cur.bad) note_poison(L0, st0 & 1);
    uint32_t sc[ITEMS][NKS];
    scales(L0, cur, sc);
#pragma unroll
    for (int x = 0; x < 4; ++x) decode(L0, st0 & 1, sc, x);
    publish(L, st0 + 1);
  }
  for (int st = st0; st < st1; ++st) {
    const int par = st & 1, tok0 = t.base + st * kTile;
    __syncthreads();   // tile st is in LDS, tile st - 1 done with, tile st + 1's exponents published
    nxt = exps(par ^ 1);   // (past the last tile: of an earlier one, and what is decoded is not used)
    if (nxt.bad) note_poison(L, par ^ 1);
    uint32_t sc[ITEMS][NKS];
    scales(L, nxt, sc);

    if (SKIP && (tok0 >= w_hi || tok0 + kTile <= w_lo)) {   // nothing that this wave's rows see
#pragma unroll
      for (int x = 0; x < 4; ++x) decode(L, par ^ 1, sc, x);
      load(L, pg, st + 2);
      load_pages(pg, st + 3);
      cur = nxt;
      if (st + 1 < st1) publish(L, st + 2);
      continue;
    }

    // S^T: 64 tokens x 32 rows; a key operand is read four products ahead of its own, and the next tile is decoded
    // between the products
    f32x16 S[2];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 16; ++i) S[tt][i] = 0.0f;
    // a wave in its products goes before the SIMD's other one, which then finds the matrix core free for its own (1% here)
    __builtin_amdgcn_s_setprio(1);
    const unsigned char* const kp = kt[par] + l32 * KS + 16 * h32;
    constexpr int QK = 2 * KK, RING = 4;
    u32x4 kf[RING];
    auto read_k = [&](int n) { return *reinterpret_cast<const u32x4*>(kp + (n / KK) * 32 * KS + 32 * (n % KK)); };
#pragma unroll
    for (int n = 0; n < RING; ++n) kf[n] = read_k(n);
#pragma unroll
    for (int n = 0; n < QK; ++n) {
      S[n / KK] = mfma32h(kf[n % RING], qf[n % KK], S[n / KK]);
      if (n + RING < QK) kf[n % RING] = read_k(n + RING);
      if (n % (QK / 4) == QK / 8) decode(L, par ^ 1, sc, n / (QK / 4));
    }
    __builtin_amdgcn_s_setprio(0);
    load(L, pg, st + 2);
    load_pages(pg, st + 3);
    // register i of tile tt is token 32 tt + 8 (i / 4) + 4 h32 + i % 4
    const bool edge = tok0 < t.lo_max || tok0 + kTile > t.hi_min;
    if (edge) {
      const int hi = r_hi - tok0 - 4 * h32, lo = r_lo - tok0 - 4 * h32;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int n = 32 * tt + 8 * (i / 4) + i % 4;
          if (n >= hi || n < lo) S[tt][i] = neg_inf();
        }
    }
    // Not 0 (zero queries and zero keys have exponents that add up to -200), which the -inf of a masked token would turn into
    // NaN.  The products are below 2^14, so logits of a smaller factor are 0 all the same.
    const float f = fmaxf(rs * pow2(cur.k), 0x1p-126f);
    float mx = S[0][0];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, S[tt][i]);
    mx = pair_max(mx) * f;
    const int ve_new = max(ve, cur.v);
    if (__any(mx > m + kMoveAt) || ve_new != ve) {
      const float mn = fmaxf(mx, m), mu = mn == neg_inf() ? 0.0f : mn;
      const float alpha = __builtin_amdgcn_exp2f(m - mu);
      m = mn;
      l *= alpha;
      const float fo = alpha * pow2(max(ve - ve_new, -126));
      ve = ve_new;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[d][i] *= fo;
    }
    // a tile of smaller values than the largest so far: its probabilities are made smaller instead
    const float shift = (float)(cur.v - ve);
    const float off = kManyBits - (m == neg_inf() ? 0.0f : m) + shift, back = pow2(min(ve - cur.v, 126));
    uint32_t pp[2][8];
    float ls = 0.0f;
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[tt][2 * i], f, off));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[tt][2 * i + 1], f, off));
        ls += p0;
        ls += p1;
        pp[tt][i] = pack_f16x2(p0, p1);
      }
    l = __builtin_fmaf(ls, back, l);

    // O^T += V^T P^T: 16 tokens at a time, slot (h32, j) of them token 4 h32 + j, or 8 + 4 h32 + j - 4 from j = 4 on
    __builtin_amdgcn_s_setprio(1);
    const int G = lane >> 4, j = lane & 15;
    const unsigned char* vp = vt[par] + (4 * (G >> 1) + (j >> 2)) * VS + 2 * (16 * (G & 1) + 4 * (j & 3));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const u32x4 pf = {pp[x / 2][4 * (x % 2)], pp[x / 2][4 * (x % 2) + 1], pp[x / 2][4 * (x % 2) + 2],
                        pp[x / 2][4 * (x % 2) + 3]};
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const unsigned char* p = vp + 16 * x * VS + 64 * d;
        const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p));
        const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p + 8 * VS));
        const uint2 w0 = __builtin_bit_cast(uint2, v0), w1 = __builtin_bit_cast(uint2, v1);
        O[d] = mfma32h(u32x4{w0.x, w0.y, w1.x, w1.y}, pf, O[d]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (cur.bad) {   // rare: which blocks hold a NaN that this row sees
      for (int b = 0; b < NB; ++b)
        for (int n = 0; n < kTile; ++n)
          if ((poison[par][2 * b + (n >> 5)] >> (n & 31) & 1u) && tok0 + n < r_hi && tok0 + n >= r_lo) nan_blocks |= 1u << b;
    }
    cur = nxt;
    if (st + 1 < st1) publish(L, st + 2);
  }

  l = pair_sum(l) * pow2(-(int)kManyBits);
  const float ofs = pow2(ve - (int)kManyBits) * cp.inv;
  if (!ok) return;
  if (splits == 1) {
    float inv = l == 0.0f ? 0.0f : ofs / l;
    if (s.len < 0) inv = __builtin_nanf("");
    uint16_t* op = a.o.data + (s.row0 + ri) * a.o.rs + qh * a.o.hs + 4 * h32;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = nan_blocks >> (32 * d / B) & 1u ? __builtin_nanf("") : inv;
        uint2 w;
        w.x = pack_bf16x2(O[d][4 * i] * g, O[d][4 * i + 1] * g);
        w.y = pack_bf16x2(O[d][4 * i + 2] * g, O[d][4 * i + 3] * g);
        *reinterpret_cast<uint2*>(op + 32 * d + 8 * i) = w;
      }
    if (a.lse && h32 == 0)
      a.lse[(s.row0 + ri) * (int64_t)a.q.n + qh] =
          s.len < 0 ? __builtin_nanf("") : l == 0.0f ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
    return;
  }
  float* dst = a.part + (int64_t)blockIdx.x * (TR * (D + 2));
  const float inv = s.len < 0 ? __builtin_nanf("") : ofs;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g = nan_blocks >> (32 * d / B) & 1u ? __builtin_nanf("") : inv;
      *reinterpret_cast<f32x4*>(dst + rr * D + 32 * d + 8 * i + 4 * h32) =
          f32x4{O[d][4 * i] * g, O[d][4 * i + 1] * g, O[d][4 * i + 2] * g, O[d][4 * i + 3] * g};
    }
  if (h32 == 0) {
    dst[TR * D + rr] = m;
    dst[TR * D + TR + rr] = s.len < 0 ? __builtin_nanf("") : l;
  }
  if (part == 0 && threadIdx.x == 0) {   // (its row is always there)
    int32_t* mt = a.meta + (1 + item) * kMetaInts;
    mt[1] = (int32_t)s.row0;
    mt[2] = t.rho0;
    mt[3] = t.nval;
    mt[4] = h;
  }
}

// Adds the parts of a tile: workgroup (item, y), wave v row 4y + v.
template <int D>
__global__ __launch_bounds__(256) void k_kv_attn_many_join(AttnArgs a) {
  constexpr int TR = many_threads(D) / 2;
  const int splits = a.meta[1];
  if (splits == 1 || (int)blockIdx.x / a.c.heads >= a.meta[0]) return;
  const int32_t* mt = a.meta + (1 + blockIdx.x) * kMetaInts;
  const int rr = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (rr >= mt[3]) return;
  constexpr int64_t P = TR * (D + 2);
  join_row<D>(
      a, splits, TR, rr, mt, [&](int k) { return a.part + ((int64_t)blockIdx.x * splits + k) * P; }, [](int d) { return d; });
}

}  // namespace

template <int D, int NB>
static hipError_t launch_many(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  {
    ProfScope ps("k_kv_attn_many", s);
    const dim3 g((unsigned)pl.many_wgs), t(many_threads(D));
    const CodePlanes cp = code_planes(a.c.cb);
    // (for D = 64 such tiles are the other kernel's, 160 rows 83 us either way; for D = 256 the second loop body spills
    // registers, 16 sequences of 40 rows 305 us with it, 289 without)
    const int cuts = (int)pl.many_split;
    if (D == 128 && pl.sparse)
      hipLaunchKernelGGL((k_kv_attn_many<D, NB, D == 128>), g, t, 0, s, a, cp, pl.split_tokens, cuts);
    else
      hipLaunchKernelGGL((k_kv_attn_many<D, NB, false>), g, t, 0, s, a, cp, pl.split_tokens, cuts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !pl.many_split) return e;
  }
  ProfScope ps("k_kv_attn_many_join", s);
  hipLaunchKernelGGL((k_kv_attn_many_join<D>), dim3((unsigned)pl.many_split, many_threads(D) / 8), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_attn_many(const AttnArgs& a, const AttnPlan& pl, int D, int block, hipStream_t s) {
  const int nb = D / block;
  if (D == 64) return nb == 1 ? launch_many<64, 1>(a, pl, s) : launch_many<64, 2>(a, pl, s);
  if (D == 128)
    return nb == 1 ? launch_many<128, 1>(a, pl, s) : nb == 2 ? launch_many<128, 2>(a, pl, s) : launch_many<128, 4>(a, pl, s);
  return nb == 2 ? launch_many<256, 2>(a, pl, s) : nb == 4 ? launch_many<256, 4>(a, pl, s) : launch_many<256, 8>(a, pl, s);
}

}  // namespace qlora
