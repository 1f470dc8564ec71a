// Fused forward for large token counts ("QLoRA: Efficient Finetuning of Quantized
// LLMs", section "The QLoRA layer, end to end": every product runs in bf16 on a
// weight decoded from its 4-bit storage, and no bf16 copy of the weight is kept;
// y = x W + s (x L1) L2):
//
//   Y[M][N] = bf16( X[M][K] deq(W)^T + Ts[M][rp] B~ ),   B~(j, n) = B[j][n] (j < r), 0 otherwise
//
// Ts = bf16(s * X A) comes from the rank-r kernel.  The K/64 NF4 stages are
// followed by rp/64 adapter stages that accumulate into the same registers, so
// one bf16 rounding ends the whole sum.  In an NF4 stage each thread dequantizes a
// quarter of one 64-weight block (the block's scaled 16-entry table is built by the
// four threads of the block together, the lookups are byte permutes) straight into
// the LDS feature tile.
//
// The gated block's forward, H = bf16(act(G) U) with G and U two such products of the same X, runs through the same code: the 128
// features of a tile are 64 of the gate's weight and the same 64 of the up projection's, so the waves of one feature half
// hold G and those of the other U, and meet in LDS after the reduction.  X is read once for both, and G and U
// reach memory only where the backward wants them.  2048 tokens of 4096 -> 11008 with G, U and T: 444 to 473 us by box =
// 780 to 830 TFLOP/s, of which X A takes 15 (a library product of the two weights in bf16 alone: 417).  Of 875 thousand cycles (1.8 GHz
// under this load) the matrix cores are busy in 41 %, the VALU, with decoding, in 33 %, and the waves, two to a SIMD, wait 30 % of their time.
#include <algorithm>

#include "common.h"
#include "gated.h"
#include "gemv.h"
#include "gemm_core.h"
#include "kernels.h"

namespace qlora {

namespace {

using namespace gemm;

struct FwdParams {
  const uint16_t* X;
  int64_t M, K, N;
  NF4View w;
  uint64_t codes_bytes, absmax_bytes, c1_bytes;
  const uint16_t* Ts;
  int64_t rp;
  const uint16_t* B;
  int64_t r;
  uint16_t* Y;
  NF4Table tab;
  // split mode: K-slices of `spl` stages, fp32 partials [split][M][npad], no adapter stages
  float* partial;
  int64_t npad;
  uint32_t spl;
  // gated: the up projection's weight (w, Ts, B, partial are the gate's), outputs besides Y = H
  NF4View w2;
  const uint16_t* Ts2;
  const uint16_t* B2;
  float* partial2;
  uint16_t* G;   // or NULL, with U
  uint16_t* U;
  int act;
  // gated: tiles from `whole` on are cut into `slices` of the reduction, fp32 sums to partial, partial2
  // [slice][256][npad] (GatedTail in kernels.h)
  uint32_t whole, slices;
};

// In front of the gated block's products in K-slices: the workgroups that form the partial sums of X A for both sides (a launch of
// their own takes 4.6 us of a call of 27).
static_assert(gemv::kLdsAdapter <= SMEM_ELEMS * 2 && gemv::GT == NT, "both kinds of workgroups in one launch");
struct AdapterFront {
  static constexpr bool any = true;
  gemv::GemvParams a;
  gemv::GemvSide up;
  uint32_t adapters;   // of each side

  // Whether workgroup `bid` is one of them, and then its work; else bid is made the products'.
  __device__ __forceinline__ bool run(uint32_t& bid, uint16_t* smem) {
    if (bid >= 2 * adapters) {
      bid -= 2 * adapters;
      return false;
    }
    if (bid >= adapters) {
      bid -= adapters;
      a.A = up.A;
      a.tpartial = up.tpartial;
    }
    gemv::adapter_group(a, (int)bid, reinterpret_cast<uint8_t*>(smem));
    return true;
  }
};
struct NoFront {
  static constexpr bool any = false;
};

struct WRegs {
  uint2 code;     // 16 codes (a quarter of a block)
  uint32_t c2;    // 8-bit block constant (double quant) or fp32 absmax bits
  float c1;
};

struct Stage {
  TokenRegs T;
  WRegs W;
};

// BM: 0 for blocks of 64 (one block per row per stage), 1 for 128 and 256 (a block spans
// 2 or 4 stages), 2 for 32 (two blocks per row per stage: the two halves of a quad use
// different scales, so each lane builds the whole 16-entry table itself).
// SPLIT: a workgroup covers stages [spl s, spl (s + 1)) of its tile's reduction and writes
// fp32 partial sums (few tokens: the K-slices give the GPU enough workgroups); the adapter
// term and the final sum come from the weight-streaming path's epilogue.
// GATED: a tile has 64 features of each of two weights (p.w, p.w2); see above.
// TAIL: the last tiles are cut into slices (GatedTail).
// FRONT: workgroups of another kind in front of the products (AdapterFront), or NoFront.
// (The text stands in the kernel itself: as a function that is inlined into it, the linear layer's products are scheduled
// otherwise and take 1 to 3 % longer, 4096 -> 11008 with 2048 tokens 228.8 us against 225.4.)
template <bool DQ, int BM, bool SPLIT, bool GATED, bool TAIL, class FRONT>
__global__ __launch_bounds__(NT) void k_fwd_nf4_gemm(FwdParams p, FRONT front) {
  __shared__ __attribute__((aligned(16))) uint16_t smem[SMEM_ELEMS];
  uint32_t bid = blockIdx.x;
  if constexpr (FRONT::any) {
    if (front.run(bid, smem)) return;
  }
  uint16_t* const sT[2] = {smem, smem + TILE_T};
  uint16_t* const sF[2] = {smem + 2 * TILE_T, smem + 2 * TILE_T + TILE_F};

  int64_t tt, tf;
  constexpr int FT = GATED ? BF / 2 : BF;   // features of a tile
  const int64_t tiles_t = (p.M + BT - 1) / BT, tiles_f = (p.N + FT - 1) / FT;
  const uint32_t split = SPLIT ? (uint32_t)(bid / (tiles_t * tiles_f)) : 0u;
  uint32_t part = 0;   // slice of a tile at the end of the launch
  bool tail = false;
  if constexpr (TAIL) {
    tail = bid >= p.whole;
    if (tail) {
      const uint32_t n = (uint32_t)(tiles_t * tiles_f) - p.whole, i = bid - p.whole;
      part = i / n;
      tt = tiles_t - 1;
      tf = tiles_f - n + (i - part * n);
    } else {
      // the tiles before them, a multiple of 256, in runs of one XCD each (see tile_of)
      const uint32_t L = (bid & 7) * (p.whole >> 3) + (bid >> 3);
      tt = L / tiles_f;
      tf = L - tt * tiles_f;
    }
  } else {
    tile_of(tiles_t, tiles_f, tt, tf, (int64_t)bid - (int64_t)split * tiles_t * tiles_f);
  }
  const uint32_t m0 = (uint32_t)(tt * BT), n0 = (uint32_t)(tf * FT);
  const uint32_t nkb_all = (uint32_t)(p.K / 64);
  const uint32_t it0 = SPLIT ? split * p.spl : tail ? part * nkb_all / p.slices : 0u;   // first stage
  const uint32_t nkb = SPLIT ? min(nkb_all, it0 + p.spl) - it0                           // stages of this workgroup
                             : (tail ? (part + 1) * nkb_all / p.slices : nkb_all) - it0;
  const int t = threadIdx.x;
  // weight row t/4 of the tile, quarter t%4 of its block (groups 2q and 2q+1 -> chunks
  // 2q, 2q+1 of the LDS row); rows past N read as zero (their outputs are not stored)
  const int wrow = t >> 2, wq = t & 3;
  const uint32_t wblk0 = (n0 + (GATED ? wrow & (BF / 2 - 1) : wrow)) * nkb_all;
  const uint32_t code_off = wblk0 * kBlockBytes + wq * 8;

  const TokenSrc xs = token_src(p.X, (uint64_t)p.M * p.K * 2, (uint32_t)p.K, m0);
  // (waves 4 .. 7 load rows 64 .. 127 of the tile)
  const bool up = GATED && __builtin_amdgcn_readfirstlane(t >> 6) >= 4;
  const rsrc_t rC = make_rsrc(up ? p.w2.codes : p.w.codes, p.codes_bytes);
  const rsrc_t rA = make_rsrc(up ? p.w2.absmax : p.w.absmax, p.absmax_bytes);
  const rsrc_t rC1 = make_rsrc(up ? p.w2.c1 : p.w.c1, p.c1_bytes);
  constexpr bool dq = DQ;
  const float mu = dq ? *(up ? p.w2.mu : p.w.mu) : 0.0f;
  const QuadLevels lev = quad_levels(p.tab);

  const uint32_t bsh = (uint32_t)(p.w.bshift - 6);   // BM == 1: 64-chunks per block, log2
  auto load = [&](uint32_t it, Stage& S) {
    load_tokens(S.T, xs, it * 64);
    S.W.code = ld8(rC, code_off, it * kBlockBytes);
    if constexpr (BM == 0) {
      if constexpr (dq) {
        S.W.c2 = __builtin_amdgcn_raw_buffer_load_b8(rA, wblk0, it, 0);
        S.W.c1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rC1, ((wblk0 + it) >> 8) * 4, 0, 0));
      } else {
        S.W.c2 = __builtin_amdgcn_raw_buffer_load_b32(rA, wblk0 * 4, it * 4, 0);
        S.W.c1 = 0.0f;
      }
    } else {
      // block of this thread's 16 weights
      const uint32_t sb = BM == 1 ? (wblk0 + it) >> bsh : ((wblk0 + it) << 1) + (uint32_t)(wq >> 1);
      if constexpr (dq) {
        S.W.c2 = __builtin_amdgcn_raw_buffer_load_b8(rA, sb, 0, 0);
        S.W.c1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rC1, (sb >> 8) * 4, 0, 0));
      } else {
        S.W.c2 = __builtin_amdgcn_raw_buffer_load_b32(rA, sb * 4, 0, 0);
        S.W.c1 = 0.0f;
      }
    }
  };
  auto planes = [&](float scale) -> Planes {
    if constexpr (BM == 2)
      return make_planes(p.tab, scale);
    else
      return quad_planes(lev, scale);
  };

  auto scale_of = [&](const Stage& S) -> float {
    return dq ? __fadd_rn(__fmul_rn(e4m3_decode(S.W.c2), S.W.c1), mu) : __uint_as_float(S.W.c2);
  };
  auto put = [&](const Planes& pl, uint32_t cw, int d, int sb) {
    *reinterpret_cast<u32x4*>(sF[sb] + swzF(wrow, 2 * wq + d)) = dequant8(pl, cw);
  };

  // This wave's MFMAs of the stage in LDS buffer `cb`, with the store of stage S into
  // buffer `sb` cut into pieces between the MFMA groups.
  const int kh = wave_k();
  auto compute_store = [&](Acc& acc, int cb, const Stage& S, int sb) {
    Frags Fa, Fb;
    read_frags<GATED>(Fa, sT[cb], sF[cb], 2 * kh);
    read_frags<GATED>(Fb, sT[cb], sF[cb], 2 * kh + 1);
    mma_group(acc, Fa, 0);
    store_tokens_part(S.T, sT[sb], 0);
    store_tokens_part(S.T, sT[sb], 1);
    const float scale = scale_of(S);
    mma_group(acc, Fa, 1);
    store_tokens_part(S.T, sT[sb], 2);
    store_tokens_part(S.T, sT[sb], 3);
    const Planes pl = planes(scale);
    mma_group(acc, Fb, 0);
    put(pl, S.W.code.x, 0, sb);
    mma_group(acc, Fb, 1);
    put(pl, S.W.code.y, 1, sb);
    interleave_mfma_valu();
  };

  auto store_all = [&](const Stage& S, int sb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_tokens_part(S.T, sT[sb], i);
    const Planes pl = planes(scale_of(S));
    put(pl, S.W.code.x, 0, sb);
    put(pl, S.W.code.y, 1, sb);
  };

  Acc acc;
  acc_zero(acc);
  Stage S0, S1;
  // Prefetch loads are unconditional (a stage index past the end is clamped to the last
  // stage and the data is never stored): a load under a branch would make the compiler
  // wait for every load in flight where the branch rejoins.
  const uint32_t last = it0 + nkb - 1;
  load(it0, S0);
  load(min(it0 + 1, last), S1);
  store_all(S0, 0);
  __syncthreads();
  // two stages per trip (stage it in buffer 0 with it+1 in S1, then it+1 in buffer 1 with
  // it+2 in S0); a single exit keeps the accumulators in one register set
  uint32_t it = 0;
  // (of the gated forms) a wave of tokens 128 .. 255 of a panel that has none of them stores its share of the stages alone,
  // between as many barriers: 100 tokens of 4096 -> 11008 62 us a call, with its products of zeros 71
  if (GATED && __builtin_amdgcn_readfirstlane(wave_t<GATED>()) && p.M - (int64_t)m0 <= 128) {
    for (; it + 1 < nkb; it += 2) {
      load(min(it0 + it + 2, last), S0);
      store_all(S1, 1);
      __syncthreads();
      load(min(it0 + it + 3, last), S1);
      store_all(S0, 0);
      __syncthreads();
    }
    if (it < nkb) __syncthreads();
    it = nkb;
  }
  for (; it + 1 < nkb; it += 2) {
    load(min(it0 + it + 2, last), S0);
    compute_store(acc, 0, S1, 1);
    __syncthreads();
    load(min(it0 + it + 3, last), S1);
    compute_store(acc, 1, S0, 0);
    __syncthreads();
  }
  if (it < nkb) {   // odd number of stages: the last one is in buffer 0
    mma_stage<false, GATED>(acc, sT[0], sF[0]);
    __syncthreads();
  }

  if constexpr (SPLIT && GATED) {
    // this wave's 64 features of its weight start at n0 (store_out_f32 adds the feature half's offset)
    if (combine_halves<true>(acc, smem))
      store_out_f32<true>(acc, (wave_f() ? p.partial2 : p.partial) + (int64_t)split * p.M * p.npad, p.npad, m0, p.M,
                    (int64_t)n0 - wave_f() * 64, p.N);
    return;
  }
  if constexpr (SPLIT) {
    if (combine_halves(acc, smem))
      store_out_f32(acc, p.partial + (int64_t)split * p.M * p.npad, p.npad, m0, p.M, n0, p.N);
    return;
  }

  // adapter stages: Ts [M][rp] against rows of B, kept as stored ([j][n]) in the natural
  // tile and read with transposing loads.  Rows j >= r lie past the end of B and read zero.
  // (Gated: each feature half has its own Ts, in the other token buffer, and its half of the natural tile.)
  const TokenSrc ts = token_src(p.Ts, (uint64_t)p.M * p.rp * 2, (uint32_t)p.rp, m0);
  const uint64_t bbytes = (uint64_t)p.r * p.N * 2;
  const rsrc_t rB = make_rsrc(p.B, bbytes);
  const int bj = t >> 3, be = t & 7;
  for (uint32_t j0 = part ? (uint32_t)p.rp : 0u; j0 < (uint32_t)p.rp; j0 += 64) {   // (a tile's first slice takes them)
    TokenRegs T;
    load_tokens(T, ts, j0);
    uint4 b0, b1;
    if constexpr (GATED) {
      const TokenSrc ts2 = token_src(p.Ts2, (uint64_t)p.M * p.rp * 2, (uint32_t)p.rp, m0);
      TokenRegs T2;
      load_tokens(T2, ts2, j0);
      const rsrc_t rB2 = make_rsrc(p.B2, bbytes);
      const uint32_t boff = ((j0 + bj) * (uint32_t)p.N + n0 + (be & 3) * 16) * 2;
      const uint32_t og = be < 4 ? boff : (uint32_t)bbytes, ou = be < 4 ? (uint32_t)bbytes : boff;
      const uint4 g0 = ld16(rB, og), g1 = ld16(rB, og + 16), u0 = ld16(rB2, ou), u1 = ld16(rB2, ou + 16);
      b0 = make_uint4(g0.x | u0.x, g0.y | u0.y, g0.z | u0.z, g0.w | u0.w);   // (one of the two is zero)
      b1 = make_uint4(g1.x | u1.x, g1.y | u1.y, g1.z | u1.z, g1.w | u1.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) store_tokens_part(T2, sT[1], i);
    } else {
      const uint32_t boff = ((j0 + bj) * (uint32_t)p.N + n0 + be * 16) * 2;
      b0 = ld16(rB, boff), b1 = ld16(rB, boff + 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) store_tokens_part(T, sT[0], i);
    *reinterpret_cast<uint4*>(sF[0] + swzN(bj, 2 * be)) = b0;
    *reinterpret_cast<uint4*>(sF[0] + swzN(bj, 2 * be + 1)) = b1;
    __syncthreads();
    mma_stage<true, GATED>(acc, GATED && wave_f() ? sT[1] : sT[0], sF[0]);
    __syncthreads();
  }
  if constexpr (!GATED) {
    if (combine_halves(acc, smem)) store_out(acc, p.Y, p.N, m0, p.M, n0, p.N);
  } else {
    const bool holds = combine_halves<true>(acc, smem);
    if (tail) {
      if (holds) {
        const int64_t rows = min<int64_t>(BT, p.M - m0), left = p.N - n0;
        const int64_t c0 = n0 - (tiles_f - (tiles_t * tiles_f - p.whole)) * FT;   // column of the tail
        float* const out = (wave_f() ? p.partial2 : p.partial) + (int64_t)part * BT * p.npad;
        store_out_f32<true>(acc, out, p.npad, 0, rows, c0 - wave_f() * 64, c0 + min<int64_t>(left, FT));
      }
      return;
    }
    // the wave of G keeps features 0 .. 31 of the tile and takes U's from the wave of U, which keeps 32 .. 63
    const int lane = t & 63, q = wave_t<true>() | wave_f() << 1, wf = wave_f();
    float4* const x = reinterpret_cast<float4*>(smem);
    if (holds) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int v4 = 0; v4 < 4; ++v4) {
          const f32x16 c = wf ? acc.c[0][m] : acc.c[1][m];
          x[((q * 4 + m) * 4 + v4) * 64 + lane] = make_float4(c[4 * v4], c[4 * v4 + 1], c[4 * v4 + 2], c[4 * v4 + 3]);
        }
    }
    __syncthreads();
    if (!holds) return;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t tok = (int64_t)m0 + wave_t<true>() * 128 + m * 32 + (lane & 31);
      const f32x16 own = wf ? acc.c[1][m] : acc.c[0][m];
      if (tok >= p.M) continue;
#pragma unroll
      for (int v4 = 0; v4 < 4; ++v4) {
        const int64_t feat = (int64_t)n0 + wf * 32 + 8 * v4 + 4 * (lane >> 5);
        if (feat >= p.N) continue;
        const float4 o = x[(((q ^ 2) * 4 + m) * 4 + v4) * 64 + lane];
        const float mine[4] = {own[4 * v4], own[4 * v4 + 1], own[4 * v4 + 2], own[4 * v4 + 3]};
        const float other[4] = {o.x, o.y, o.z, o.w};
        float g[4], u[4], h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = wf ? other[i] : mine[i];
          u[i] = wf ? mine[i] : other[i];
          h[i] = activate(g[i], p.act) * u[i];
        }
        const int64_t at = tok * p.N + feat;
        *reinterpret_cast<uint2*>(p.Y + at) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
        if (p.G) {
          *reinterpret_cast<uint2*>(p.G + at) = make_uint2(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
          *reinterpret_cast<uint2*>(p.U + at) = make_uint2(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
        }
      }
    }
  }
}

template <bool SPLIT, bool GATED, bool TAIL = false, class FRONT = NoFront>
void launch_variant(const FwdParams& p, unsigned wgs, hipStream_t s, const FRONT& front = FRONT{}) {
  const dim3 grid(wgs), block(NT);
  const int bm = p.w.bshift == 6 ? 0 : p.w.bshift > 6 ? 1 : 2;
#define FWD_LAUNCH(DQ, BM) \
  hipLaunchKernelGGL((k_fwd_nf4_gemm<DQ, BM, SPLIT, GATED, TAIL, FRONT>), grid, block, 0, s, p, front)
  if (p.w.dq) {
    if (bm == 0) FWD_LAUNCH(true, 0);
    else if (bm == 1) FWD_LAUNCH(true, 1);
    else FWD_LAUNCH(true, 2);
  } else {
    if (bm == 0) FWD_LAUNCH(false, 0);
    else if (bm == 1) FWD_LAUNCH(false, 1);
    else FWD_LAUNCH(false, 2);
  }
#undef FWD_LAUNCH
}

// What the launches share: the weight's buffers and their sizes.
FwdParams params_of(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& w) {
  // 64-element code chunks, and blocks (one constant each; in is a multiple of the block size)
  const uint64_t nchunk = (uint64_t)N * K / 64, nblk = ((uint64_t)N * K) >> w.bshift;
  FwdParams p{};
  p.X = X;
  p.M = M;
  p.K = K;
  p.N = N;
  p.w = w;
  p.codes_bytes = nchunk * kBlockBytes;
  p.absmax_bytes = w.dq ? nblk : nblk * 4;
  p.c1_bytes = w.dq ? ((nblk + 255) / 256) * 4 : 0;
  p.tab = nf4_table(w.cb);
  return p;
}

}  // namespace

hipError_t launch_fwd_gemm(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& w,
                           const uint16_t* Ts, int64_t rp, const uint16_t* B, int64_t r, uint16_t* Y,
                           hipStream_t s) {
  FwdParams p = params_of(X, M, K, N, w);
  p.Ts = Ts;
  p.rp = rp;
  p.B = B;
  p.r = r;
  p.Y = Y;
  ProfScope ps("k_fwd_nf4_gemm", s);
  launch_variant<false, false>(p, (unsigned)(((M + BT - 1) / BT) * ((N + BF - 1) / BF)), s);
  return hipGetLastError();
}

hipError_t launch_fwd_gemm_split(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& w, int stages,
                                 float* partial, int64_t npad, hipStream_t s) {
  FwdParams p = params_of(X, M, K, N, w);
  p.partial = partial;
  p.npad = npad;
  p.spl = (uint32_t)stages;
  const int64_t used = (K / 64 + stages - 1) / stages;   // splits that get at least one stage
  ProfScope ps("k_fwd_nf4_gemm", s);
  launch_variant<true, false>(p, (unsigned)(((M + BT - 1) / BT) * ((N + BF - 1) / BF) * used), s);
  return hipGetLastError();
}

GatedTail gated_tail(int64_t M, int64_t K, int64_t N) {
  GatedTail t{0, 0, 0, 0};
  const int64_t tiles_f = (N + BF / 2 - 1) / (BF / 2), tiles = (M + BT - 1) / BT * tiles_f, rest = tiles % 256;
  if (tiles < 256 || rest == 0 || rest > 128 || rest > tiles_f || K / 64 < 16) return t;
  t.tiles = (int)rest;
  t.slices = (int)std::min<int64_t>(256 / rest, 4);
  t.npad = rest * (BF / 2);
  t.part_floats = (size_t)t.slices * BT * t.npad;
  return t;
}

hipError_t launch_gated_gemm(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& gate, const NF4View& up,
                             const uint16_t* Tg, const uint16_t* Tu, int64_t rp, const uint16_t* Bg, const uint16_t* Bu,
                             int64_t r, int act, uint16_t* H, uint16_t* G, uint16_t* U, float* gate_partial, float* up_partial,
                             hipStream_t s) {
  FwdParams p = params_of(X, M, K, N, gate);
  p.w2 = up;
  p.Ts = Tg;
  p.Ts2 = Tu;
  p.rp = rp;
  p.B = Bg;
  p.B2 = Bu;
  p.r = r;
  p.act = act;
  p.Y = H;
  p.G = G;
  p.U = U;
  const GatedTail tail = gated_tail(M, K, N);
  const int64_t tiles_f = (N + BF / 2 - 1) / (BF / 2), tiles = (M + BT - 1) / BT * tiles_f;
  p.whole = (uint32_t)(tiles - tail.tiles);
  p.slices = (uint32_t)std::max(tail.slices, 1);
  p.partial = gate_partial;
  p.partial2 = up_partial;
  p.npad = tail.npad;
  {
    ProfScope ps("k_gated_nf4_gemm", s);
    if (tail.tiles) launch_variant<false, true, true>(p, p.whole + (unsigned)(tail.tiles * tail.slices), s);
    else launch_variant<false, true>(p, p.whole, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || tail.tiles == 0) return e;
  }
  return launch_gated_finish(gate_partial, up_partial, tail, M, N, (M - 1) / BT * BT, (tiles_f - tail.tiles) * (BF / 2), act, H,
                             G, U, s);
}

hipError_t launch_gated_gemm_split(const uint16_t* X, int64_t M, int64_t K, int64_t N, const NF4View& gate, const NF4View& up,
                                   const uint16_t* A_gate, const uint16_t* A_up, int64_t r, const GemvPlan& pl, int stages,
                                   float* gate_partial, float* up_partial, hipStream_t s) {
  FwdParams p = params_of(X, M, K, N, gate);
  p.w2 = up;
  p.partial = gate_partial;
  p.partial2 = up_partial;
  p.npad = pl.npad;
  p.spl = (uint32_t)stages;
  AdapterFront front{gemv::gemv_params(X, M, K, N, gate, A_gate, r, pl, gate_partial), {}, (uint32_t)(pl.agroups * pl.asplits * pl.ngr)};
  front.up.A = A_up;
  front.up.tpartial = up_partial + pl.tpart;
  const int64_t used = (K / 64 + stages - 1) / stages, tiles = ((M + BT - 1) / BT) * ((N + BF / 2 - 1) / (BF / 2));
  ProfScope ps("k_gated_nf4_split", s);
  launch_variant<true, true, false>(p, (unsigned)(tiles * used) + 2 * front.adapters, s, front);
  return hipGetLastError();
}

}  // namespace qlora
