// The key/value cache in 4 bits: rows quantized as they are written, and read back.
//
// Write, per block of B elements of a head's row (the block format of the weight quantizer):
//   a = max|x|,  code = #{k : fl32(x fl32(1/a)) > threshold_k},  scale = a  (exact in bf16).
// Read: bf16_RNE(fl32(level[code] scale)).
//
// Both move each byte once (write: 2 B in, 0.5 + 2/B out per element) and are bound by that, or for a
// few tokens by the launch and the chain start -> length -> page -> data.  One lane holds 8
// elements (16 bytes, one dword of codes); a workgroup takes as many consecutive rows as its lanes
// hold of one head, so that the code dwords of rows that are neighbours in a page land side by side,
// and grid.y spreads the heads.
//
// Measured: 8192 rows of 32 heads of 128 in blocks of 32 (172 MB each way): written in 38 to 41 us = 4.3 TB/s (5 us more where each
// head's row is loaded only when the last one is stored; the encoding, two thirds of the time by its instructions, hides behind
// the loads), read back in 37 us = 4.6 TB/s; 25385 rows of 16 heads read (266 MB) in 60 us = 4.4 TB/s; 64 rows of 8 heads
// 4 us each, the chain of loads.
#include "kernels.h"
#include "kv.h"

namespace qlora {

namespace {

constexpr int KT = 256;   // threads

template <int D>
struct Slot {
  bool ok;          // the row has a slot in the cache
  bool poison;      // it should have one, but an entry on the way to it is wrong
  bool empty;       // a row of the batch without a token
  int64_t page;
  int32_t off;
};

// The slots of rows t0 .. t0 + NT - 1 (row t0 + r for the lanes of group r).  The sequence of a row is the first one whose
// start entries are in order and name it: the workgroup reads all of them at once, and each that has rows here puts its
// number to them, so a batch of any size costs one round trip (a search by halves costs one per halving), and a wrong
// entry costs its own two sequences their rows and no other.  A thread puts its sequence's number to the first of its
// rows, its wave to the others, lane k to row k (a loop of the thread over up to 32 rows: 1 us).
template <int D>
__device__ __forceinline__ Slot<D> find_slot(const BatchView& b, const KvView& c, int64_t t0, int r, int* own) {
  constexpr int NT = KT / (D / 8);
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < NT; i += KT) own[i] = INT32_MAX;
  __syncthreads();
  for (int i0 = 0; i0 < b.batch; i0 += KT) {
    const int i = i0 + threadIdx.x;
    int from = 0, to = 0;   // its rows here
    if (i < b.batch) {
      const int64_t s0 = b.start[i], e = b.start[i + 1];
      if (s0 < 0 || e < s0 || e > b.rows) raise_fault(b, kFaultStart);
      else if (s0 < t0 + NT && e > t0) from = (int)(s0 > t0 ? s0 - t0 : 0), to = (int)(e < t0 + NT ? e - t0 : NT);
    }
    if (from < to) atomicMin(&own[from], i);
    for (uint64_t more = __ballot(to - from > 1); more; more &= more - 1) {
      const int l = __builtin_ctzll(more);
      const int f = __builtin_amdgcn_readlane(from, l), n = __builtin_amdgcn_readlane(to, l);
      if (lane > f && lane < n) atomicMin(&own[lane], __builtin_amdgcn_readlane(i, l));
    }
  }
  __syncthreads();
  const int seq = own[r];
  Slot<D> s{false, false, false, 0, 0};
  if (seq == INT32_MAX) return s;
  const int64_t t = t0 + r, s1 = b.start[seq + 1];
  const int len = b.length[seq];
  if (len < 0 || len > b.max_len) {
    raise_fault(b, kFaultLength);
    s.poison = true;
    return s;
  }
  const int64_t p = (int64_t)len - (s1 - t);
  if (p < 0) {
    s.empty = true;
    return s;
  }
  const int pid = b.table[(int64_t)seq * b.max_pages + (p >> c.pshift)];
  if (pid < 0 || pid >= c.pages) {
    raise_fault(b, kFaultPage);
    s.poison = true;
    return s;
  }
  s.ok = true;
  s.page = pid;
  s.off = (int)(p & ((1 << c.pshift) - 1));
  return s;
}

template <int D>
__global__ __launch_bounds__(KT) void k_kv_write(Heads k, Heads v, KvView c, BatchView b, int bl, int zero, ThrLut lut) {
  constexpr int LR = D / 8, NT = KT / LR;   // lanes per row, rows per workgroup
  __shared__ float2 slut[kLutBins];
  __shared__ int own[NT];
  if (threadIdx.x < kLutBins) slut[threadIdx.x] = make_float2(lut.t[threadIdx.x], __uint_as_float(lut.base[threadIdx.x]));
  const int r = threadIdx.x / LR, e = threadIdx.x % LR;
  const int64_t t0 = (int64_t)blockIdx.x * NT;
  const Slot<D> s = find_slot<D>(b, c, t0, r, own);
  if (!s.ok) return;
  const int nb = LR >> bl;   // blocks per row (1 << bl lanes each)
  const uint16_t* const kp = k.data + (t0 + r) * k.rs + e * 8;
  const uint16_t* const vp = v.data + (t0 + r) * v.rs + e * 8;
  const int64_t row0 = ((s.page * c.heads) << c.pshift) + s.off;   // of head 0, in the cache's buffers
  uint8_t* const kcp = c.kc + row0 * (D / 2) + 4 * key_dword<D>(e);
  uint8_t* const vcp = c.vc + row0 * (D / 2) + 4 * e;
  uint16_t* const ksp = c.ks + row0 * nb + (e >> bl);
  uint16_t* const vsp = c.vs + row0 * nb + (e >> bl);
  auto load = [&](int item) {
    return *reinterpret_cast<const uint4*>(item < c.heads ? kp + item * k.hs : vp + (item - c.heads) * v.hs);
  };
  uint4 next = load(blockIdx.y);
  for (int item = blockIdx.y; item < 2 * c.heads; item += gridDim.y) {
    const bool key = item < c.heads;
    const int h = key ? item : item - c.heads;
    const uint4 w = next;
    if (item + (int)gridDim.y < 2 * c.heads) next = load(item + gridDim.y);   // the next head's row, a head ahead
    uint32_t u[8] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16, w.z & 0xFFFFu, w.z >> 16, w.w & 0xFFFFu, w.w >> 16};
    // largest magnitude: on bf16 bit patterns the magnitude order is the integer order
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7FFFu);
    // over the block's lanes: 1 and 2 away, then the other half of 8 and of 16 (mirrored)
    m = dpp_max<0xB1>(m);
    m = dpp_max<0x4E>(m);
    if (bl >= 3) m = dpp_max<0x141>(m);
    if (bl >= 4) m = dpp_max<0x140>(m);
    if (m < 0x0080u) m = 0;   // below the smallest normal: a zero block
    uint32_t scale = m;
    if (m >= 0x7F80u) {       // an infinity or a NaN: the block reads back as NaN
      scale = kBf16NaN;
      m = 0;
    }
    // correctly rounded fp32 reciprocal (a float64 quotient rounded to fp32 is exact-rounded)
    const float inv = m ? (float)(1.0 / (double)bf16_to_f32(m)) : 0.0f;
    uint32_t packed = 0;
    if (m) {
      uint32_t cd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) cd[i] = lut_encode(__fmul_rn(bf16_to_f32(u[i]), inv), slut);
#pragma unroll
      for (int i = 0; i < 4; ++i) packed |= (cd[i] | (cd[i + 4] << 4)) << (8 * i);
    } else {
      packed = (uint32_t)zero * 0x11111111u;
    }
    const int64_t ahead = (int64_t)h << c.pshift;   // rows from head 0's
    *reinterpret_cast<uint32_t*>((key ? kcp : vcp) + ahead * (D / 2)) = packed;
    if ((e & ((1 << bl) - 1)) == 0) (key ? ksp : vsp)[ahead * nb] = (uint16_t)scale;
  }
}

template <int D>
__global__ __launch_bounds__(KT) void k_kv_read(Heads k, Heads v, KvView c, BatchView b, int bl, NF4Table tab) {
  constexpr int LR = D / 8, NT = KT / LR;
  // 16 levels in 16 LDS banks: the lanes of a wave read any mix of them without a conflict
  __shared__ float lv[16];
  __shared__ int own[NT];
  if (threadIdx.x < 16) lv[threadIdx.x] = tab.level[threadIdx.x];
  const int r = threadIdx.x / LR, e = threadIdx.x % LR;
  const int64_t t0 = (int64_t)blockIdx.x * NT;
  const Slot<D> s = find_slot<D>(b, c, t0, r, own);
  if (!s.ok && !s.poison && !s.empty) return;
  const int nb = LR >> bl;
  for (int item = blockIdx.y; item < 2 * c.heads; item += gridDim.y) {
    const bool key = item < c.heads;
    const int h = key ? item : item - c.heads;
    const Heads& x = key ? k : v;
    uint4 o;
    if (s.ok) {
      const int64_t row = ((s.page * c.heads + h) << c.pshift) + s.off;
      const uint8_t* codes = (key ? c.kc : c.vc) + row * (D / 2);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + 4 * (key ? key_dword<D>(e) : e));
      const float sc = bf16_to_f32((key ? c.ks : c.vs)[row * nb + (e >> bl)]);
      uint32_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int sh = 16 * (i & 1) + 4 * (i >> 1);   // elements 2i, 2i + 1: bytes 2(i % 2), + 1; high nibbles from 4 on
        d[i] = pack_bf16x2(__fmul_rn(lv[(w >> sh) & 15u], sc), __fmul_rn(lv[(w >> (sh + 8)) & 15u], sc));
      }
      o = make_uint4(d[0], d[1], d[2], d[3]);
    } else {
      const uint32_t f = s.poison ? kBf16NaN * 0x10001u : 0u;
      o = make_uint4(f, f, f, f);
    }
    *reinterpret_cast<uint4*>(x.data + (t0 + r) * x.rs + h * x.hs + e * 8) = o;
  }
}

// Workgroups of one head pair and NT rows each, up to 8 per CU; past that each takes several heads, so
// that the slots are looked up less often.
dim3 kv_grid(int64_t rows, int nt, int heads) {
  const int64_t gx = (rows + nt - 1) / nt;
  int64_t gy = (2048 + gx - 1) / gx;
  if (gy > 2 * heads) gy = 2 * heads;
  return dim3((unsigned)gx, (unsigned)gy);
}

int lanes_log2(int block) { return block == 32 ? 2 : block == 64 ? 3 : 4; }   // block / 8 lanes

}  // namespace

hipError_t launch_kv_write(const Heads& k, const Heads& v, const KvView& c, const BatchView& b, int D, int block,
                           hipStream_t s) {
  ProfScope ps("k_kv_write", s);
  const dim3 g = kv_grid(b.rows, KT / (D / 8), c.heads);
  const int bl = lanes_log2(block);
  const ThrLut& lut = thr_lut_host(c.cb);
  int zero = 0;   // the code of the table's exact zero
  while (codebook_levels_host(c.cb)[zero] != 0.0f) ++zero;
  if (D == 64) hipLaunchKernelGGL(k_kv_write<64>, g, dim3(KT), 0, s, k, v, c, b, bl, zero, lut);
  else if (D == 128) hipLaunchKernelGGL(k_kv_write<128>, g, dim3(KT), 0, s, k, v, c, b, bl, zero, lut);
  else hipLaunchKernelGGL(k_kv_write<256>, g, dim3(KT), 0, s, k, v, c, b, bl, zero, lut);
  return hipGetLastError();
}

hipError_t launch_kv_read(const Heads& k, const Heads& v, const KvView& c, const BatchView& b, int D, int block,
                          hipStream_t s) {
  ProfScope ps("k_kv_read", s);
  const dim3 g = kv_grid(b.rows, KT / (D / 8), c.heads);
  const int bl = lanes_log2(block);
  const NF4Table tab = nf4_table(c.cb);
  if (D == 64) hipLaunchKernelGGL(k_kv_read<64>, g, dim3(KT), 0, s, k, v, c, b, bl, tab);
  else if (D == 128) hipLaunchKernelGGL(k_kv_read<128>, g, dim3(KT), 0, s, k, v, c, b, bl, tab);
  else hipLaunchKernelGGL(k_kv_read<256>, g, dim3(KT), 0, s, k, v, c, b, bl, tab);
  return hipGetLastError();
}

}  // namespace qlora
