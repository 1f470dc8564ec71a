// Entry points between the projections: head norms and rotation, the 4-bit key/value cache, and the
// attention over it (include/qlora.h).  Validates every argument on the host, then launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "host.h"
#include "kernels.h"
#include "kv.h"
#include "qlora.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int64_t kMaxStride = int64_t(1) << 36;   // times the most rows: offsets stay within 62 bits
constexpr int32_t kMaxHeads = 1024;

bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

// One view of rows x heads x head_dim.  `out`: rows must not overlap.
qlora_status check_heads(const qlora_heads* x, int64_t rows, int32_t dim, bool out) {
  if (!x) return QLORA_ERR_NULL;
  if (x->heads < 1 || x->heads > kMaxHeads) return QLORA_ERR_SHAPE;
  if (rows > 0 && !x->data) return QLORA_ERR_NULL;
  if (!aligned16(x->data)) return QLORA_ERR_ALIGN;
  const int64_t rs = x->row_stride, hs = x->head_stride;
  if (rs < 0 || hs < 0 || rs >= kMaxStride || hs >= kMaxStride) return QLORA_ERR_SHAPE;
  if ((rows > 1 && rs % 8 != 0) || (x->heads > 1 && hs % 8 != 0)) return QLORA_ERR_ALIGN;
  if (out && rows > 0) {
    const int64_t hspan = x->heads > 1 ? (x->heads - 1) * hs + dim : dim;
    const int64_t rspan = rows > 1 ? (rows - 1) * rs + dim : dim;
    const bool row_major = (x->heads == 1 || hs >= dim) && (rows == 1 || rs >= hspan);
    const bool head_major = (rows == 1 || rs >= dim) && (x->heads == 1 || hs >= rspan);
    if (!row_major && !head_major) return QLORA_ERR_SHAPE;
  }
  return QLORA_OK;
}

Heads heads_of(const qlora_heads* x) { return x ? Heads{x->data, x->row_stride, x->head_stride, x->heads} : Heads{nullptr, 0, 0, 0}; }

int cache_block(const qlora_kv_cache* c) { return c->block_size == 0 ? 64 : c->block_size; }

// the sizes of a cache, not its buffers
qlora_status check_cache_sizes(const qlora_kv_cache* c) {
  if (!c) return QLORA_ERR_NULL;
  if (!head_dim_ok(c->head_dim)) return QLORA_ERR_UNSUPPORTED;
  const int b = cache_block(c);
  if ((b != 32 && b != 64 && b != 128) || b > c->head_dim) return QLORA_ERR_UNSUPPORTED;
  if (c->codebook < 0 || c->codebook >= kNumCodebooks) return QLORA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1))) return QLORA_ERR_UNSUPPORTED;
  if (c->heads < 1 || c->heads > kMaxHeads || c->pages < 1 || c->pages >= (int64_t(1) << 31)) return QLORA_ERR_SHAPE;
  // a page's offsets are 32-bit
  if ((int64_t)c->heads * c->page_size * c->head_dim >= (int64_t(1) << 32)) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

qlora_status check_cache(const qlora_kv_cache* c) {
  const qlora_status st = check_cache_sizes(c);
  if (st != QLORA_OK) return st;
  if (!c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale) return QLORA_ERR_NULL;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scale) || !aligned16(c->v_codes) || !aligned16(c->v_scale))
    return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

KvView cache_view(const qlora_kv_cache* c) {
  KvView v;
  v.kc = c->k_codes;
  v.ks = c->k_scale;
  v.vc = c->v_codes;
  v.vs = c->v_scale;
  v.pages = c->pages;
  v.heads = c->heads;
  v.pshift = __builtin_ctz((unsigned)c->page_size);
  v.cb = c->codebook;
  return v;
}

qlora_status check_batch_sizes(const qlora_kv_batch* b, const qlora_kv_cache* c) {
  if (!b) return QLORA_ERR_NULL;
  if (b->batch < 0 || b->batch > 65536 || b->max_pages < 1) return QLORA_ERR_SHAPE;
  // token indexes a few tiles past the last one, and sums of a position and a window, stay within 32 bits
  if ((int64_t)b->max_pages * c->page_size > kMaxTokens) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

qlora_status check_batch(const qlora_kv_batch* b, const qlora_kv_cache* c) {
  const qlora_status st = check_batch_sizes(b, c);
  if (st != QLORA_OK) return st;
  if (b->batch > 0 && (!b->start || !b->length || !b->table)) return QLORA_ERR_NULL;
  if (!aligned4(b->start) || !aligned4(b->length) || !aligned4(b->table) || !aligned4(b->fault)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

BatchView batch_view(const qlora_kv_batch* b, const qlora_kv_cache* c, int64_t rows) {
  BatchView v;
  v.start = b->start;
  v.length = b->length;
  v.table = b->table;
  v.fault = b->fault;
  v.rows = rows;
  v.batch = b->batch;
  v.max_pages = b->max_pages;
  v.max_len = b->max_pages * c->page_size;
  return v;
}

// What forward and backward of the norm and rotation share.
qlora_status check_qk(int64_t rows, int32_t dim, const uint16_t* wq, const uint16_t* wk, float eps, const int64_t* pos,
                      const float* freq, int32_t rot, int32_t inter) {
  if (!head_dim_ok(dim)) return QLORA_ERR_UNSUPPORTED;
  if (rows < 0 || rows >= kMaxRows) return QLORA_ERR_SHAPE;
  if (rot < 0 || rot > dim || rot % 16 != 0) return QLORA_ERR_SHAPE;
  if (inter != 0 && inter != 1) return QLORA_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return QLORA_ERR_UNSUPPORTED;
  if (rot > 0 && rows > 0 && (!pos || !freq)) return QLORA_ERR_NULL;
  if (!aligned16(wq) || !aligned16(wk) || !aligned8(pos) || !aligned4(freq)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// Rows of q and k of one cache write or read.
qlora_status check_kv_rows(const qlora_heads* k, const qlora_heads* v, int64_t rows, const qlora_kv_cache* cache,
                           const qlora_kv_batch* batch, bool out) {
  qlora_status st = check_cache(cache);
  if (st != QLORA_OK) return st;
  if ((st = check_batch(batch, cache)) != QLORA_OK) return st;
  if (rows < 0 || rows >= kMaxRows) return QLORA_ERR_SHAPE;
  if ((st = check_heads(k, rows, cache->head_dim, out)) != QLORA_OK) return st;
  if ((st = check_heads(v, rows, cache->head_dim, out)) != QLORA_OK) return st;
  if (k->heads != cache->heads || v->heads != cache->heads) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

AttnPlan plan_of(const qlora_kv_cache* c, const qlora_kv_batch* b, int64_t rows, int32_t q_heads) {
  return attn_plan(rows, q_heads, c->heads, b->batch, (int64_t)b->max_pages * c->page_size, c->head_dim);
}

qlora_status check_attn_sizes(const qlora_kv_cache* c, const qlora_kv_batch* b, int64_t rows, int32_t q_heads) {
  qlora_status st = check_cache_sizes(c);
  if (st != QLORA_OK) return st;
  if ((st = check_batch_sizes(b, c)) != QLORA_OK) return st;
  if (rows < 0 || rows >= kMaxRows || q_heads < 1 || q_heads > kMaxHeads || q_heads % c->heads != 0)
    return QLORA_ERR_SHAPE;
  // rows of one cache head, and their tiles of 16 over all heads: 32-bit indexes
  const int64_t rows_h = rows * (q_heads / c->heads);
  if (rows_h >= (int64_t(1) << 30) || (rows_h / 16 + 1 + b->batch) * c->heads >= (int64_t(1) << 29)) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

struct AttnWs {
  float* part;
  int32_t* meta;
  size_t bytes;
};
AttnWs attn_layout(void* base, const AttnPlan& p) {
  Carve c(base);
  AttnWs w;
  w.part = c.take<float>(p.part_floats);
  w.meta = c.take<int32_t>(p.meta_ints);
  w.bytes = std::max<size_t>(round_up(c.off, 256), 256);   // never 0, which the query gives for sizes that are refused
  return w;
}

}  // namespace

extern "C" {

qlora_status qlora_qk_norm_rope(const qlora_heads* q, const qlora_heads* k, int64_t rows, int32_t head_dim,
                                const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                const int64_t* positions, const float* inv_freq, int32_t rot_dim,
                                int32_t interleaved, const qlora_heads* q_out, const qlora_heads* k_out,
                                hipStream_t stream) {
  qlora_status st = check_qk(rows, head_dim, q_weight, k_weight, eps, positions, inv_freq, rot_dim, interleaved);
  if (st != QLORA_OK) return st;
  if ((k == nullptr) != (k_out == nullptr)) return QLORA_ERR_NULL;
  if ((st = check_heads(q, rows, head_dim, false)) != QLORA_OK) return st;
  if ((st = check_heads(q_out, rows, head_dim, true)) != QLORA_OK) return st;
  if (q->heads != q_out->heads) return QLORA_ERR_SHAPE;
  if (k) {
    if ((st = check_heads(k, rows, head_dim, false)) != QLORA_OK) return st;
    if ((st = check_heads(k_out, rows, head_dim, true)) != QLORA_OK) return st;
    if (k->heads != k_out->heads) return QLORA_ERR_SHAPE;
  }
  if (rows == 0) return QLORA_OK;
  QkArgs a{};
  a.q = heads_of(q);
  a.k = heads_of(k);
  a.qo = heads_of(q_out);
  a.ko = heads_of(k_out);
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.freq = inv_freq;
  a.rows = rows;
  a.eps = eps;
  a.rot = rot_dim;
  QL_HIP(launch_qk(a, head_dim, interleaved != 0, stream));
  return QLORA_OK;
}

size_t qlora_qk_norm_rope_bwd_workspace(int64_t rows, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  if (rows < 0 || rows >= kMaxRows || q_heads < 1 || q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads ||
      !head_dim_ok(head_dim))
    return 0;
  return round_up((size_t)qk_bwd_partials(std::max<int64_t>(rows, 1), q_heads, k_heads, head_dim) * 2 * head_dim * sizeof(float),
                  256);
}

qlora_status qlora_qk_norm_rope_bwd(const qlora_heads* dq_out, const qlora_heads* dk_out, const qlora_heads* q,
                                    const qlora_heads* k, int64_t rows, int32_t head_dim, const uint16_t* q_weight,
                                    const uint16_t* k_weight, float eps, const int64_t* positions,
                                    const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                                    const qlora_heads* dq, const qlora_heads* dk, float* dq_weight,
                                    float* dk_weight, void* ws, size_t ws_bytes, hipStream_t stream) {
  qlora_status st = check_qk(rows, head_dim, q_weight, k_weight, eps, positions, inv_freq, rot_dim, interleaved);
  if (st != QLORA_OK) return st;
  if ((dk_out == nullptr) != (dk == nullptr)) return QLORA_ERR_NULL;
  if (!dk_out && (k || k_weight || dk_weight)) return QLORA_ERR_NULL;
  if ((q_weight == nullptr) != (dq_weight == nullptr) || (k_weight == nullptr) != (dk_weight == nullptr))
    return QLORA_ERR_NULL;
  if (!aligned4(dq_weight) || !aligned4(dk_weight)) return QLORA_ERR_ALIGN;
  const struct {
    const qlora_heads *g, *x, *d;
    const uint16_t* w;
  } sides[2] = {{dq_out, q, dq, q_weight}, {dk_out, k, dk, k_weight}};
  for (int i = 0; i < (dk_out ? 2 : 1); ++i) {
    const auto& s = sides[i];
    if ((st = check_heads(s.g, rows, head_dim, false)) != QLORA_OK) return st;
    if ((st = check_heads(s.d, rows, head_dim, true)) != QLORA_OK) return st;
    if (s.g->heads != s.d->heads) return QLORA_ERR_SHAPE;
    if (!s.w) continue;
    if ((st = check_heads(s.x, rows, head_dim, false)) != QLORA_OK) return st;
    if (s.g->heads != s.x->heads) return QLORA_ERR_SHAPE;
  }
  const bool sums = q_weight || k_weight;
  if (sums) {
    const size_t need = qlora_qk_norm_rope_bwd_workspace(rows, dq_out->heads, dk_out ? dk_out->heads : 0, head_dim);
    if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
    if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  }
  if (rows == 0) {
    if (dq_weight) QL_HIP(launch_fill_u32(reinterpret_cast<uint32_t*>(dq_weight), head_dim, 0u, stream));
    if (dk_weight) QL_HIP(launch_fill_u32(reinterpret_cast<uint32_t*>(dk_weight), head_dim, 0u, stream));
    return QLORA_OK;
  }
  QkArgs a{};
  a.q = heads_of(dq_out);
  a.k = heads_of(dk_out);
  a.qo = heads_of(dq);
  a.ko = heads_of(dk);
  a.xq = heads_of(q);
  a.xk = heads_of(k);
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.freq = inv_freq;
  a.rows = rows;
  a.eps = eps;
  a.rot = rot_dim;
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  QL_HIP(launch_qk_bwd(a, head_dim, interleaved != 0, dq_weight, dk_weight, stream));
  return QLORA_OK;
}

qlora_status qlora_kv_sizes(const qlora_kv_cache* c, size_t* codes_bytes, size_t* scale_bytes) {
  const qlora_status st = check_cache_sizes(c);
  if (st != QLORA_OK) return st;
  const size_t rows = (size_t)c->pages * c->heads * c->page_size;
  if (codes_bytes) *codes_bytes = rows * (c->head_dim / 2);
  if (scale_bytes) *scale_bytes = rows * (c->head_dim / cache_block(c)) * 2;
  return QLORA_OK;
}

qlora_status qlora_kv_write(const qlora_heads* k, const qlora_heads* v, int64_t rows, const qlora_kv_cache* cache,
                            const qlora_kv_batch* batch, hipStream_t stream) {
  const qlora_status st = check_kv_rows(k, v, rows, cache, batch, false);
  if (st != QLORA_OK) return st;
  if (rows == 0 || batch->batch == 0) return QLORA_OK;
  QL_HIP(launch_kv_write(heads_of(k), heads_of(v), cache_view(cache), batch_view(batch, cache, rows), cache->head_dim,
                         cache_block(cache), stream));
  return QLORA_OK;
}

qlora_status qlora_kv_read(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int64_t rows,
                           const qlora_heads* k, const qlora_heads* v, hipStream_t stream) {
  const qlora_status st = check_kv_rows(k, v, rows, cache, batch, true);
  if (st != QLORA_OK) return st;
  if (rows == 0 || batch->batch == 0) return QLORA_OK;
  QL_HIP(launch_kv_read(heads_of(k), heads_of(v), cache_view(cache), batch_view(batch, cache, rows), cache->head_dim,
                        cache_block(cache), stream));
  return QLORA_OK;
}

size_t qlora_kv_attn_workspace(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int64_t rows,
                               int32_t q_heads) {
  if (check_attn_sizes(cache, batch, rows, q_heads) != QLORA_OK) return 0;
  return attn_layout(nullptr, plan_of(cache, batch, std::max<int64_t>(rows, 1), q_heads)).bytes;
}

qlora_status qlora_kv_attn(const qlora_heads* q, int64_t rows, const qlora_kv_cache* cache,
                           const qlora_kv_batch* batch, float scale, int32_t causal, int32_t window,
                           const qlora_heads* o, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  qlora_status st = check_cache(cache);
  if (st != QLORA_OK) return st;
  if ((st = check_batch(batch, cache)) != QLORA_OK) return st;
  if (!q || !o) return QLORA_ERR_NULL;
  if ((st = check_attn_sizes(cache, batch, rows, q->heads)) != QLORA_OK) return st;
  if ((st = check_heads(q, rows, cache->head_dim, false)) != QLORA_OK) return st;
  if ((st = check_heads(o, rows, cache->head_dim, true)) != QLORA_OK) return st;
  if (q->heads != o->heads || window < 0) return QLORA_ERR_SHAPE;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return QLORA_ERR_UNSUPPORTED;
  if ((causal != 0 && causal != 1) || (window > 0 && !causal)) return QLORA_ERR_UNSUPPORTED;
  if (!aligned4(lse)) return QLORA_ERR_ALIGN;
  const AttnPlan p = plan_of(cache, batch, std::max<int64_t>(rows, 1), q->heads);
  if (!ws || ws_bytes < attn_layout(nullptr, p).bytes) return QLORA_ERR_WORKSPACE;
  if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  if (rows == 0 || batch->batch == 0) return QLORA_OK;
  const AttnWs w = attn_layout(ws, p);
  AttnArgs a{};
  a.q = heads_of(q);
  a.o = heads_of(o);
  a.lse = lse;
  a.c = cache_view(cache);
  a.b = batch_view(batch, cache, rows);
  a.group = q->heads / cache->heads;
  // 2^s >= group > 2^(s - 1), so the multiplier, 2^(31 + s) / group rounded up, is at most 2^32 - 1 past group 1 and off by
  // less than 1, which an n below 2^31 takes less than 2^31 <= 2^(31 + s) / group of the way to the next quotient
  int s = 0;
  while (1 << s < a.group) ++s;
  a.group_shift = 31 + s;
  a.group_mul = (uint32_t)(((uint64_t(1) << a.group_shift) + a.group - 1) / a.group);
  a.scale = scale;
  a.causal = causal;
  // (a window that no cache of this batch outgrows is none)
  a.window = window < (int64_t)batch->max_pages * cache->page_size ? window : 0;
  a.part = w.part;
  a.meta = w.meta;
  QL_HIP(launch_kv_attn(a, p, cache->head_dim, cache_block(cache), stream));
  return QLORA_OK;
}

}  // extern "C"
