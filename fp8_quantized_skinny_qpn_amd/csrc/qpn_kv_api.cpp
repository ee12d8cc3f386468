// qpn_kv_api.cpp -- the C ABI declared in include/qpn_kv.h and qpn_kv4.h: host-side argument
// checks and launches.  Every check runs before anything is enqueued; nothing
// here allocates, copies, synchronises or prints.
#include "qpn_kv.h"
#include "qpn_kv4.h"

#include <cmath>

#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace {

using namespace qpn;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int status_of(hipError_t e) { return e == hipSuccess ? QPN_OK : QPN_ERR_LAUNCH; }

bool dim_ok(int dim) { return dim == 64 || dim == 128 || dim == 256; }

bool heads_ok(int q_heads, int heads) {
  return heads >= 1 && heads <= kKvMaxHeads && q_heads >= 1 && q_heads % heads == 0 &&
         q_heads / heads <= kKvMaxGroup;
}

int cache_check(const qpn_kv_cache* c) {
  if (!c) return QPN_ERR_NULL;
  if (!dim_ok(c->dim) || c->heads < 1 || c->heads > kKvMaxHeads || c->pages < 1 || c->pages > kKvMaxPages)
    return QPN_ERR_SHAPE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return QPN_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return QPN_ERR_ALIGN;
  return QPN_OK;
}

int cache_check(const qpn_kv4_cache* c) {
  if (!c) return QPN_ERR_NULL;
  if (!dim_ok(c->dim) || c->heads < 1 || c->heads > kKvMaxHeads || c->pages < 1 || c->pages > kKvMaxPages)
    return QPN_ERR_SHAPE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_unit || !c->v_unit) return QPN_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->k_unit, 4) || !aligned(c->v_unit, 4))
    return QPN_ERR_ALIGN;
  return QPN_OK;
}

KvCache4 cache_of(const qpn_kv4_cache* c) {
  return {(uint8_t*)c->k, (uint8_t*)c->v, (uint8_t*)c->k_scale, (uint8_t*)c->v_scale, c->k_unit, c->v_unit, c->pages,
          c->heads, c->dim};
}

KvCache cache_of(const qpn_kv_cache* c) {
  return {(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->pages, c->heads, c->dim};
}

template <typename Cache, typename Launch>
int rope_append(Launch launch, const Cache* cache, const uint16_t* qkv, int64_t qkv_stride, int rows, int q_heads,
                const uint16_t* q_weight, const uint16_t* k_weight, double eps, const float* inv_freq,
                int rot, int interleaved, const int32_t* positions, const int32_t* slots, uint16_t* q_out,
                int64_t q_stride, void* stream) {
  int rc = cache_check(cache);
  if (rc != QPN_OK) return rc;
  if (rows < 0 || rows > kKvMaxRows || !heads_ok(q_heads, cache->heads) || rot < 0 || rot > cache->dim ||
      rot % 16 != 0 || !(eps >= 0.0) || !std::isfinite(eps))
    return QPN_ERR_SHAPE;
  const int64_t dim = cache->dim;
  if (qkv_stride < (q_heads + 2 * (int64_t)cache->heads) * dim || qkv_stride % 8 != 0 ||
      q_stride < q_heads * dim || q_stride % 8 != 0)
    return QPN_ERR_SHAPE;
  if (rows == 0) return QPN_OK;
  // a launch has less than 2^32 threads: those of the cache are up to 64 for a row and head
  if ((int64_t)rows * (cache->heads + q_heads) > (int64_t(1) << 30) ||
      (int64_t)rows * cache->heads > (int64_t(1) << 25))
    return QPN_ERR_SHAPE;
  if (!qkv || !q_out || !positions || !slots || (rot > 0 && !inv_freq)) return QPN_ERR_NULL;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(inv_freq, 4) || !aligned(positions, 4) || !aligned(slots, 4))
    return QPN_ERR_ALIGN;
  rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch({cache_of(cache), qkv, qkv_stride, rows, q_heads, q_weight, k_weight, eps, inv_freq, rot,
                           interleaved != 0, positions, slots, q_out, q_stride, stream}));
}

template <typename Cache, typename Launch>
int attention(Launch launch, const Cache* cache, const uint16_t* q, int64_t q_stride, uint16_t* y, int64_t y_stride,
              int q_heads, int rows, int requests, int max_rows, const int32_t* row_start, const int32_t* seq_lens,
              const int32_t* table, int64_t table_stride, int table_width, float scale, int window, void* scratch,
              size_t scratch_bytes, void* stream) {
  int rc = cache_check(cache);
  if (rc != QPN_OK) return rc;
  if (rows < 0 || rows > kKvMaxRows || requests < 0 || requests > kKvMaxRequests || max_rows < 0 ||
      max_rows > kKvMaxRows || !heads_ok(q_heads, cache->heads) || table_width < 0 || table_width > kKvMaxPages ||
      table_stride < table_width || !(scale > 0.0f) || !std::isfinite(scale) || window < 0)
    return QPN_ERR_SHAPE;
  const int64_t dim = cache->dim;
  if (q_stride < q_heads * dim || q_stride % 8 != 0 || y_stride < q_heads * dim || y_stride % 4 != 0)
    return QPN_ERR_SHAPE;
  if (rows == 0 || requests == 0) return QPN_OK;
  if ((int64_t)rows * q_heads > (int64_t(1) << 30)) return QPN_ERR_SHAPE;  // segments are counted in 31 bits
  if (!q || !y || !row_start || !seq_lens || (table_width > 0 && !table)) return QPN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(y, 8) || !aligned(row_start, 4) || !aligned(seq_lens, 4) || !aligned(table, 4) ||
      !aligned(scratch, 16))
    return QPN_ERR_ALIGN;
  if (!scratch) scratch_bytes = 0;
  rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch({cache_of(cache), q, q_stride, y, y_stride, q_heads, rows, requests, max_rows, row_start,
                           seq_lens, table, table_stride, table_width, scale, window, scratch, scratch_bytes, stream}));
}

}  // namespace

int qpn_kv_plan_round(const int32_t* before, const int32_t* rows, const int32_t* held, int requests,
                      int32_t* table, int64_t table_stride, int table_width, const int32_t* free_pages,
                      int64_t free_capacity, const int32_t* free_count, int capacity, int32_t* seq_lens,
                      int32_t* row_start, int32_t* held_out, int32_t* free_count_out, int32_t* slots,
                      int32_t* positions, void* stream) {
  if (requests < 0 || requests > kKvMaxRequests || capacity < 0 || capacity > kKvMaxRows || table_width < 0 ||
      table_width > kKvMaxPages || table_stride < table_width || free_capacity < 0 || free_capacity > kKvMaxPages)
    return QPN_ERR_SHAPE;
  if (!row_start || !free_count || !free_count_out) return QPN_ERR_NULL;
  if (requests > 0 && (!before || !rows || !held || !seq_lens || !held_out)) return QPN_ERR_NULL;
  if (requests > 0 && table_width > 0 && !table) return QPN_ERR_NULL;
  if (free_capacity > 0 && !free_pages) return QPN_ERR_NULL;
  if (capacity > 0 && (!slots || !positions)) return QPN_ERR_NULL;
  for (const void* p : {(const void*)before, (const void*)rows, (const void*)held, (const void*)table,
                        (const void*)free_pages, (const void*)free_count, (const void*)seq_lens,
                        (const void*)row_start, (const void*)held_out, (const void*)free_count_out,
                        (const void*)slots, (const void*)positions})
    if (!aligned(p, 4)) return QPN_ERR_ALIGN;
  const int rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch_plan_round({before, rows, held, requests, table, table_stride, table_width, free_pages,
                                      free_capacity, free_count, capacity, seq_lens, row_start, held_out,
                                      free_count_out, slots, positions, stream}));
}

int qpn_kv_rope_append(const qpn_kv_cache* cache, const uint16_t* qkv, int64_t qkv_stride, int rows, int q_heads,
                       const uint16_t* q_weight, const uint16_t* k_weight, double eps, const float* inv_freq,
                       int rot, int interleaved, const int32_t* positions, const int32_t* slots, uint16_t* q_out,
                       int64_t q_stride, void* stream) {
  return rope_append(launch_rope_append, cache, qkv, qkv_stride, rows, q_heads, q_weight, k_weight, eps,
                     inv_freq, rot, interleaved, positions, slots, q_out, q_stride, stream);
}

size_t qpn_kv_attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim,
                                      int table_width) {
  if (requests < 0 || requests > kKvMaxRequests || max_rows < 0 || max_rows > kKvMaxRows ||
      !heads_ok(q_heads, heads) || !dim_ok(dim) || table_width < 0 || table_width > kKvMaxPages)
    return (size_t)-1;
  return attention_scratch_bytes(requests, max_rows, q_heads, heads, dim, table_width);
}

int qpn_kv_attention(const qpn_kv_cache* cache, const uint16_t* q, int64_t q_stride, uint16_t* y, int64_t y_stride,
                     int q_heads, int rows, int requests, int max_rows, const int32_t* row_start,
                     const int32_t* seq_lens, const int32_t* table, int64_t table_stride, int table_width,
                     float scale, int window, void* scratch, size_t scratch_bytes, void* stream) {
  return attention(launch_attention, cache, q, q_stride, y, y_stride, q_heads, rows, requests, max_rows, row_start,
                   seq_lens, table, table_stride, table_width, scale, window, scratch, scratch_bytes, stream);
}

int qpn_kv4_rope_append(const qpn_kv4_cache* cache, const uint16_t* qkv, int64_t qkv_stride, int rows, int q_heads,
                        const uint16_t* q_weight, const uint16_t* k_weight, double eps, const float* inv_freq,
                        int rot, int interleaved, const int32_t* positions, const int32_t* slots, uint16_t* q_out,
                        int64_t q_stride, void* stream) {
  return rope_append(launch_rope_append4, cache, qkv, qkv_stride, rows, q_heads, q_weight, k_weight, eps,
                     inv_freq, rot, interleaved, positions, slots, q_out, q_stride, stream);
}

int qpn_kv4_read(const qpn_kv4_cache* cache, const int32_t* slots, int rows, uint16_t* k_out, int64_t k_stride,
                 uint16_t* v_out, int64_t v_stride, void* stream) {
  int rc = cache_check(cache);
  if (rc != QPN_OK) return rc;
  const int64_t width = (int64_t)cache->heads * cache->dim;
  // (a launch has less than 2^32 threads: up to 32 for a row and head)
  if (rows < 0 || rows > kKvMaxRows || (int64_t)rows * cache->heads > (int64_t(1) << 25) || k_stride < width ||
      k_stride % 8 != 0 || v_stride < width || v_stride % 8 != 0)
    return QPN_ERR_SHAPE;
  if (rows == 0) return QPN_OK;
  if (!slots || !k_out || !v_out) return QPN_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return QPN_ERR_ALIGN;
  rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch_read4({cache_of(cache), slots, rows, k_out, k_stride, v_out, v_stride, stream}));
}

size_t qpn_kv4_attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim,
                                       int table_width) {
  if (requests < 0 || requests > kKvMaxRequests || max_rows < 0 || max_rows > kKvMaxRows ||
      !heads_ok(q_heads, heads) || !dim_ok(dim) || table_width < 0 || table_width > kKvMaxPages)
    return (size_t)-1;
  return attention4_scratch_bytes(requests, max_rows, q_heads, heads, dim, table_width);
}

int qpn_kv4_attention(const qpn_kv4_cache* cache, const uint16_t* q, int64_t q_stride, uint16_t* y, int64_t y_stride,
                      int q_heads, int rows, int requests, int max_rows, const int32_t* row_start,
                      const int32_t* seq_lens, const int32_t* table, int64_t table_stride, int table_width,
                      float scale, int window, void* scratch, size_t scratch_bytes, void* stream) {
  return attention(launch_attention4, cache, q, q_stride, y, y_stride, q_heads, rows, requests, max_rows, row_start,
                   seq_lens, table, table_stride, table_width, scale, window, scratch, scratch_bytes, stream);
}

size_t qpn_kv_verify_scratch_bytes(int rows, int requests, int64_t n) {
  if (rows < 0 || rows > 65535 || requests < 0 || requests > kKvMaxRequests || n < 1 || n > kMaxN) return (size_t)-1;
  return verify_scratch_bytes(rows, requests, n);
}

int qpn_kv_verify_sampled(const uint16_t* logits, int64_t logits_stride, const uint16_t* draft_logits,
                          int64_t draft_stride, const int32_t* tokens, const int32_t* row_start, int rows,
                          int requests, int64_t n, double inv_temperature, const float* accept_u,
                          const float* sample_u, int32_t* accepted, int32_t* next, float* accept_prob,
                          void* scratch, size_t scratch_bytes, void* stream) {
  if (rows < 0 || rows > 65535 || requests < 0 || requests > kKvMaxRequests || n < 1 || n > kMaxN ||
      !(inv_temperature > 0.0) || !std::isfinite(inv_temperature))
    return QPN_ERR_SHAPE;
  if (logits_stride < n || (draft_logits && draft_stride < n)) return QPN_ERR_SHAPE;
  if (requests == 0) return QPN_OK;
  if (!row_start || !accepted || !next || !scratch || !sample_u) return QPN_ERR_NULL;
  if (rows > 0 && (!logits || !tokens || !accept_u || !accept_prob)) return QPN_ERR_NULL;
  for (const void* p : {(const void*)tokens, (const void*)row_start, (const void*)accept_u, (const void*)sample_u,
                        (const void*)accepted, (const void*)next, (const void*)accept_prob})
    if (!aligned(p, 4)) return QPN_ERR_ALIGN;
  if (!aligned(logits, 2) || !aligned(draft_logits, 2) || !aligned(scratch, 16)) return QPN_ERR_ALIGN;
  if (scratch_bytes < verify_scratch_bytes(rows, requests, n)) return QPN_ERR_BUFFER;
  const int rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch_verify({logits, logits_stride, draft_logits, draft_stride, tokens, row_start, rows,
                                  requests, n, inv_temperature, accept_u, sample_u, accepted, next, accept_prob,
                                  scratch, stream}));
}

size_t qpn_kv_logprobs_scratch_bytes(int rows, int64_t n) {
  if (rows < 0 || rows > 65535 || n < 1 || n > kMaxN) return (size_t)-1;
  return logprobs_scratch_bytes(rows, n);
}

int qpn_kv_logprobs(const uint16_t* logits, int64_t logits_stride, const int32_t* tokens, int rows, int64_t n,
                    double inv_temperature, int top, float* logprob, float* entropy, int32_t* top_ids,
                    float* top_logprobs, void* scratch, size_t scratch_bytes, void* stream) {
  if (rows < 0 || rows > 65535 || n < 1 || n > kMaxN || top < 0 || top > kLogprobsMaxTop || top > n ||
      logits_stride < n || !(inv_temperature > 0.0) || !std::isfinite(inv_temperature))
    return QPN_ERR_SHAPE;
  if (rows == 0) return QPN_OK;
  if (!logits || !tokens || !logprob || !entropy || !scratch || (top > 0 && (!top_ids || !top_logprobs)))
    return QPN_ERR_NULL;
  for (const void* p : {(const void*)tokens, (const void*)logprob, (const void*)entropy, (const void*)top_ids,
                        (const void*)top_logprobs})
    if (!aligned(p, 4)) return QPN_ERR_ALIGN;
  if (!aligned(logits, 2) || !aligned(scratch, 16)) return QPN_ERR_ALIGN;
  if (scratch_bytes < logprobs_scratch_bytes(rows, n)) return QPN_ERR_BUFFER;
  const int rc = device_status();
  if (rc != QPN_OK) return rc;
  return status_of(launch_logprobs({logits, logits_stride, tokens, rows, n, inv_temperature, top, logprob, entropy,
                                    top_ids, top_logprobs, scratch, stream}));
}
