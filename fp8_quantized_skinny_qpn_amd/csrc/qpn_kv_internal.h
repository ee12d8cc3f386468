// qpn_kv_internal.h -- launchers of the speculative-round operators, shared
// between their C-ABI layer and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qpn {

constexpr int kKvPage = 64;               // tokens of a page
constexpr int64_t kKvMaxPages = (int64_t(1) << 25) - 1;  // slots fit 31 bits
constexpr int kKvMaxHeads = 1024;
constexpr int kKvMaxGroup = 64;           // query heads per KV head
constexpr int kKvMaxRequests = 4096;
constexpr int kKvMaxRows = 1 << 20;
constexpr size_t kKvZeroedBytes = 65536;  // counters at the head of a scratch

// The cache of one layer on the device (layout: include/qpn_kv.h).
struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int heads;
  int dim;
};

struct PlanRoundArgs {
  const int32_t *before, *rows, *held;
  int requests;
  int32_t* table;
  int64_t table_stride;
  int table_width;
  const int32_t* free_pages;
  int64_t free_capacity;
  const int32_t* free_count;
  int capacity;
  int32_t *seq_lens, *row_start, *held_out, *free_count_out, *slots, *positions;
  void* stream;
};
hipError_t launch_plan_round(const PlanRoundArgs& a);

struct RopeAppendArgs {
  KvCache cache;
  const uint16_t* qkv;
  int64_t qkv_stride;
  int rows, q_heads;
  const uint16_t *q_weight, *k_weight;
  double eps;
  const float* inv_freq;
  int rot, interleaved;
  const int32_t *positions, *slots;
  uint16_t* q_out;
  int64_t q_stride;
  void* stream;
};
hipError_t launch_rope_append(const RopeAppendArgs& a);

struct AttentionArgs {
  KvCache cache;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* y;
  int64_t y_stride;
  int q_heads, rows, requests, max_rows;
  const int32_t *row_start, *seq_lens, *table;
  int64_t table_stride;
  int table_width;
  float scale;
  int window;
  void* scratch;
  size_t scratch_bytes;
  void* stream;
};
size_t attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim,
                               int table_width);
hipError_t launch_attention(const AttentionArgs& a);

struct VerifyArgs {
  const uint16_t* logits;
  int64_t logits_stride;
  const uint16_t* draft_logits;
  int64_t draft_stride;
  const int32_t *tokens, *row_start;
  int rows, requests;
  int64_t n;
  double inv_temperature;
  const float *accept_u, *sample_u;
  int32_t *accepted, *next;
  float* accept_prob;
  void* scratch;
  void* stream;
};
size_t verify_scratch_bytes(int rows, int requests, int64_t n);
hipError_t launch_verify(const VerifyArgs& a);

// QPN_OK when the current device can run the library's kernels.
int device_status();

}  // namespace qpn
