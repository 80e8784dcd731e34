// attn_params.h -- parameter blocks shared by the host side (attn_api.cpp) and
// the kernels of the attention operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace agmm {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxAxes = 4;

struct NormRopeParams {
  const uint16_t* qkv;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const void* positions;
  uint16_t* q;
  uint16_t* k;
  uint16_t* k_cache;
  uint16_t* v_cache;
  const int64_t* slots;
  int64_t tokens;
  int64_t qkv_ts, qkv_hs, q_ts, q_hs, k_ts, k_hs;  // token and head strides, elements
  int64_t cache_ps, cache_ts, cache_hs;            // page, place and head strides
  int64_t num_slots, position_axis_stride;
  int q_heads, kv_heads, pairs, page_size;
  int page_shift;  // log2(page_size), or -1
  int adjacent, position64;
  float eps;
  double turns[kMaxHeadDim / 2];      // inv_freq / (2 pi): turns per position
  uint8_t axis[kMaxHeadDim / 2];      // position axis of each pair
};

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, bool f16, cudaStream_t stream);

// One attention problem.  Prompts: packed rows, `paged` false.  Trees: a
// paged cache.
struct AttnParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  const int32_t* starts;     // query rows of each sequence (nodes of a tree)
  const int32_t* kv_starts;  // prompts: key rows of each sequence
  const int32_t* context_lens;
  const int32_t* page_table;
  const int64_t* mask;
  int64_t tokens, kv_tokens, sequences;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, out_ts, out_hs;
  int64_t page_stride, table_stride, pages;
  int mask_words, page_shift;
  int q_heads, kv_heads, causal, max_nodes;
  float scale;
};

cudaError_t launch_attention(const AttnParams& p, int head_dim, bool f16, bool paged, cudaStream_t stream);

}  // namespace agmm
