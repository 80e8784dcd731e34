// attn_api.cpp -- the C ABI of include/agmm_attention.h: argument checks,
// plans and launches of the attention operators.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "agmm_attention.h"
#include "attn_params.h"

namespace agmm {
agmm_status_t set_last_error(agmm_status_t status, const char* message);
}

using namespace agmm;

struct agmm_norm_rope_s {
  NormRopeParams params;  // the plan's fields; each run copies it
  int head_dim;
  bool f16;
  int device;
};

struct AttnPlan {
  int q_heads, kv_heads, head_dim, causal, page_size, max_nodes;
  bool f16;
  float scale;
  int device, num_sms;
};
struct agmm_prompt_s : AttnPlan {};
struct agmm_tree_s : AttnPlan {};

namespace {

constexpr size_t kStatusBytes = 256;

agmm_status_t fail(agmm_status_t s, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return set_last_error(s, text);
}

agmm_status_t check_device(int* device, int* num_sms) {
  int major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, *device);
  if (e != cudaSuccess) return fail(AGMM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  if (major != 10 || minor != 3)
    return fail(AGMM_ERR_UNSUPPORTED, "this library is built for sm_103a only; device is sm_%d%d", major, minor);
  return AGMM_OK;
}

agmm_status_t check_heads(int q_heads, int kv_heads, int dtype) {
  if (q_heads < 1 || q_heads > 65536 || kv_heads < 1 || kv_heads > 65536)
    return fail(AGMM_ERR_INVALID_ARG, "q_heads and kv_heads must be in [1, 65536]: %d, %d", q_heads, kv_heads);
  if (dtype != AGMM_BF16 && dtype != AGMM_F16)
    return fail(AGMM_ERR_INVALID_ARG, "dtype must be AGMM_BF16 or AGMM_F16: %d", dtype);
  return AGMM_OK;
}

agmm_status_t check_attention(int q_heads, int kv_heads, int head_dim, int dtype, float scale) {
  agmm_status_t st = check_heads(q_heads, kv_heads, dtype);
  if (st != AGMM_OK) return st;
  if (q_heads % kv_heads)
    return fail(AGMM_ERR_INVALID_ARG, "q_heads (%d) must be a multiple of kv_heads (%d)", q_heads, kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(AGMM_ERR_UNSUPPORTED, "head_dim must be 64 or 128: %d", head_dim);
  if (!std::isfinite(scale)) return fail(AGMM_ERR_INVALID_ARG, "scale is not finite");
  return AGMM_OK;
}

// A matrix operand: there, 16-byte aligned, strides of whole 16-byte pieces.
agmm_status_t check_operand(const char* name, const void* p, int64_t ts, int64_t hs) {
  if (!p) return fail(AGMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (ts < 0 || hs < 0 || ts >= (int64_t)1 << 38 || hs >= (int64_t)1 << 38)
    return fail(AGMM_ERR_INVALID_ARG, "%s: strides out of range", name);
  if ((reinterpret_cast<uintptr_t>(p) & 15) || ts % 8 || hs % 8)
    return fail(AGMM_ERR_ALIGNMENT, "%s must be 16-byte aligned, its strides multiples of 8 elements", name);
  return AGMM_OK;
}

agmm_status_t check_range(const char* name, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi)
    return fail(AGMM_ERR_INVALID_ARG, "%s must be in [%lld, %lld]: %lld", name, (long long)lo, (long long)hi, (long long)v);
  return AGMM_OK;
}

agmm_status_t check_pointer(const char* name, const void* p, size_t align) {
  if (!p) return fail(AGMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align) return fail(AGMM_ERR_ALIGNMENT, "%s is not %zu-byte aligned", name, align);
  return AGMM_OK;
}

int shift_of(int64_t v) {  // log2, or -1
  if (v < 1 || (v & (v - 1))) return -1;
  int s = 0;
  while ((int64_t)1 << s < v) ++s;
  return s;
}

agmm_status_t launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? AGMM_OK : fail(AGMM_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

#define AGMM_TRY(expr)                        \
  do {                                        \
    const agmm_status_t st_ = (expr);         \
    if (st_ != AGMM_OK) return st_;           \
  } while (0)

extern "C" {

// ------------------------------------------------------------------ norm_rope
agmm_status_t agmm_norm_rope_plan(const agmm_norm_rope_desc_t* d, agmm_norm_rope_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  AGMM_TRY(check_heads(d->q_heads, d->kv_heads, d->dtype));
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(AGMM_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256: %d", d->head_dim);
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 16)
    return fail(AGMM_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim]: %d", d->rotary_dim);
  AGMM_TRY(check_range("axes", d->axes, 1, kMaxAxes));
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return fail(AGMM_ERR_INVALID_ARG, "eps must be finite and not negative");
  const int pairs = d->rotary_dim / 2;
  if (pairs && !d->inv_freq) return fail(AGMM_ERR_INVALID_ARG, "inv_freq is NULL");
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(d->inv_freq[i])) return fail(AGMM_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
    if (d->axis_of_pair && (d->axis_of_pair[i] < 0 || d->axis_of_pair[i] >= d->axes))
      return fail(AGMM_ERR_INVALID_ARG, "axis_of_pair[%d] must be in [0, axes): %d", i, d->axis_of_pair[i]);
  }
  int device = 0, sms = 0;
  AGMM_TRY(check_device(&device, &sms));
  agmm_norm_rope_s* pl = new (std::nothrow) agmm_norm_rope_s();
  if (!pl) return fail(AGMM_ERR_NOMEM, "plan allocation");
  NormRopeParams& p = pl->params;
  p.q_heads = d->q_heads;
  p.kv_heads = d->kv_heads;
  p.pairs = pairs;
  p.adjacent = d->adjacent != 0;
  p.eps = d->eps;
  for (int i = 0; i < pairs; ++i) {
    p.turns[i] = d->inv_freq[i] / 6.283185307179586476925;  // 2 pi
    p.axis[i] = (uint8_t)(d->axis_of_pair ? d->axis_of_pair[i] : 0);
  }
  pl->head_dim = d->head_dim;
  pl->f16 = d->dtype == AGMM_F16;
  pl->device = device;
  *out = pl;
  return AGMM_OK;
}

void agmm_norm_rope_destroy(agmm_norm_rope_t plan) { delete plan; }

agmm_status_t agmm_norm_rope_run(agmm_norm_rope_t plan, const agmm_norm_rope_args_t* a, void* stream) {
  if (!plan || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_range("tokens", a->tokens, 0, INT_MAX));
  if (a->tokens == 0) return AGMM_OK;
  AGMM_TRY(check_operand("qkv", a->qkv, a->qkv_token_stride, a->qkv_head_stride));
  AGMM_TRY(check_operand("q", a->q, a->q_token_stride, a->q_head_stride));
  if (a->k) AGMM_TRY(check_operand("k", a->k, a->k_token_stride, a->k_head_stride));
  if (!a->q_weight != !a->k_weight)
    return fail(AGMM_ERR_INVALID_ARG, "q_weight and k_weight are given together or not at all");
  if (a->q_weight) {
    AGMM_TRY(check_pointer("q_weight", a->q_weight, 16));
    AGMM_TRY(check_pointer("k_weight", a->k_weight, 16));
  }
  NormRopeParams p = plan->params;
  if (p.pairs) {
    if (a->position_bytes != 4 && a->position_bytes != 8)
      return fail(AGMM_ERR_INVALID_ARG, "position_bytes must be 4 or 8");
    AGMM_TRY(check_pointer("positions", a->positions, (size_t)a->position_bytes));
    AGMM_TRY(check_range("position_axis_stride", a->position_axis_stride, 0, (int64_t)1 << 38));
  }
  if (!a->k_cache != !a->v_cache)
    return fail(AGMM_ERR_INVALID_ARG, "k_cache and v_cache are given together or not at all");
  if (!a->k && !a->k_cache) return fail(AGMM_ERR_INVALID_ARG, "the keys have no destination: give k, or the caches");
  p.num_slots = 0;
  p.page_size = 1;
  p.page_shift = 0;
  if (a->k_cache) {
    AGMM_TRY(check_operand("k_cache", a->k_cache, a->cache_token_stride, a->cache_head_stride));
    AGMM_TRY(check_operand("v_cache", a->v_cache, a->cache_page_stride, a->cache_head_stride));
    AGMM_TRY(check_range("pages", a->pages, 0, INT_MAX));
    AGMM_TRY(check_range("page_size", a->page_size, 1, 1 << 20));
    AGMM_TRY(check_pointer("slots", a->slots, 8));
    p.num_slots = a->pages * a->page_size;
    p.page_size = (int)a->page_size;
    p.page_shift = shift_of(a->page_size);
  }
  p.qkv = static_cast<const uint16_t*>(a->qkv);
  p.q_weight = static_cast<const uint16_t*>(a->q_weight);
  p.k_weight = static_cast<const uint16_t*>(a->k_weight);
  p.positions = a->positions;
  p.position64 = a->position_bytes == 8;
  p.position_axis_stride = a->position_axis_stride;
  p.q = static_cast<uint16_t*>(a->q);
  p.k = static_cast<uint16_t*>(a->k);
  p.k_cache = static_cast<uint16_t*>(a->k_cache);
  p.v_cache = static_cast<uint16_t*>(a->v_cache);
  p.slots = a->slots;
  p.tokens = a->tokens;
  p.qkv_ts = a->qkv_token_stride;
  p.qkv_hs = a->qkv_head_stride;
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.k_ts = a->k_token_stride;
  p.k_hs = a->k_head_stride;
  p.cache_ps = a->cache_page_stride;
  p.cache_ts = a->cache_token_stride;
  p.cache_hs = a->cache_head_stride;
  return launched(launch_norm_rope(p, plan->head_dim, plan->f16, static_cast<cudaStream_t>(stream)), "norm_rope");
}

// --------------------------------------------------------------------- prompt
agmm_status_t agmm_prompt_plan(const agmm_prompt_desc_t* d, agmm_prompt_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  AGMM_TRY(check_attention(d->q_heads, d->kv_heads, d->head_dim, d->dtype, d->scale));
  int device = 0, sms = 0;
  AGMM_TRY(check_device(&device, &sms));
  agmm_prompt_s* pl = new (std::nothrow) agmm_prompt_s();
  if (!pl) return fail(AGMM_ERR_NOMEM, "plan allocation");
  pl->q_heads = d->q_heads;
  pl->kv_heads = d->kv_heads;
  pl->head_dim = d->head_dim;
  pl->causal = d->causal != 0;
  pl->f16 = d->dtype == AGMM_F16;
  pl->scale = d->scale;
  pl->device = device;
  pl->num_sms = sms;
  *out = pl;
  return AGMM_OK;
}

void agmm_prompt_destroy(agmm_prompt_t plan) { delete plan; }

size_t agmm_prompt_workspace_bytes(agmm_prompt_t plan) { return plan ? kStatusBytes : 0; }

agmm_status_t agmm_prompt_run(agmm_prompt_t plan, const agmm_prompt_args_t* a, void* stream) {
  if (!plan || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_range("tokens", a->tokens, 0, INT_MAX));
  AGMM_TRY(check_range("kv_tokens", a->kv_tokens, 0, INT_MAX));
  AGMM_TRY(check_range("sequences", a->sequences, 0, 1 << 20));
  if (a->tokens == 0 || a->sequences == 0) return AGMM_OK;
  AGMM_TRY(check_operand("q", a->q, a->q_token_stride, a->q_head_stride));
  AGMM_TRY(check_operand("out", a->out, a->out_token_stride, a->out_head_stride));
  if (a->kv_tokens) {
    AGMM_TRY(check_operand("k", a->k, a->k_token_stride, a->k_head_stride));
    AGMM_TRY(check_operand("v", a->v, a->v_token_stride, a->v_head_stride));
  }
  AGMM_TRY(check_pointer("starts", a->starts, 4));
  if (a->kv_starts) AGMM_TRY(check_pointer("kv_starts", a->kv_starts, 4));
  AGMM_TRY(check_pointer("workspace", a->workspace, 16));
  AttnParams p = {};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.starts = a->starts;
  p.kv_starts = a->kv_starts ? a->kv_starts : a->starts;
  p.tokens = a->tokens;
  p.kv_tokens = a->kv_tokens;
  p.sequences = a->sequences;
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.k_ts = a->k_token_stride;
  p.k_hs = a->k_head_stride;
  p.v_ts = a->v_token_stride;
  p.v_hs = a->v_head_stride;
  p.out_ts = a->out_token_stride;
  p.out_hs = a->out_head_stride;
  p.q_heads = plan->q_heads;
  p.kv_heads = plan->kv_heads;
  p.causal = plan->causal;
  p.scale = plan->scale;
  return launched(launch_attention(p, plan->head_dim, plan->f16, false, static_cast<cudaStream_t>(stream)), "prompt");
}

// ----------------------------------------------------------------------- tree
agmm_status_t agmm_tree_plan(const agmm_tree_desc_t* d, agmm_tree_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  AGMM_TRY(check_attention(d->q_heads, d->kv_heads, d->head_dim, d->dtype, d->scale));
  if (d->q_heads / d->kv_heads > 128)
    return fail(AGMM_ERR_UNSUPPORTED, "more than 128 query heads to a key head: %d", d->q_heads / d->kv_heads);
  if (shift_of(d->page_size) < 3 || d->page_size > 256)
    return fail(AGMM_ERR_UNSUPPORTED, "page_size must be a power of two in [8, 256]: %d", d->page_size);
  AGMM_TRY(check_range("max_nodes", d->max_nodes, 1, 1024));
  int device = 0, sms = 0;
  AGMM_TRY(check_device(&device, &sms));
  agmm_tree_s* pl = new (std::nothrow) agmm_tree_s();
  if (!pl) return fail(AGMM_ERR_NOMEM, "plan allocation");
  pl->q_heads = d->q_heads;
  pl->kv_heads = d->kv_heads;
  pl->head_dim = d->head_dim;
  pl->causal = 1;
  pl->page_size = d->page_size;
  pl->max_nodes = d->max_nodes;
  pl->f16 = d->dtype == AGMM_F16;
  pl->scale = d->scale;
  pl->device = device;
  pl->num_sms = sms;
  *out = pl;
  return AGMM_OK;
}

void agmm_tree_destroy(agmm_tree_t plan) { delete plan; }

size_t agmm_tree_workspace_bytes(agmm_tree_t plan) { return plan ? kStatusBytes : 0; }

agmm_status_t agmm_tree_run(agmm_tree_t plan, const agmm_tree_args_t* a, void* stream) {
  if (!plan || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_range("tokens", a->tokens, 0, INT_MAX));
  AGMM_TRY(check_range("sequences", a->sequences, 0, 1 << 20));
  if (a->tokens == 0 || a->sequences == 0) return AGMM_OK;
  AGMM_TRY(check_operand("q", a->q, a->q_token_stride, a->q_head_stride));
  AGMM_TRY(check_operand("out", a->out, a->out_token_stride, a->out_head_stride));
  AGMM_TRY(check_operand("k_cache", a->k_cache, a->cache_token_stride, a->cache_head_stride));
  AGMM_TRY(check_operand("v_cache", a->v_cache, a->cache_page_stride, a->cache_head_stride));
  AGMM_TRY(check_range("pages", a->pages, 1, INT_MAX));
  AGMM_TRY(check_range("table_stride", a->table_stride, 1, INT_MAX / plan->page_size));
  AGMM_TRY(check_pointer("page_table", a->page_table, 4));
  AGMM_TRY(check_pointer("context_lens", a->context_lens, 4));
  AGMM_TRY(check_pointer("node_starts", a->node_starts, 4));
  if (a->mask) {
    AGMM_TRY(check_pointer("mask", a->mask, 8));
    AGMM_TRY(check_range("mask_words", a->mask_words, (plan->max_nodes + 63) / 64, 1 << 20));
  }
  AGMM_TRY(check_pointer("workspace", a->workspace, 16));
  AttnParams p = {};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k_cache);
  p.v = static_cast<const uint16_t*>(a->v_cache);
  p.out = static_cast<uint16_t*>(a->out);
  p.starts = a->node_starts;
  p.context_lens = a->context_lens;
  p.page_table = a->page_table;
  p.mask = a->mask;
  p.tokens = a->tokens;
  p.sequences = a->sequences;
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.k_ts = a->cache_token_stride;
  p.k_hs = a->cache_head_stride;
  p.out_ts = a->out_token_stride;
  p.out_hs = a->out_head_stride;
  p.page_stride = a->cache_page_stride;
  p.table_stride = a->table_stride;
  p.pages = a->pages;
  p.mask_words = (int)a->mask_words;
  p.page_shift = shift_of(plan->page_size);
  p.q_heads = plan->q_heads;
  p.kv_heads = plan->kv_heads;
  p.causal = 1;
  p.max_nodes = plan->max_nodes;
  p.scale = plan->scale;
  return launched(launch_attention(p, plan->head_dim, plan->f16, true, static_cast<cudaStream_t>(stream)), "tree");
}

}  // extern "C"
