// attn_api.cpp -- the C ABI of include/agmm_attention.h: argument checks,
// plans and launches of the attention operators.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <new>

#include <cudaTypedefs.h>

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
  AttnFn kernel;
  int pack, tile_tokens, partial_rows;
  uint64_t wait_limit_cycles;
  int test_drop;
};
struct agmm_prompt_s : AttnPlan {};
struct agmm_tree_s : AttnPlan {};

namespace {

// A part of a prompt's item is at least this many key tiles: its results make a
// round trip through device memory, 256 rows in float32.
constexpr int kMinPromptTiles = 4;
// From this many items for each CTA on, prompts draw whole items; fewer are cut along
// the keys.  Measured, each pair in one build: 1.5 items (two pieces of 1024 and 700 tokens
// behind 8000 to 15000 keys, 32 heads) 332 us drawn, 239 us cut; 4.1 items (prompts of 17
// to 4001 tokens, 16 heads) 87 us drawn, 118 us cut; 6.7 items (one of 8191 tokens, 32
// heads) 341 us drawn, 418 us cut.  Between 1.5 and 4.1 nothing was measured.  The
// rule goes by the most items that the rows can make, not by those they make, and not
// by their keys, which the host does not know.
constexpr int kDrawnItems = 2;

// Most rows, and most places of a sequence: the kernels count both in 32 bits, and
// go past an end by a tile of keys, two of rows, or a tree's nodes.
constexpr int64_t kMostPlaces = INT_MAX - 4096;

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
  if (!std::isfinite(scale) || !(scale > 0.0f)) return fail(AGMM_ERR_INVALID_ARG, "scale must be positive and finite");
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

// The device's peak clock.  Asked once per device: the driver takes most of a
// millisecond to answer.
int peak_clock_khz(int device) {
  static std::atomic<int> known[64];
  const bool cached = device >= 0 && device < 64;
  int khz = cached ? known[device].load(std::memory_order_relaxed) : 0;
  if (khz > 0) return khz;
  if (cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, device) != cudaSuccess || khz <= 0) {
    (void)cudaGetLastError();
    khz = 2100000;  // above the part's 2.07 GHz peak
  }
  if (cached) known[device].store(khz, std::memory_order_relaxed);
  return khz;
}

// What both attention plans hold, from the checked description.
agmm_status_t fill_plan(AttnPlan* pl, int q_heads, int kv_heads, int head_dim, agmm_dtype_t dtype, float scale, bool tree) {
  pl->q_heads = q_heads;
  pl->kv_heads = kv_heads;
  pl->head_dim = head_dim;
  pl->f16 = dtype == AGMM_F16;
  pl->scale = scale;
  pl->pack = tree ? q_heads / kv_heads : 1;
  pl->tile_tokens = kRows / pl->pack;
  pl->partial_rows = 2 * pl->tile_tokens * pl->pack;
  pl->kernel = tree ? tree_kernel(head_dim, pl->f16) : prompt_kernel(head_dim, pl->f16);
  const int khz = peak_clock_khz(pl->device);
  const char* ms = std::getenv("AGMM_WAIT_LIMIT_MS");
  const int limit = ms && *ms ? std::atoi(ms) : 0;
  pl->wait_limit_cycles = (uint64_t)(limit > 0 ? limit : 2000) * (uint64_t)khz;
  const char* drop = std::getenv("AGMM_TEST_DROP_ARRIVE");
  pl->test_drop = drop && std::atoi(drop) != 0;
  const cudaError_t e = prepare_attention(pl->kernel);
  if (e != cudaSuccess) return fail(AGMM_ERR_CUDA, "kernel attributes: %s", cudaGetErrorString(e));
  return AGMM_OK;
}

// Where the join records of a workspace end and its partial results begin.
size_t joins_end(const AttnPlan* pl) {
  return (kAttnStatusBytes + (size_t)pl->num_sms * kJoinInts * sizeof(int) + 255) / 256 * 256;
}

size_t workspace_bytes(const AttnPlan* pl) {
  const size_t rows = (size_t)pl->num_sms * 2 * pl->partial_rows;
  return joins_end(pl) + rows * ((size_t)pl->head_dim + 2) * sizeof(float);
}

// The plan's fields of a launch, and the Q tiles' tensor map.
void fill_params(const AttnPlan* pl, AttnParams* p, void* workspace) {
  p->q_heads = pl->q_heads;
  p->kv_heads = pl->kv_heads;
  p->group = pl->q_heads / pl->kv_heads;
  p->pack = pl->pack;
  p->tile_tokens = pl->tile_tokens;
  p->scale_log2 = (float)((double)pl->scale * 1.4426950408889634074);  // log2(e)
  p->wait_limit_cycles = pl->wait_limit_cycles;
  p->test_drop_first_load = pl->test_drop;
  p->status = static_cast<int*>(workspace);
  char* const ws = static_cast<char*>(workspace);
  p->counter = reinterpret_cast<int*>(ws + kCounterOffset);
  p->joins = reinterpret_cast<int*>(ws + kAttnStatusBytes);
  p->partial = reinterpret_cast<float*>(ws + joins_end(pl));
  p->partial_rows = pl->partial_rows;
}

agmm_status_t check_plan_device(int device) {
  int now = -1;
  const cudaError_t e = cudaGetDevice(&now);
  if (e != cudaSuccess) return fail(AGMM_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (now != device) return fail(AGMM_ERR_INVALID_ARG, "the plan belongs to device %d, the current device is %d", device, now);
  return AGMM_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A tensor map of 16-bit values whose boxes are 64 columns wide, 128-byte
// swizzled, zero-filled outside.  dims, box: innermost first; strides of the
// dimensions after the first, in elements.
agmm_status_t encode(CUtensorMap* map, const char* name, const void* ptr, int rank, const int64_t* dims, const int64_t* strides,
                     const int* box, bool f16) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(AGMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], es[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    es[i] = 1;
    // a dimension of one value has no stride to speak of; the map wants some
    if (i) st[i - 1] = (cuuint64_t)((dims[i] == 1 ? dims[0] : strides[i - 1]) * 2);
  }
  const CUresult r = enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                         const_cast<void*>(ptr), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(AGMM_ERR_CUDA, "tensor map of %s: cuTensorMapEncodeTiled gave %d", name, (int)r);
  return AGMM_OK;
}

agmm_status_t encode_q(CUtensorMap* map, const AttnPlan* pl, const void* q, int64_t tokens, int64_t ts, int64_t hs) {
  const int64_t dims[3] = {pl->head_dim, pl->q_heads, tokens}, strides[2] = {hs, ts};
  const int box[3] = {64, pl->pack, pl->tile_tokens};
  return encode(map, "q", q, 3, dims, strides, box, pl->f16);
}

// Keys or values: rows (tokens, or the places of a page), heads, pages.
agmm_status_t encode_kv(CUtensorMap* map, const char* name, const AttnPlan* pl, const void* x, int64_t rows, int64_t pages,
                        int64_t ts, int64_t hs, int64_t ps, int box_rows) {
  const int64_t dims[4] = {pl->head_dim, rows, pl->kv_heads, pages}, strides[3] = {ts, hs, ps};
  const int box[4] = {64, box_rows, 1, 1};
  return encode(map, name, x, 4, dims, strides, box, pl->f16);
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
  AGMM_TRY(check_plan_device(plan->device));
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
  pl->causal = d->causal != 0;
  pl->device = device;
  pl->num_sms = sms;
  const agmm_status_t st = fill_plan(pl, d->q_heads, d->kv_heads, d->head_dim, d->dtype, d->scale, false);
  if (st != AGMM_OK) {
    delete pl;
    return st;
  }
  *out = pl;
  return AGMM_OK;
}

void agmm_prompt_destroy(agmm_prompt_t plan) { delete plan; }

size_t agmm_prompt_workspace_bytes(agmm_prompt_t plan) { return plan ? workspace_bytes(plan) : 0; }

agmm_status_t agmm_prompt_run(agmm_prompt_t plan, const agmm_prompt_args_t* a, void* stream) {
  if (!plan || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_range("tokens", a->tokens, 0, kMostPlaces));
  AGMM_TRY(check_range("kv_tokens", a->kv_tokens, 0, kMostPlaces));
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
  // row-tile pairs there can be
  const int64_t pairs = a->tokens / (2 * kRows) + (a->sequences < a->tokens ? a->sequences : a->tokens);
  if (pairs * plan->q_heads >= kMostItems)
    return fail(AGMM_ERR_UNSUPPORTED, "too many rows for one run: %lld tokens of %d heads", (long long)a->tokens, plan->q_heads);
  AGMM_TRY(check_plan_device(plan->device));
  AttnParams p = {};
  fill_params(plan, &p, a->workspace);
  AGMM_TRY(encode_q(&p.qmap, plan, a->q, a->tokens, a->q_token_stride, a->q_head_stride));
  if (a->kv_tokens) {
    AGMM_TRY(encode_kv(&p.kmap, "k", plan, a->k, a->kv_tokens, 1, a->k_token_stride, a->k_head_stride, 0, kKeys));
    AGMM_TRY(encode_kv(&p.vmap, "v", plan, a->v, a->kv_tokens, 1, a->v_token_stride, a->v_head_stride, 0, kKeys));
  }
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.k = static_cast<const uint16_t*>(a->k);
  p.k_ts = a->k_token_stride;
  p.k_hs = a->k_head_stride;
  p.v = static_cast<const uint16_t*>(a->v);
  p.v_ts = a->v_token_stride;
  p.v_hs = a->v_head_stride;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_ts = a->out_token_stride;
  p.out_hs = a->out_head_stride;
  p.starts = a->starts;
  p.kv_starts = a->kv_starts ? a->kv_starts : a->starts;
  p.tokens = a->tokens;
  p.kv_tokens = a->kv_tokens;
  p.sequences = (int)a->sequences;
  p.causal = plan->causal;
  p.min_tiles = kMinPromptTiles;
  p.by_draw = pairs * plan->q_heads >= (int64_t)kDrawnItems * plan->num_sms;
  // then there are enough items for a one-tile set to take two heads, which share its keys
  p.pair_heads = p.by_draw && p.group % 2 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  AGMM_TRY(launched(launch_attention(plan->kernel, p, plan->num_sms, s), "prompt"));
  // no cuts, or nothing long enough to be cut
  if (p.by_draw || a->kv_tokens <= (2 * kMinPromptTiles - 1) * kKeys) return AGMM_OK;
  return launched(launch_join(p, plan->head_dim, plan->f16, plan->num_sms, s), "prompt join");
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
  pl->causal = 1;
  pl->page_size = d->page_size;
  pl->max_nodes = d->max_nodes;
  pl->device = device;
  pl->num_sms = sms;
  const agmm_status_t st = fill_plan(pl, d->q_heads, d->kv_heads, d->head_dim, d->dtype, d->scale, true);
  if (st != AGMM_OK) {
    delete pl;
    return st;
  }
  pl->partial_rows = (d->max_nodes < 2 * pl->tile_tokens ? d->max_nodes : 2 * pl->tile_tokens) * pl->pack;
  *out = pl;
  return AGMM_OK;
}

void agmm_tree_destroy(agmm_tree_t plan) { delete plan; }

size_t agmm_tree_workspace_bytes(agmm_tree_t plan) { return plan ? workspace_bytes(plan) : 0; }

agmm_status_t agmm_tree_run(agmm_tree_t plan, const agmm_tree_args_t* a, void* stream) {
  if (!plan || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_range("tokens", a->tokens, 0, kMostPlaces));
  AGMM_TRY(check_range("sequences", a->sequences, 0, 1 << 20));
  if (a->tokens == 0 || a->sequences == 0) return AGMM_OK;
  AGMM_TRY(check_operand("q", a->q, a->q_token_stride, a->q_head_stride));
  AGMM_TRY(check_operand("out", a->out, a->out_token_stride, a->out_head_stride));
  AGMM_TRY(check_operand("k_cache", a->k_cache, a->cache_token_stride, a->cache_head_stride));
  AGMM_TRY(check_operand("v_cache", a->v_cache, a->cache_page_stride, a->cache_head_stride));
  AGMM_TRY(check_range("pages", a->pages, 1, INT_MAX));
  AGMM_TRY(check_range("table_pages", a->table_pages, 1, kMostPlaces / plan->page_size));
  AGMM_TRY(check_range("table_stride", a->table_stride, 0, (int64_t)1 << 38));
  AGMM_TRY(check_pointer("page_table", a->page_table, 4));
  AGMM_TRY(check_pointer("context_lens", a->context_lens, 4));
  AGMM_TRY(check_pointer("node_starts", a->node_starts, 4));
  if (a->mask) {
    AGMM_TRY(check_pointer("mask", a->mask, 8));
    AGMM_TRY(check_range("mask_words", a->mask_words, (plan->max_nodes + 63) / 64, 1 << 20));
  }
  AGMM_TRY(check_pointer("workspace", a->workspace, 16));
  AGMM_TRY(check_plan_device(plan->device));
  AttnParams p = {};
  fill_params(plan, &p, a->workspace);
  const int box_rows = plan->page_size < kKeys ? plan->page_size : kKeys;
  AGMM_TRY(encode_q(&p.qmap, plan, a->q, a->tokens, a->q_token_stride, a->q_head_stride));
  AGMM_TRY(encode_kv(&p.kmap, "k_cache", plan, a->k_cache, plan->page_size, a->pages, a->cache_token_stride,
                     a->cache_head_stride, a->cache_page_stride, box_rows));
  AGMM_TRY(encode_kv(&p.vmap, "v_cache", plan, a->v_cache, plan->page_size, a->pages, a->cache_token_stride,
                     a->cache_head_stride, a->cache_page_stride, box_rows));
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.k = static_cast<const uint16_t*>(a->k_cache);
  p.v = static_cast<const uint16_t*>(a->v_cache);
  p.k_ts = p.v_ts = a->cache_token_stride;
  p.k_hs = p.v_hs = a->cache_head_stride;
  p.k_ps = p.v_ps = a->cache_page_stride;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_ts = a->out_token_stride;
  p.out_hs = a->out_head_stride;
  p.starts = a->node_starts;
  p.context_lens = a->context_lens;
  p.page_table = a->page_table;
  p.table_pages = a->table_pages;
  p.table_stride = a->table_stride;
  p.pages = a->pages;
  p.page_shift = shift_of(plan->page_size);
  p.mask = a->mask;
  p.mask_words = (int)a->mask_words;
  p.tokens = a->tokens;
  p.sequences = (int)a->sequences;
  p.causal = 1;
  p.max_nodes = plan->max_nodes;
  p.min_tiles = 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  AGMM_TRY(launched(launch_attention(plan->kernel, p, plan->num_sms, s), "tree"));
  return launched(launch_join(p, plan->head_dim, plan->f16, plan->num_sms, s), "tree join");
}

}  // extern "C"
