// attn_simple.cu -- the plainest right form of both attentions: one warp per
// query row, one pass over the keys with the running maximum and sum.
//
// Each lane holds head_dim / 32 values of the query and of the output; a
// score is a dot product summed over the lanes.  Bound: instruction issue
// (about 30 warp instructions for each key of each row).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_params.h"

namespace agmm {
namespace {

template <bool kF16>
__device__ __forceinline__ float value(uint16_t b) {
  if constexpr (kF16)
    return __half2float(__ushort_as_half(b));
  else
    return __bfloat162float(__ushort_as_bfloat16(b));
}
template <bool kF16>
__device__ __forceinline__ uint16_t rounded(float x) {
  if constexpr (kF16)
    return __half_as_ushort(__float2half_rn(x));
  else
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <int kD, bool kF16, bool kPaged>
__global__ void __launch_bounds__(128) agmm_attention_simple(const __grid_constant__ AttnParams p) {
  constexpr int kN = kD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.tokens * p.q_heads) return;
  const int64_t t = row / p.q_heads;
  const int h = (int)(row % p.q_heads), hk = h / (p.q_heads / p.kv_heads);
  // the sequence of this row
  int64_t s = 0;
  for (; s < p.sequences; ++s)
    if (t < p.starts[s + 1] && t >= p.starts[s]) break;
  if (s == p.sequences) return;  // a row of no sequence
  const int64_t q0 = p.starts[s], n = min((int64_t)p.starts[s + 1], p.tokens) - q0, i = t - q0;
  int64_t m, kv0 = 0, ctx = 0;
  if constexpr (kPaged) {
    if (i >= p.max_nodes) return;
    ctx = max(p.context_lens[s], 0);
    m = min(ctx + n, p.table_stride << p.page_shift);
  } else {
    kv0 = max(p.kv_starts[s], 0);
    m = max(min((int64_t)p.kv_starts[s + 1], p.kv_tokens) - kv0, (int64_t)0);
    ctx = m - n;
  }
  float q[kN], o[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) {
    q[e] = value<kF16>(p.q[t * p.q_ts + h * p.q_hs + lane * kN + e]) * p.scale;
    o[e] = 0.0f;
  }
  float top = -INFINITY, total = 0.0f;
  for (int64_t j = 0; j < m; ++j) {
    bool seen;
    if (kPaged && p.mask != nullptr) {
      const int64_t node = j - ctx;
      seen = node < 0 || (node >> 6 < p.mask_words && (p.mask[t * p.mask_words + (node >> 6)] >> (node & 63) & 1));
    } else {
      seen = !p.causal || j <= i + ctx;
    }
    if (!seen) continue;
    const uint16_t *k, *v;
    if constexpr (kPaged) {
      const int64_t page = p.page_table[s * p.table_stride + (j >> p.page_shift)];
      if (page < 0 || page >= p.pages) {
        k = v = nullptr;
      } else {
        const int64_t at = page * p.page_stride + (j & ((1 << p.page_shift) - 1)) * p.k_ts + hk * p.k_hs;
        k = p.k + at;
        v = p.v + at;
      }
    } else {
      k = p.k + (kv0 + j) * p.k_ts + hk * p.k_hs;
      v = p.v + (kv0 + j) * p.v_ts + hk * p.v_hs;
    }
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < kN; ++e) dot += q[e] * (k ? value<kF16>(k[lane * kN + e]) : 0.0f);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
    const float next = fmaxf(top, dot);
    const float keep = top == -INFINITY ? 0.0f : __expf(top - next), w = __expf(dot - next);
    top = next;
    total = total * keep + w;
#pragma unroll
    for (int e = 0; e < kN; ++e) o[e] = o[e] * keep + w * (v ? value<kF16>(v[lane * kN + e]) : 0.0f);
  }
#pragma unroll
  for (int e = 0; e < kN; ++e)
    p.out[t * p.out_ts + h * p.out_hs + lane * kN + e] = rounded<kF16>(total == 0.0f ? 0.0f : o[e] / total);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, int head_dim, bool f16, bool paged, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.tokens * p.q_heads + 3) / 4));
#define AGMM_SIMPLE(D, F)                                                  \
  if (paged)                                                               \
    agmm_attention_simple<D, F, true><<<grid, 128, 0, stream>>>(p);        \
  else                                                                     \
    agmm_attention_simple<D, F, false><<<grid, 128, 0, stream>>>(p)
  if (head_dim == 64) {
    if (f16) {
      AGMM_SIMPLE(64, true);
    } else {
      AGMM_SIMPLE(64, false);
    }
  } else {
    if (f16) {
      AGMM_SIMPLE(128, true);
    } else {
      AGMM_SIMPLE(128, false);
    }
  }
#undef AGMM_SIMPLE
  return cudaGetLastError();
}

}  // namespace agmm
