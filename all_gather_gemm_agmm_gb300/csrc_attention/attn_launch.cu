// attn_launch.cu -- launches of the attention kernel, and the sum of the parts
// of work that was cut along the keys (trees, and prompts with few items).
#include "attn_params.h"
#include "attn_ptx.cuh"

namespace agmm {
namespace {

constexpr int kJoinThreads = 256;

// A row's parts hold O, m and l over disjoint keys:
//   out = sum 2^(c (m_i - M)) O_i / sum 2^(c (m_i - M)) l_i,   M = max m_i
// always in the order of the CTAs that hold them.  Bound: latency (the parts are
// in L2).  The last CTA of an item could do this without another launch, but
// then few warps do it: one decode step over 1000 keys took 15.3 us so, against 13.0 us,
// in one build (14.7 us now).
//
// One warp joins one row of an item: row `part_row` of its parts, `row` of its tile;
// parts in the CTAs [first, last].  Part of CTA c: slot 2 c, or 2 c + 1 for the first.
template <int kD, bool kF16>
__device__ __forceinline__ void join_row(const AttnParams& p, int first, int last, int part_row, int row, int token0,
                                         int head0) {
  constexpr int kN = kD / 32;  // columns of a lane
  const int lane = threadIdx.x & 31;
  const float2* const ml = reinterpret_cast<const float2*>(p.partial + (size_t)gridDim.x * 2 * p.partial_rows * kD);
  float top = -INFINITY, l = 0.0f, o[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) o[e] = 0.0f;
  // Eight parts at a time, all their loads in flight together.
#pragma unroll 1
  for (int c0 = first; c0 <= last; c0 += 8) {
    float2 x[8];
    float v[8][kN];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i;
      const size_t at = (size_t)(2 * c + (c == first)) * p.partial_rows + part_row;
      x[i] = make_float2(-INFINITY, 0.0f);
      if (c <= last) {
        x[i] = __ldcg(ml + at);
        const float* const src = p.partial + at * kD + lane * kN;
        if constexpr (kN == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
          v[i][0] = y.x;
          v[i][1] = y.y;
          v[i][2] = y.z;
          v[i][3] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
          v[i][0] = y.x;
          v[i][1] = y.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) v[i][e] = 0.0f;
      }
    }
    float next = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) next = fmaxf(next, x[i].x);
    const float keep = top == -INFINITY ? (l != l ? 1.0f : 0.0f) : ptx::exp2_approx((top - next) * p.scale_log2);
    l *= keep;
#pragma unroll
    for (int e = 0; e < kN; ++e) o[e] *= keep;
    top = next;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = x[i].x == -INFINITY ? (x[i].y != x[i].y ? 1.0f : 0.0f) : ptx::exp2_approx((x[i].x - top) * p.scale_log2);
      l += w * x[i].y;
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] += w * v[i][e];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int token = row / p.pack;
  uint16_t* const out = p.out + (int64_t)(token0 + token) * p.out_ts + (head0 + row - token * p.pack) * p.out_hs + lane * kN;
  uint32_t packed[kN / 2];
#pragma unroll
  for (int e = 0; e < kN / 2; ++e) packed[e] = ptx::round_pair<kF16>(o[2 * e] * inv, o[2 * e + 1] * inv);
  if constexpr (kN == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[1]);
  else
    *reinterpret_cast<uint32_t*>(out) = packed[0];
}

// Block (c, y) joins 8 rows of the item whose first part lies in CTA c.
template <int kD, bool kF16>
__global__ void __launch_bounds__(kJoinThreads) agmm_attn_join(const __grid_constant__ AttnParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int* const join = p.joins + (size_t)blockIdx.x * kJoinInts;
  if (join[0] == 0) return;
  const int tile_rows = p.tile_tokens * p.pack;
  int row = blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32;
  const int s = row >= tile_rows;  // the item's second tile
  if (row - s * tile_rows >= join[s ? 6 : 2]) return;
  join_row<kD, kF16>(p, blockIdx.x, join[4], row, row - s * tile_rows, join[s ? 5 : 1], join[s ? 7 : 3]);
}

cudaError_t launch(void (*fn)(AttnParams), const AttnParams& p, dim3 grid, int threads, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  // The prologue may overlap the previous kernel's tail; the kernels wait
  // (griddepcontrol.wait) before their first access to global memory.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t prepare_attention(const AttnFn& k) {
  return cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
}

cudaError_t launch_attention(const AttnFn& k, const AttnParams& p, int ctas, cudaStream_t stream) {
  return launch(k.fn, p, dim3((unsigned)ctas), kAttnThreads, k.smem, stream);
}

cudaError_t launch_join(const AttnParams& p, int head_dim, bool f16, int ctas, cudaStream_t stream) {
  const int per_block = kJoinThreads / 32;
  const dim3 grid((unsigned)ctas, (unsigned)((p.partial_rows + per_block - 1) / per_block));
  void (*fn)(AttnParams) = head_dim == 128 ? (f16 ? &agmm_attn_join<128, true> : &agmm_attn_join<128, false>)
                                           : (f16 ? &agmm_attn_join<64, true> : &agmm_attn_join<64, false>);
  return launch(fn, p, grid, kJoinThreads, 0, stream);
}

}  // namespace agmm
