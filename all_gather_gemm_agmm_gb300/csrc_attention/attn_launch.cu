// attn_launch.cu -- launches of the attention kernel, and the sum of the parts
// of a tree's split work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_params.h"
#include "attn_ptx.cuh"

namespace agmm {
namespace {

constexpr int kJoinThreads = 256;

// A row's parts hold O, m and l over disjoint keys:
//   out = sum 2^(c (m_i - M)) O_i / sum 2^(c (m_i - M)) l_i,   M = max m_i
// in the order of the CTAs that hold them.  Block (c, y): rows of the item whose
// first part lies in CTA c; head_dim / 4 threads to a row.  Bound: latency (the
// parts are in L2).
template <int kD, bool kF16>
__global__ void __launch_bounds__(kJoinThreads) agmm_attn_join(const __grid_constant__ AttnParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kPer = kD / 4;
  const int first = blockIdx.x;
  const int* const join = p.joins + (size_t)first * kJoinInts;
  if (join[0] == 0) return;
  const int last = join[1], rows = join[3];
  const int row = blockIdx.y * (kJoinThreads / kPer) + threadIdx.x / kPer;
  if (row >= rows) return;
  const int col = threadIdx.x % kPer * 4;
  const float* const ml = p.partial + (size_t)gridDim.x * 2 * p.partial_rows * kD;
  auto at = [&](int c) { return (size_t)(2 * c + (c == first)) * p.partial_rows + row; };
  float top = -INFINITY;
  for (int c = first; c <= last; ++c) top = fmaxf(top, ml[at(c) * 2]);
  float l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int c = first; c <= last; ++c) {
    const float2 x = *reinterpret_cast<const float2*>(ml + at(c) * 2);
    const float4 v = *reinterpret_cast<const float4*>(p.partial + at(c) * kD + col);
    const float w = x.x == -INFINITY ? (x.y != x.y ? 1.0f : 0.0f) : ptx::exp2_approx((x.x - top) * p.scale_log2);
    l += w * x.y;
    o.x += w * v.x;
    o.y += w * v.y;
    o.z += w * v.z;
    o.w += w * v.w;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int token = row / p.pack;
  uint16_t* const out = p.out + (int64_t)(join[2] + token) * p.out_ts + (join[4] + row - token * p.pack) * p.out_hs + col;
  uint2 packed;
  if constexpr (kF16) {
    const __half2 a = __floats2half2_rn(o.x * inv, o.y * inv), b = __floats2half2_rn(o.z * inv, o.w * inv);
    packed = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    packed = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(out) = packed;
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
  const int per_block = kJoinThreads / (head_dim / 4);
  const dim3 grid((unsigned)ctas, (unsigned)((p.partial_rows + per_block - 1) / per_block));
  void (*fn)(AttnParams) = head_dim == 128 ? (f16 ? &agmm_attn_join<128, true> : &agmm_attn_join<128, false>)
                                           : (f16 ? &agmm_attn_join<64, true> : &agmm_attn_join<64, false>);
  return launch(fn, p, grid, kJoinThreads, 0, stream);
}

}  // namespace agmm
