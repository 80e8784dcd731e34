// ff_launch.cu -- launches of the feed-forward products' kernel.
#include "ff_params.h"

namespace agmm {
namespace ff {

GemmFn select_gemm(int bn, int epi, bool f16, bool save_f32) {
  if (bn == kWideN) return epi == kEpiGated ? wide_gated(f16, save_f32) : epi == kEpiLinear ? wide_linear(f16, save_f32) : wide_plain(f16);
  if (bn == kNarrowN) return epi == kEpiGated ? narrow_gated(f16, save_f32) : epi == kEpiLinear ? narrow_linear(f16, save_f32) : narrow_plain(f16);
  return epi == kEpiGated ? swap_gated(f16, save_f32) : epi == kEpiLinear ? swap_linear(f16, save_f32) : swap_plain(f16);
}

namespace {

template <class P>
cudaError_t prepare(void (*fn)(P), int cluster, int* clusters) {
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(clusters, fn, &cfg);
}

template <class P>
cudaError_t launch(void (*fn)(P), const P& p, int clusters, int cluster, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  // The prologue may overlap the previous kernel's tail; the kernel waits
  // (griddepcontrol.wait) before its first access to global memory.
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t prepare_gemm(GemmFn fn, int cluster, int* clusters) { return prepare(fn, cluster, clusters); }
cudaError_t prepare_two(TwoFn fn, int* clusters) { return prepare(fn, 2, clusters); }
cudaError_t launch_gemm(GemmFn fn, const GemmParams& p, int clusters, int cluster, size_t smem, cudaStream_t stream) {
  return launch(fn, p, clusters, cluster, smem, stream);
}
cudaError_t launch_two(TwoFn fn, const TwoParams& p, int clusters, size_t smem, cudaStream_t stream) {
  return launch(fn, p, clusters, 2, smem, stream);
}

}  // namespace ff
}  // namespace agmm
