// ff_wide_linear.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn wide_linear(bool f16, bool save_f32) {
  if (save_f32) return f16 ? &agmm_ff_gemm<kWideN, kEpiLinear, true, false, true> : &agmm_ff_gemm<kWideN, kEpiLinear, false, false, true>;
  return f16 ? &agmm_ff_gemm<kWideN, kEpiLinear, true> : &agmm_ff_gemm<kWideN, kEpiLinear, false>;
}
}  // namespace ff
}  // namespace agmm
