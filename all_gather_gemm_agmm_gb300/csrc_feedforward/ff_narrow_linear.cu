// ff_narrow_linear.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn narrow_linear(bool f16, bool save_f32) {
  if (save_f32) return f16 ? &agmm_ff_gemm<kNarrowN, kEpiLinear, true, false, true> : &agmm_ff_gemm<kNarrowN, kEpiLinear, false, false, true>;
  return f16 ? &agmm_ff_gemm<kNarrowN, kEpiLinear, true> : &agmm_ff_gemm<kNarrowN, kEpiLinear, false>;
}
}  // namespace ff
}  // namespace agmm
