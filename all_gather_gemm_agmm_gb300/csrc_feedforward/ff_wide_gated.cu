// ff_wide_gated.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn wide_gated(bool f16, bool save_f32) {
  if (save_f32) return f16 ? &agmm_ff_gemm<kWideN, kEpiGated, true, false, true> : &agmm_ff_gemm<kWideN, kEpiGated, false, false, true>;
  return f16 ? &agmm_ff_gemm<kWideN, kEpiGated, true> : &agmm_ff_gemm<kWideN, kEpiGated, false>;
}
}  // namespace ff
}  // namespace agmm
