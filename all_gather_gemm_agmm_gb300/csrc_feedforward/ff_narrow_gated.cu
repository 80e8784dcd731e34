// ff_narrow_gated.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn narrow_gated(bool f16, bool save_f32) {
  if (save_f32) return f16 ? &agmm_ff_gemm<kNarrowN, kEpiGated, true, false, true> : &agmm_ff_gemm<kNarrowN, kEpiGated, false, false, true>;
  return f16 ? &agmm_ff_gemm<kNarrowN, kEpiGated, true> : &agmm_ff_gemm<kNarrowN, kEpiGated, false>;
}
}  // namespace ff
}  // namespace agmm
