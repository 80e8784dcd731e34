// ff_swap_gated.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn swap_gated(bool f16, bool save_f32) {
  if (save_f32) return f16 ? &agmm_ff_gemm<0, kEpiGated, true, false, true> : &agmm_ff_gemm<0, kEpiGated, false, false, true>;
  return f16 ? &agmm_ff_gemm<0, kEpiGated, true> : &agmm_ff_gemm<0, kEpiGated, false>;
}
}  // namespace ff
}  // namespace agmm
