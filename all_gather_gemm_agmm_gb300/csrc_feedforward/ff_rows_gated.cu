// ff_rows_gated.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn rows_gated(bool f16) {
  return f16 ? &agmm_ff_gemm<false, kEpiGated, true> : &agmm_ff_gemm<false, kEpiGated, false>;
}
}  // namespace ff
}  // namespace agmm
