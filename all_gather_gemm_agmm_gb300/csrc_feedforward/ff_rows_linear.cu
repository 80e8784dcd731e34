// ff_rows_linear.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn rows_linear(bool f16) {
  return f16 ? &agmm_ff_gemm<false, kEpiLinear, true> : &agmm_ff_gemm<false, kEpiLinear, false>;
}
}  // namespace ff
}  // namespace agmm
