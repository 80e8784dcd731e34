// ff_rows_plain.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn rows_plain(bool f16) {
  return f16 ? &agmm_ff_gemm<false, kEpiPlain, true> : &agmm_ff_gemm<false, kEpiPlain, false>;
}
}  // namespace ff
}  // namespace agmm
