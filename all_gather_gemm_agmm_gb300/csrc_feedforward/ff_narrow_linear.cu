// ff_narrow_linear.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn narrow_linear(bool f16) { return f16 ? &agmm_ff_gemm<kNarrowN, kEpiLinear, true> : &agmm_ff_gemm<kNarrowN, kEpiLinear, false>; }
}  // namespace ff
}  // namespace agmm
