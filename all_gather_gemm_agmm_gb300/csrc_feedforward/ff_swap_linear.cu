// ff_swap_linear.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn swap_linear(bool f16) { return f16 ? &agmm_ff_gemm<0, kEpiLinear, true> : &agmm_ff_gemm<0, kEpiLinear, false>; }
}  // namespace ff
}  // namespace agmm
