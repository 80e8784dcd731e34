// ff_wide_gated.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn wide_gated(bool f16) { return f16 ? &agmm_ff_gemm<kWideN, kEpiGated, true> : &agmm_ff_gemm<kWideN, kEpiGated, false>; }
}  // namespace ff
}  // namespace agmm
