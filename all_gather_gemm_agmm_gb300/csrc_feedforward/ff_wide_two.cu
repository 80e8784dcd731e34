// ff_wide_two.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
TwoFn wide_two(bool f16) { return f16 ? &agmm_ff_gemm<kWideN, kEpiPlain, true, true> : &agmm_ff_gemm<kWideN, kEpiPlain, false, true>; }
}  // namespace ff
}  // namespace agmm
