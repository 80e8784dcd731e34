// ff_wide_plain.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn wide_plain(bool f16) { return f16 ? &agmm_ff_gemm<kWideN, kEpiPlain, true> : &agmm_ff_gemm<kWideN, kEpiPlain, false>; }
}  // namespace ff
}  // namespace agmm
