// ff_narrow_plain.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn narrow_plain(bool f16) { return f16 ? &agmm_ff_gemm<kNarrowN, kEpiPlain, true> : &agmm_ff_gemm<kNarrowN, kEpiPlain, false>; }
}  // namespace ff
}  // namespace agmm
