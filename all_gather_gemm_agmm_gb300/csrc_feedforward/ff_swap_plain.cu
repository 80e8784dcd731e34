// ff_swap_plain.cu -- instantiations of the feed-forward products' kernel.
#include "ff_gemm.cuh"

namespace agmm {
namespace ff {
GemmFn swap_plain(bool f16) { return f16 ? &agmm_ff_gemm<0, kEpiPlain, true> : &agmm_ff_gemm<0, kEpiPlain, false>; }
}  // namespace ff
}  // namespace agmm
