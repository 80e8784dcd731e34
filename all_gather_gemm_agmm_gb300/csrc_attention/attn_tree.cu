// attn_tree.cu -- the attention kernel over a paged cache.
#include "attn_kernel.cuh"

namespace agmm {

AttnFn tree_kernel(int head_dim, bool f16) {
  if (head_dim == 128) return f16 ? AGMM_ATTN_VARIANT(128, true, true) : AGMM_ATTN_VARIANT(128, false, true);
  return f16 ? AGMM_ATTN_VARIANT(64, true, true) : AGMM_ATTN_VARIANT(64, false, true);
}

}  // namespace agmm
