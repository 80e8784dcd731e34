// attn_prompt.cu -- the attention kernel for packed prompts.
#include "attn_kernel.cuh"

namespace agmm {

AttnFn prompt_kernel(int head_dim, bool f16) {
  if (head_dim == 128) return f16 ? AGMM_ATTN_VARIANT(128, true, false) : AGMM_ATTN_VARIANT(128, false, false);
  return f16 ? AGMM_ATTN_VARIANT(64, true, false) : AGMM_ATTN_VARIANT(64, false, false);
}

}  // namespace agmm
