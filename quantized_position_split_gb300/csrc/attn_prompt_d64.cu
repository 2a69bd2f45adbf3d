// The prompt attention kernel for head_dim 64, fp16 keys (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d64(const PromptParams& p, cudaStream_t s) {
  return p.v_parts == 2 ? prompt::launch_prompt<64, 1, 2>(p, s) : prompt::launch_prompt<64, 1, 1>(p, s);
}
}  // namespace qps
