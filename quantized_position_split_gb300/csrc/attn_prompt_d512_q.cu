// The prompt attention kernel for head_dim 512, compressed keys (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d512_q(const PromptParams& p, cudaStream_t s) {
  return p.v_parts == 2 ? prompt::launch_prompt<512, 2, 2>(p, s) : prompt::launch_prompt<512, 2, 1>(p, s);
}
}  // namespace qps
