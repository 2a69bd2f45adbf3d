// The prompt attention kernel for head_dim 128, compressed keys (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d128_q(const PromptParams& p, cudaStream_t s) {
  return p.v_parts == 2 ? prompt::launch_prompt<128, 2, 2>(p, s) : prompt::launch_prompt<128, 2, 1>(p, s);
}
}  // namespace qps
