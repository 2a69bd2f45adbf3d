// The prompt attention kernel for head_dim 256 (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d256(const PromptParams& p, cudaStream_t s) { return prompt::launch_prompt_d<256>(p, s); }
}  // namespace qps
