// The prompt attention kernel for head_dim 512 (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d512(const PromptParams& p, cudaStream_t s) { return prompt::launch_prompt_d<512>(p, s); }
}  // namespace qps
