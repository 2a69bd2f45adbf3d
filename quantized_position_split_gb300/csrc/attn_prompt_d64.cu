// The prompt attention kernel for head_dim 64 (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d64(const PromptParams& p, cudaStream_t s) { return prompt::launch_prompt_d<64>(p, s); }
}  // namespace qps
