// The prompt attention kernel for head_dim 128 (see attn_prompt.cuh).
#include "attn_prompt.cuh"

namespace qps {
qps_status launch_prompt_d128(const PromptParams& p, cudaStream_t s) { return prompt::launch_prompt_d<128>(p, s); }
}  // namespace qps
