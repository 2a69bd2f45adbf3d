// The many-row windowed attention kernel for head_dim 64 (see attn_tm.cuh).
#include "attn_tm.cuh"

namespace qps {
qps_status launch_window_tm_d64(const WindowAttnParams& p, cudaStream_t s) { return tm::launch_tm<64>(p, s); }
}  // namespace qps
