// The many-row paged attention kernel for head_dim 64 (see attn_tm.cuh).
#include "attn_tm.cuh"

namespace qps {
qps_status launch_paged_tm_d64(const PagedAttnParams& p, cudaStream_t s) { return tm::launch_tm<64>(p, s); }
}  // namespace qps
