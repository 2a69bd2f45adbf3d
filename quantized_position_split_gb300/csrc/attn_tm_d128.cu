// The many-row paged attention kernel for head_dim 128 (see attn_tm.cuh).
#include "attn_tm.cuh"

namespace qps {
qps_status launch_paged_tm_d128(const PagedAttnParams& p, cudaStream_t s) { return tm::launch_tm<128>(p, s); }
}  // namespace qps
