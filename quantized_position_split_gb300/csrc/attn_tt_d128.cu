// The many-row paged attention kernel over compressed pages, head_dim 128 (see attn_tt.cuh).
#include "attn_tt.cuh"

namespace qps {
qps_status launch_paged_tt_d128(const PagedAttnParams& p, cudaStream_t s) { return tt::launch_tt_d<128>(p, s); }
}  // namespace qps
