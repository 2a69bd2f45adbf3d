// The many-row windowed attention kernel over compressed and fp16 pages, head_dim 256 (see attn_tt.cuh).
#include "attn_tt.cuh"

namespace qps {
qps_status launch_window_tt_d256(const WindowAttnParams& p, cudaStream_t s) { return tt::launch_tt_d<256>(p, s); }
}  // namespace qps
