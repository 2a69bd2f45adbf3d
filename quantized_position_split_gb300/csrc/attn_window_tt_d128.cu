// The many-row windowed attention kernel over compressed pages, head_dim 128 (see attn_tt.cuh).
#include "attn_tt.cuh"

namespace qps {
qps_status launch_window_tt_d128(const WindowAttnParams& p, cudaStream_t s) { return tt::launch_tt_d<128>(p, s); }
}  // namespace qps
