// The many-row windowed attention kernel over compressed and fp16 pages, head_dim 512 (see attn_tt.cuh).
#include "attn_tt.cuh"

namespace qps {
qps_status launch_window_tt_d512(const WindowAttnParams& p, cudaStream_t s) { return tt::launch_tt_d<512>(p, s); }
}  // namespace qps
