// Windowed decode attention instances for head_dim 64 (see attn_mma.cuh): K F16 / Q8_0 with
// V F16 / Q8_0 / TQ3; the other TurboQuant pairings are in attn_window_d64_tq.cu.
#include "attn_mma.cuh"

namespace qps {
qps_status launch_window_mma_d64_tq(const WindowAttnParams& p, cudaStream_t s);
qps_status launch_window_mma_d64(const WindowAttnParams& p, cudaStream_t s) {
  if (is_tq(p.kfmt) || p.vfmt == QPS_FMT_TQ2 || p.vfmt == QPS_FMT_TQ4) return launch_window_mma_d64_tq(p, s);
  return mma::launch_mma_d<64, false, 0>(p, s);
}
}  // namespace qps
