// Paged decode attention instances for head_dim 128 (see attn_mma.cuh): K F16 / Q8_0 with
// V F16 / Q8_0 / TQ3; the other TurboQuant pairings are in attn_paged_d128_tq.cu.
#include "attn_mma.cuh"

namespace qps {
qps_status launch_paged_mma_d128_tq(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_mma_d128(const PagedAttnParams& p, cudaStream_t s) {
  if (is_tq(p.kfmt) || p.vfmt == QPS_FMT_TQ2 || p.vfmt == QPS_FMT_TQ4) return launch_paged_mma_d128_tq(p, s);
  return mma::launch_mma_d<128, false, 0>(p, s);
}
}  // namespace qps
