// Paged decode attention instances for head_dim 512 with a TQ2 / TQ4 V or a TurboQuant K
// (see attn_mma.cuh).
#include "attn_mma.cuh"

namespace qps {
qps_status launch_paged_mma_d512_tq(const PagedAttnParams& p, cudaStream_t s) {
  return is_tq(p.kfmt) ? mma::launch_mma_d<512, false, 2>(p, s) : mma::launch_mma_d<512, false, 1>(p, s);
}
}  // namespace qps
