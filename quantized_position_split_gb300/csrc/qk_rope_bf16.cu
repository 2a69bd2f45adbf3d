// qk_norm_rope instances for bfloat16 rows (see head_rows.cuh).
#include "head_rows.cuh"

namespace qps {
qps_status rope_bf16(int d, const RopeP& p, cudaStream_t s) { return rows::rope_by_d<__nv_bfloat16>(d, p, s); }
}  // namespace qps
