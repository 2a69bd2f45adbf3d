// qk_norm_rope instances for float32 rows (see head_rows.cuh).
#include "head_rows.cuh"

namespace qps {
qps_status rope_f32(int d, const RopeP& p, cudaStream_t s) { return rows::rope_by_d<float>(d, p, s); }
}  // namespace qps
