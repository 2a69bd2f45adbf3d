// kv_append_paged instances for float32 rows (see head_rows.cuh).
#include "head_rows.cuh"

namespace qps {
qps_status append_f32(int d, const AppendP& p, cudaStream_t s) { return rows::append_by_d<float>(d, p, s); }
}  // namespace qps
