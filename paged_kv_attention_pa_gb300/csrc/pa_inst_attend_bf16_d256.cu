// Attention of many query rows with bf16 queries, head_dim 256.
#include "pa_attend.cuh"

namespace pa {
cudaError_t launch_attend_bf16_d256(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st) {
  return launch_attend<__nv_bfloat16, 256>(p, maps, load, st);
}
}  // namespace pa
