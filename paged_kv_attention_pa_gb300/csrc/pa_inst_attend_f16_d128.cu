// Attention of many query rows with f16 queries, head_dim 128.
#include "pa_attend.cuh"

namespace pa {
cudaError_t launch_attend_f16_d128(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st) {
  return launch_attend<__half, 128>(p, maps, load, st);
}
}  // namespace pa
