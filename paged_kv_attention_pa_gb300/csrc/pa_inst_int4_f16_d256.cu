// Decode kernels for 4-bit caches with fp16 queries, head_dim 256.
#include "pa_decode_int4.cuh"

namespace pa {
cudaError_t launch_decode_int4_f16_d256(const DecodeParams& p, cudaStream_t st, int* kernels) {
  return launch_decode_dispatch<__half, int4g32, 256>(p, st, kernels);
}
}  // namespace pa
