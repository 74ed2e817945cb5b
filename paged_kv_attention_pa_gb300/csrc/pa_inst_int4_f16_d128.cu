// Decode kernels for 4-bit caches with fp16 queries, head_dim 128.
#include "pa_decode_int4.cuh"

namespace pa {
cudaError_t launch_decode_int4_f16_d128(const DecodeParams& p, cudaStream_t st, int* kernels) {
  return launch_decode_dispatch<__half, int4g32, 128>(p, st, kernels);
}
}  // namespace pa
