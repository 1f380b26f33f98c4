// Paged-decode kernels for __half queries over 4-bit caches, head_dim 64.
#include "paged_decode_impl.cuh"

namespace pa {

cudaError_t launch_decode_f16_d64_int4(const DecodeArgs& a, int group, cudaStream_t stream) {
  return launch_decode_typed<__half, 64, Int4>(a, group, PA_F16, stream);
}

}  // namespace pa
