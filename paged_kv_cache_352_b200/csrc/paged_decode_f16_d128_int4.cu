// Paged-decode kernels for __half queries over 4-bit caches, head_dim 128.
#include "decode_int4.cuh"

namespace pa {

cudaError_t launch_decode_f16_d128_int4(const DecodeArgs& a, int group, cudaStream_t stream) {
  return launch_decode_int4_typed<__half, 128>(a, group, stream);
}

}  // namespace pa
