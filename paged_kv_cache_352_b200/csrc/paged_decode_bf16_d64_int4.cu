// Paged-decode kernels for __nv_bfloat16 queries over 4-bit caches, head_dim 64.
#include "decode_int4.cuh"

namespace pa {

cudaError_t launch_decode_bf16_d64_int4(const DecodeArgs& a, int group, cudaStream_t stream) {
  return launch_decode_int4_typed<__nv_bfloat16, 64>(a, group, stream);
}

}  // namespace pa
