// Rotary append of f16 queries, keys and values.
#include "rotate_kernel.cuh"

namespace wllm {
int launch_rotate_f16(const RotateParams& p, unsigned blocks, int ring_smem, int num_sms, cudaStream_t stream) {
  return launch_rotate_typed<__half>(p, blocks, ring_smem, num_sms, stream);
}
}  // namespace wllm
