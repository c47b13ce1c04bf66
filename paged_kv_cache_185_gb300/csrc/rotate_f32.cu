// Rotary append of binary32 queries, keys and values.
#include "rotate_kernel.cuh"

namespace wllm {
int launch_rotate_f32(const RotateParams& p, unsigned blocks, int ring_smem, int num_sms, cudaStream_t stream) {
  return launch_rotate_typed<float>(p, blocks, ring_smem, num_sms, stream);
}
}  // namespace wllm
