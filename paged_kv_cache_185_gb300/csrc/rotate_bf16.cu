// Rotary append of bfloat16 queries, keys and values.
#include "rotate_kernel.cuh"

namespace wllm {
int launch_rotate_bf16(const RotateParams& p, unsigned blocks, int ring_smem, int num_sms, cudaStream_t stream) {
  return launch_rotate_typed<__nv_bfloat16>(p, blocks, ring_smem, num_sms, stream);
}
}  // namespace wllm
