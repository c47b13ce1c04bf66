// rotate.cu -- which form of the rotary append runs (rotate_kernel.cuh).
#include "launch.h"

namespace wllm {

// `ring_smem` > 0: the resident form with that much shared memory.
int launch_rotate_f32(const RotateParams&, unsigned, int, int, cudaStream_t);
int launch_rotate_f16(const RotateParams&, unsigned, int, int, cudaStream_t);
int launch_rotate_bf16(const RotateParams&, unsigned, int, int, cudaStream_t);

int launch_rotate(RotateParams p, int num_sms, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 16 < p.head_dim) lanes *= 2;
  p.row_lanes = lanes;
  const int rows_per_step = 32 / lanes;
  const int steps = (p.num_q_heads + rows_per_step - 1) / rows_per_step + 2 * ((p.num_kv_heads + rows_per_step - 1) / rows_per_step);
  const int64_t token_bytes = int64_t(p.num_q_heads + 2 * p.num_kv_heads) * p.head_dim * (p.src_dtype == 0 ? 4 : 2) +
                              int64_t(p.num_axes) * p.rot_dim * 4;
  // The resident form where every SM has a token and the tokens' steps, one a warp,
  // no longer fit the SMs at once (16 warps each).  GPU time with norms, spread over
  // warps and resident: 28/4 heads of 128, bf16: 256 tokens 3.3 and 4.0 us, 280: 5.5
  // and 3.9, 1024: 9.8 and 5.3, 4096: 24.6 and 16.7; 32/8 of 64, f16: 400 tokens
  // (just fitting) 3.4 and 3.7; 128/8 of 128: 100 tokens 5.9 and 6.8.
  const bool many = p.num_tokens >= num_sms && int64_t(p.num_tokens) * steps > int64_t(num_sms) * 16;
  const bool ring = many && p.vec && p.table_vec && 2 * token_bytes <= 100 * 1024;
  const int ring_smem = ring ? static_cast<int>(2 * token_bytes + 2 * p.head_dim * 4) : 0;  // and the weights
  // otherwise one warp walks over a token's rows once the tokens alone give every
  // SM 32 warps; below that its steps are spread, down to one a warp
  int64_t w = (int64_t(num_sms) * 32 + p.num_tokens - 1) / p.num_tokens;
  if (w > steps) w = steps;
  p.warps_per_token = static_cast<int>(w < 1 ? 1 : w);
  const int64_t warps = int64_t(p.num_tokens) * p.warps_per_token;
  const unsigned blocks = static_cast<unsigned>((warps + kRotateWarps - 1) / kRotateWarps);
  int e = cudaErrorInvalidValue;
  if (p.src_dtype == 0) e = launch_rotate_f32(p, blocks, ring_smem, num_sms, stream);
  if (p.src_dtype == 1) e = launch_rotate_f16(p, blocks, ring_smem, num_sms, stream);
  if (p.src_dtype == 2) e = launch_rotate_bf16(p, blocks, ring_smem, num_sms, stream);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
