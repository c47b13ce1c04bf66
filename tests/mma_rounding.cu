// Two chained mma.sync m16n8k16 from a zero accumulator, as block selection uses them: A [n][2][16][16] and
// B [n][2][16][8] of 16-bit elements, D [n][16][8] binary32.  One warp a tile.
#include "common.cuh"

namespace {

template <typename T>
__global__ void chain(const uint16_t* a, const uint16_t* b, float* d) {
  const int lane = threadIdx.x, g = lane >> 2, c = lane & 3;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < 2; ++s) {
    const uint16_t* at = a + (2 * blockIdx.x + s) * 256;
    const uint16_t* bt = b + (2 * blockIdx.x + s) * 128;
    auto pair = [](uint16_t lo, uint16_t hi) { return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16); };
    uint32_t af[4], bf[2];
    for (int i = 0; i < 4; ++i) {  // rows g and g + 8, k 2c and 2c + 1, then 2c + 8 and 2c + 9
      const uint16_t* x = at + (g + 8 * (i & 1)) * 16 + 2 * c + 8 * (i >> 1);
      af[i] = pair(x[0], x[1]);
    }
    for (int i = 0; i < 2; ++i) {
      const uint16_t* x = bt + (2 * c + 8 * i) * 8 + g;
      bf[i] = pair(x[0], x[8]);
    }
    wllm::Mma<T>::run(acc, af, bf);
  }
  float* out = d + blockIdx.x * 128;
  out[g * 8 + 2 * c] = acc[0], out[g * 8 + 2 * c + 1] = acc[1];
  out[(g + 8) * 8 + 2 * c] = acc[2], out[(g + 8) * 8 + 2 * c + 1] = acc[3];
}

}  // namespace

extern "C" int mma_chain(int bf16, int tiles, const void* a, const void* b, void* d) {
  const uint16_t *x = static_cast<const uint16_t*>(a), *y = static_cast<const uint16_t*>(b);
  if (bf16)
    chain<__nv_bfloat16><<<tiles, 32>>>(x, y, static_cast<float*>(d));
  else
    chain<__half><<<tiles, 32>>>(x, y, static_cast<float*>(d));
  return cudaDeviceSynchronize();
}
