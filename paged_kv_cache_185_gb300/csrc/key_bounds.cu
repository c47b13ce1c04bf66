// key_bounds.cu -- elementwise minimum and maximum of the keys of every cache
// block that new tokens filled, the summary that block selection scores.
//
// Mathematics: lo[d] = min over the block's bs keys of k[d], hi[d] = max; a NaN
// among them makes both NaN.  Both are elements of the cache's own type, so
// nothing is rounded, and for E4M3 codes the order of codes' values is the
// order of the keys (the scale is positive).
//
// Work split: one warp per (filled block, kv head).  The block's rows are one
// contiguous run; a lane owns one 16-byte column and the warp reads 512
// contiguous bytes a load, so a row takes D*elt/16 lanes and the lanes above
// that take further rows, met by shuffles at the end.  Bound: memory, each key
// is read once and a bs/2-th of it written.  16 chunks of 2048 tokens, 8 kv heads
// of 128, bf16 (75 MB): 14.8 us, 0.75 of the measured copy rate; f32 (150 MB)
// 25.0 us, 0.88; E4M3 (37 MB) 12.2 us, 0.45: as many blocks to look up for half the
// bytes, and two conversions a word.  A call that fills 17 blocks, all latency,
// takes 2.0 us.
#include "common.cuh"
#include "launch.h"

namespace wllm {
namespace {

constexpr int kBoundsWarps = 4;
constexpr int kStartsPerThread = 4;  // compared by the CTAs that check them

// Packed extrema of one 32-bit word of elements, NaN carried along.
struct F32Ops {
  static constexpr uint32_t kTop = 0x7f800000u, kBottom = 0xff800000u;  // infinities
  static constexpr int kWords = 1;  // registers that hold one 32-bit word's elements
  static __device__ __forceinline__ void open(uint32_t x, uint32_t (&y)[1]) { y[0] = x; }
  static __device__ __forceinline__ uint32_t shut(const uint32_t (&y)[1]) { return y[0]; }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

struct F16Ops {
  static constexpr uint32_t kTop = 0x7c007c00u, kBottom = 0xfc00fc00u;  // infinities
  static constexpr int kWords = 1;
  static __device__ __forceinline__ void open(uint32_t x, uint32_t (&y)[1]) { y[0] = x; }
  static __device__ __forceinline__ uint32_t shut(const uint32_t (&y)[1]) { return y[0]; }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

struct BF16Ops {
  static constexpr uint32_t kTop = 0x7f807f80u, kBottom = 0xff80ff80u;  // infinities
  static constexpr int kWords = 1;
  static __device__ __forceinline__ void open(uint32_t x, uint32_t (&y)[1]) { y[0] = x; }
  static __device__ __forceinline__ uint32_t shut(const uint32_t (&y)[1]) { return y[0]; }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

// E4M3 codes: widened to f16 pairs and narrowed back, both exact.
struct E4M3Ops {
  static constexpr uint32_t kTop = 0x7c007c00u, kBottom = 0xfc00fc00u;  // infinities
  static constexpr int kWords = 2;
  static __device__ __forceinline__ void open(uint32_t x, uint32_t (&y)[2]) { e4m3x4_to_f16x2x2(x, y[0], y[1]); }
  static __device__ __forceinline__ uint32_t shut(const uint32_t (&y)[2]) {
    uint16_t l, h;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(y[1]));
    return static_cast<uint32_t>(l) | (static_cast<uint32_t>(h) << 16);
  }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) { return F16Ops::lo(a, b); }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return F16Ops::hi(a, b); }
};

// Extrema over the rows of one (block, head) run; the lanes of the first row
// store lo and hi.  `cols`: 16-byte columns of a row, a power of two.
template <typename Ops, int COLS>
__device__ __forceinline__ void bounds_of_block(const uint8_t* src, uint8_t* dst, int bs, int lane) {
  constexpr int kRows = COLS >= 32 ? 1 : 32 / COLS;    // rows of one warp load
  constexpr int kTurns = COLS >= 32 ? COLS / 32 : 1;   // warp loads of one row
  constexpr int kN = 4 * Ops::kWords;
#pragma unroll
  for (int turn = 0; turn < kTurns; ++turn) {
    const int col = COLS >= 32 ? lane + 32 * turn : lane & (COLS - 1);
    const int row0 = COLS >= 32 ? 0 : lane / COLS;
    uint32_t lo[kN], hi[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) lo[n] = Ops::kTop, hi[n] = Ops::kBottom;
    for (int r = row0; r < bs; r += 8 * kRows) {  // bs >= 8 >= kRows: every lane has a row
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i * kRows < bs) x[i] = reinterpret_cast<const uint4*>(src)[(r + i * kRows) * COLS + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r + i * kRows >= bs) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t y[Ops::kWords];
          Ops::open(w[j], y);
#pragma unroll
          for (int e = 0; e < Ops::kWords; ++e) {
            const int n = j * Ops::kWords + e;
            lo[n] = Ops::lo(lo[n], y[e]);
            hi[n] = Ops::hi(hi[n], y[e]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int m = COLS; m < 32; m <<= 1) {
        lo[n] = Ops::lo(lo[n], __shfl_xor_sync(kFullMask, lo[n], m));
        hi[n] = Ops::hi(hi[n], __shfl_xor_sync(kFullMask, hi[n], m));
      }
    if (row0 == 0) {
      uint32_t l[4], h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t y[Ops::kWords], z[Ops::kWords];
#pragma unroll
        for (int e = 0; e < Ops::kWords; ++e) y[e] = lo[j * Ops::kWords + e], z[e] = hi[j * Ops::kWords + e];
        l[j] = Ops::shut(y);
        h[j] = Ops::shut(z);
      }
      reinterpret_cast<uint4*>(dst)[col] = make_uint4(l[0], l[1], l[2], l[3]);
      reinterpret_cast<uint4*>(dst)[COLS + col] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

// Units of the packed form.  Sequence b, whose new tokens are packed rows
// r = qsl[b] - qsl[0] .. qsl[b+1] - qsl[0], owns the unit numbers from
// floor(r / bs) + b on: n tokens fill at most ceil(n / bs) blocks, which is no
// more than the distance to the next sequence's first unit.
template <typename Ops, int COLS>
__global__ void __launch_bounds__(kBoundsWarps * 32) key_bounds_kernel(const BoundsParams p) {
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x < p.check_ctas) {  // starts that decrease are recorded whether or not a unit meets them
#pragma unroll
    for (int k = 0; k < kStartsPerThread; ++k) {
      const int64_t i = (int64_t(blockIdx.x) * kStartsPerThread + k) * blockDim.x + threadIdx.x;
      if (i < p.num_seqs && p.query_start_loc[i + 1] < p.query_start_loc[i]) atomicOr(p.err, kErrLen);
    }
    return;
  }
  const unsigned gw = (blockIdx.x - p.check_ctas) * kBoundsWarps + (threadIdx.x >> 5);
  const unsigned stride = (gridDim.x - p.check_ctas) * kBoundsWarps;
  const int bs = 1 << p.log2_bs;
  int units = p.num_seqs;  // of every head
  int row0 = 0;            // of the first sequence: rows of others may lie before it
  if (p.query_start_loc != nullptr) {
    row0 = p.query_start_loc[0];
    const int64_t total = int64_t(p.query_start_loc[p.num_seqs]) - row0;
    if (total < 0 || total > int64_t(p.num_seqs) * p.max_tokens) {  // more new tokens than the tables can name
      if (gw == 0 && lane == 0) atomicOr(p.err, kErrLen);
      return;
    }
    units += static_cast<int>(total >> p.log2_bs);
  }
  const unsigned heads = p.num_kv_heads;
  const int hop = stride / heads, hop_h = stride % heads;
  for (int slot = gw / heads, h = gw % heads; slot < units; slot += hop, h += hop_h) {
    if (h >= p.num_kv_heads) {
      h -= p.num_kv_heads;
      if (++slot >= units) break;
    }
    int b = slot, n = 1, j = 0;
    if (p.query_start_loc != nullptr) {
      // largest b whose first unit is not behind this one: 32 probes at a time
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool before = at <= hi && ((p.query_start_loc[at] - row0) >> p.log2_bs) + at <= slot;
        const int k = __popc(__ballot_sync(kFullMask, before));
        hi = min(hi, lo + (k + 1) * step - 1);
        lo += k * step;
      }
      b = lo;
      const int first = p.query_start_loc[b] - row0;
      n = p.query_start_loc[b + 1] - row0 - first;
      j = slot - ((first >> p.log2_bs) + b);
    }
    const int len = p.context_lens[b];
    if (n < 0 || n > len || len > p.max_tokens || j < 0) {
      if (!(p.query_start_loc == nullptr && len == 0) && lane == 0) atomicOr(p.err, kErrLen);
      continue;  // an empty sequence of the one-token form has no new token
    }
    const int at = ((len - n) >> p.log2_bs) + j;
    if (at >= (len >> p.log2_bs)) continue;  // not filled yet
    const int id = p.block_tables[b * p.bt_stride + at];
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0) atomicOr(p.err, kErrBlock);
      continue;
    }
    const int64_t run = static_cast<int64_t>(id) * p.num_kv_heads + h;
    bounds_of_block<Ops, COLS>(p.k_cache + run * bs * (COLS * 16), p.bounds + run * 2 * (COLS * 16), bs, lane);
  }
}

template <typename Ops, int COLS>
int launch_one(const BoundsParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_dependent(&key_bounds_kernel<Ops, COLS>, dim3(blocks), dim3(kBoundsWarps * 32), 0, 0, stream, p);
}

template <typename Ops, int ELT>
int launch_dim(const BoundsParams& p, int head_dim, unsigned blocks, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_one<Ops, 64 * ELT / 16>(p, blocks, stream);
    case 128: return launch_one<Ops, 128 * ELT / 16>(p, blocks, stream);
    case 256: return launch_one<Ops, 256 * ELT / 16>(p, blocks, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int launch_key_bounds(int dtype, int head_dim, BoundsParams p, int num_sms, cudaStream_t stream) {
  // one new token a sequence: a warp per (sequence, head), most of which find
  // an open block and leave; packed chunks: how many blocks they fill is on the
  // device, so a resident grid walks over them
  const int64_t resident = int64_t(num_sms) * 12 * kBoundsWarps;
  int64_t warps = int64_t(p.num_seqs) * p.num_kv_heads;
  if (p.query_start_loc != nullptr || warps > (int64_t(1) << 31)) warps = resident;
  // CTAs of their own compare the starts: at the end of the others' walk they took 0.5 us of a call, 3.9 instead of 3.4
  // for 2 chunks of 512
  constexpr int kStarts = kStartsPerThread * kBoundsWarps * 32;
  p.check_ctas = p.query_start_loc != nullptr ? static_cast<unsigned>((int64_t(p.num_seqs) + kStarts - 1) / kStarts) : 0u;
  const unsigned blocks = static_cast<unsigned>((warps + kBoundsWarps - 1) / kBoundsWarps) + p.check_ctas;
  int e;
  switch (dtype) {
    case 0: e = launch_dim<F32Ops, 4>(p, head_dim, blocks, stream); break;
    case 1: e = launch_dim<F16Ops, 2>(p, head_dim, blocks, stream); break;
    case 2: e = launch_dim<BF16Ops, 2>(p, head_dim, blocks, stream); break;
    case 5: e = launch_dim<E4M3Ops, 1>(p, head_dim, blocks, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
