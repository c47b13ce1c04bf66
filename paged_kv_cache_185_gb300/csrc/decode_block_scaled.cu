// decode_block_scaled.cu -- single-query attention over a paged cache of E4M3
// codes with a scale for each block and kv head.
//
// Mathematics: token t of a sequence has K_t = ks_t k_t and V_t = vs_t v_t, with
// k_t, v_t its codes' values and ks_t, vs_t its block's scales.  With the base 2,
// x_t = scale log2(e) ks_t (q . k_t) + log2(vs_t) and a running maximum m of x,
//   w_t = 2^(x_t - m),  O <- O 2^(m - m') + sum_t w_t v_t,  l <- ... + sum_t w_t / vs_t,
// and out = O / l: the value's scale is part of the weight, so that one maximum
// serves the products (w <= 1 whatever the scales) and the sum, which counts the
// weights without it.  log2(vs) of a power of two is exact.
//
// A warp takes units of 32 tokens (16 with head_dim 256) through its own ring of
// shared-memory stages, filled by TMA (128-byte swizzle) and, for the unit's
// scales, by 4-byte asynchronous copies on the same mbarrier.  The products are
// those of the fp8 decode (mma_e4m3.cuh): codes widened to f16 in registers, which
// is exact, S^T = K Q^T and O^T += V^T P^T by mma.sync m16n8k16 with 8 or 16 query
// heads of a kv head as columns.  Query rows go to f16 after a power of two was
// divided out, so bf16 rows of any size do.  Weights, times 2^14, go to the products as
// two words of f16 (what the first leaves off is the second): 22 bits, or 2^-39 of the
// largest.  One word put up to 2^-12 of each weight into the output, as much as the
// rounding of an f16 output.  The second product costs little where memory sets the
// pace: 8 sequences of 32K to 131K 225 us with it and 228 without, 256 of 300 to 6000
// 147.6 and 145.6, one of 16000 12.5 and 12.5.
//
// Work split: all units, ordered by sequence, kv head and head tile, are cut into
// as many equal runs as CTAs fit the GPU, so that rows of any length fill it
// evenly; a CTA's warps take its units in turn.  At the end of a row each warp
// leaves its results in shared memory and goes on; behind its next unit it merges a
// quarter of what all left, so hardly a warp waits for another.  A row that several
// runs share is left as partial results (two at most a run: the row it begins in and
// the row it ends in), which a second kernel, a programmatic dependent, merges in
// their order: the result does not depend on timing, and nothing in the workspace
// outlives the call.
//
// Bound: memory, each code is read once.  8 sequences of 32K to 131K tokens, 32/8
// heads of 128 (1407 MB): 225 us, 0.94 of the measured copy rate; 256 of 300 to 6000,
// 28/4 heads (829 MB): 148 us, 0.84, the rest the setup and the ends of 4 rows a CTA;
// one of 16000, 32/4 heads of 64 (8 MB): 12.5 us, all latency.  What it took (with
// weights of one word): warps that wait for nothing at a row's end 171 us instead of
// 235 (256 sequences), the quarters merged behind the next unit 153, partial results
// merged by the second kernel instead of the CTA that counts in last, and entries
// looked up 8 units at a time, 144 (16000 tokens: 17.0 and 12.3).
#include <atomic>
#include <climits>

#include "decode_kernel.cuh"
#include "launch.h"
#include "mma_e4m3.cuh"

namespace wllm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kWeightShift = 14.f;
constexpr int kMostCtas = 4;      // of an SM
constexpr int kLeastUnits = 4;    // of a warp, before another CTA takes part (where rows have as many)

template <int D, int NT>
struct Shape {
  using G = Geom<uint8_t, D>;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kSub = D == 256 ? 1 : 2;          // 16-token tiles of a unit
  static constexpr int kUnit = 16 * kSub;                // its tokens
  static constexpr int kOctets = 2 * kSub;               // runs of 8 tokens, each of one block
  static constexpr int kSide = kSub * G::kTileBytes;     // a unit's K (or V)
  static constexpr int kStage = 2 * kSide;
  static constexpr int kStages = D == 64 ? 4 : D * NT == 128 ? 3 : 2;
  static constexpr int kRing = kStages * kStage;         // a warp's
  static constexpr int kScales = 8;                      // of a stage: K's octets at 0, V's at 4
  static constexpr int kOut = kHeads * D;                // a warp's outputs
  static constexpr int kPart = kOut + 2 * kHeads;        // floats of a partial result: outputs, maxima, sums
};

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kNone = -3.402823466e38f;  // the maximum of nothing: 2^(kNone - m) is 0

__device__ __forceinline__ int length_of(const ScaledDecodeParams& p, int b) {
  return min(max(p.context_lens[b], 0), p.max_tokens);
}

// x / y of numbers that are not negative; 32-bit division where they allow it.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// A CTA's run of units as segments: the units of one row (sequence, kv head, head
// tile) that are in it.  The same in every lane.
template <int UNIT>
struct Segments {
  long long remaining;  // units of the run from this segment on
  int b, h, tile;       // the row
  int len, units;       // the sequence's
  int at, count;        // the segment: units at .. at + count - 1 of the row
  int turn;             // the run's units before it, modulo the warps
  int window, lens;     // lengths of sequences window .. window + 31, a lane each

  __device__ __forceinline__ void look_at(const ScaledDecodeParams& p, int i) {
    window = i & ~31;
    const int mine = window + (threadIdx.x & 31);
    lens = mine < p.num_seqs ? length_of(p, mine) : 0;
  }
  __device__ __forceinline__ int length(const ScaledDecodeParams& p, int i) {
    if ((i & ~31) != window) look_at(p, i);
    return __shfl_sync(kFullMask, lens, i & 31);
  }
  // A run that begins with unit `offset` of sequence `first`, which has `length` tokens.
  __device__ __forceinline__ void start(const ScaledDecodeParams& p, int first, int length, long long offset, long long run) {
    b = first, len = length, turn = 0, remaining = run;
    look_at(p, first);
    units = (len + UNIT - 1) / UNIT;
    const int row = static_cast<int>(quotient(offset, units));
    at = static_cast<int>(offset - static_cast<long long>(row) * units);
    h = row / p.head_tiles, tile = row - h * p.head_tiles;
    count = static_cast<int>(min(static_cast<long long>(units - at), remaining));
  }
  __device__ __forceinline__ bool next(const ScaledDecodeParams& p) {
    remaining -= count;
    turn = (turn + count) & (kWarps - 1);
    if (remaining <= 0) return false;
    at = 0;
    if (++tile == p.head_tiles) tile = 0, ++h;
    if (h == p.num_kv_heads) {
      h = 0;
      do {
        if (++b >= p.num_seqs) return false;
        len = length(p, b);
      } while (len == 0);
      units = (len + UNIT - 1) / UNIT;
    }
    count = static_cast<int>(min(static_cast<long long>(units), remaining));
    return true;
  }
  // this warp's first unit of the segment, counted from `at`
  __device__ __forceinline__ int first_of(int warp) const { return (warp - turn) & (kWarps - 1); }
};

// The products of one warp and their running state.
template <int D, int NT>
struct Math {
  using S = Shape<D, NT>;
  static constexpr int kKS = D / 16;
  uint32_t q[NT][kKS][2];
  float o[kKS][NT][4], m[NT][2], l[NT][2], factor[NT][2];  // factor: of a raw score, without the block's scale

  // Elements of heads 0 .. heads-1 from `src` on, rows `sh` elements apart, as they are: asked for here, ...
  __device__ __forceinline__ void ask_q(const uint16_t* src, int64_t sh, int heads, bool pairs) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool valid = 8 * nt + g < heads;
      const uint16_t* at = src + (valid ? 8 * nt + g : 0) * sh + 4 * c;
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint16_t* d = at + 16 * s + 2 * e;
          const uint32_t x = pairs ? *reinterpret_cast<const uint32_t*>(d) : d[0] | static_cast<uint32_t>(d[1]) << 16;
          q[nt][s][e] = x;
        }
    }
  }
  // ... and taken to f16 here (columns without a head become zero); the state begins anew.
  template <typename T>
  __device__ __forceinline__ void take_q(int heads, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (8 * nt + g >= heads) {
#pragma unroll
        for (int s = 0; s < kKS; ++s) q[nt][s][0] = q[nt][s][1] = 0u;
      }
      uint32_t most = 0u;  // magnitudes' order is their bits'
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) most = max(most, max(q[nt][s][e] & 0x7fffu, (q[nt][s][e] >> 16) & 0x7fffu));
      most = max(most, __shfl_xor_sync(kFullMask, most, 1));
      most = max(most, __shfl_xor_sync(kFullMask, most, 2));
      // largest magnitude to 2^14 .. 2^15; exponent fields of binary32
      const uint16_t top_bits = static_cast<uint16_t>(most);
      const float top = to_f32(*reinterpret_cast<const T*>(&top_bits));
      const int field = min(max(127 + 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
      const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
      const float undo = __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * scale_log2;
      const float down = fminf(fmaxf(undo, -kMostRowFactor), kMostRowFactor);
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const T* x = reinterpret_cast<const T*>(&q[nt][s][e]);
          q[nt][s][e] = Mma<__half>::pack(to_f32(x[0]) * up, to_f32(x[1]) * up);
        }
      factor[nt][0] = __shfl_sync(kFullMask, down, 8 * c);
      factor[nt][1] = __shfl_sync(kFullMask, down, 8 * c + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = kNone, l[nt][i] = 0.f;
#pragma unroll
      for (int t = 0; t < kKS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
    }
  }

  // A unit whose K codes are at shared address kt and V codes behind them, the
  // first `live` tokens of it; `scales`: its octets' scales.
  __device__ __forceinline__ void step(uint32_t kt, const float* scales, int live) {
    constexpr int kTile = S::G::kTileBytes;
    const uint32_t vt = kt + S::kSide;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // lanes 0-7 / 8-15 / 16-23 / 24-31 address rows 0-7 / 8-15 of a chunk, then of the next
    const int a_row = (lane & 7) + (((lane >> 3) & 1) << 3), a_chunk = lane >> 4;
    float s[S::kSub][NT][4];
#pragma unroll
    for (int j = 0; j < S::kSub; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][nt][e] = 0.f;
#pragma unroll
    for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
      for (int j = 0; j < S::kSub; ++j) {
        uint32_t r[4];
        ldsm_x4(kt + j * kTile + code_offset<D>(a_row, 2 * kp + a_chunk), r);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a[4];
          e4m3x4_to_f16x2x2(r[2 * half], a[0], a[2]);
          e4m3x4_to_f16x2x2(r[2 * half + 1], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) Mma<__half>::run(s[j][nt], a, q[nt][2 * kp + half]);
        }
      }
    // this lane's tokens: g and g + 8 of each tile, in octets 2j and 2j + 1
    float ks[S::kOctets], add[S::kOctets], inv[S::kOctets];
#pragma unroll
    for (int i = 0; i < S::kOctets; ++i) {
      ks[i] = scale_in_range(scales[i]);
      const float vs = scale_in_range(scales[4 + i]);
      add[i] = lg2(vs);
      inv[i] = rcp(vs);
    }
    uint32_t w[S::kSub][NT][2], rest[S::kSub][NT][2];  // the weights' two words
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2] = {m[nt][0], m[nt][1]};
#pragma unroll
      for (int j = 0; j < S::kSub; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 2 * j + (e >> 1);
          s[j][nt][e] = fmaf(s[j][nt][e], factor[nt][e & 1] * ks[i], add[i]);
        }
      if (live < S::kUnit) {
#pragma unroll
        for (int j = 0; j < S::kSub; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + 8 * (e >> 1) + g >= live) s[j][nt][e] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < S::kSub; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[j][nt][e]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(kFullMask, top[i], off));
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        alpha[nt][i] = ex2_approx(m[nt][i] - top[i]);
        moved |= top[i] > m[nt][i];
        m[nt][i] = top[i];
        base[i] = top[i] - kWeightShift;
        l[nt][i] *= alpha[nt][i];
      }
#pragma unroll
      for (int j = 0; j < S::kSub; ++j) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = ex2_approx(s[j][nt][i] - base[i & 1]);
          l[nt][i & 1] = fmaf(e[i], inv[2 * j + (i >> 1)], l[nt][i & 1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t first = Mma<__half>::pack(e[2 * i], e[2 * i + 1]);
          const float2 taken = __half22float2(*reinterpret_cast<const __half2*>(&first));
          w[j][nt][i] = movmatrix_trans(first);
          rest[j][nt][i] = movmatrix_trans(Mma<__half>::pack(e[2 * i] - taken.x, e[2 * i + 1] - taken.y));
        }
      }
    }
    if (__any_sync(kFullMask, moved)) {
#pragma unroll
      for (int t = 0; t < kKS; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][nt][e] *= alpha[nt][e & 1];
    }
    // O^T += V^T P^T; V rows past the context are zeroed (they may hold anything)
#pragma unroll
    for (int j = 0; j < S::kSub; ++j) {
      const int left = live - 16 * j;
      const bool tail = left < 16;
      const uint32_t keep_lo = (2 * c < left ? 0x0000ffffu : 0u) | (2 * c + 1 < left ? 0xffff0000u : 0u);
      const uint32_t keep_hi = (2 * c + 8 < left ? 0x0000ffffu : 0u) | (2 * c + 9 < left ? 0xffff0000u : 0u);
#pragma unroll
      for (int mp = 0; mp < D / 32; ++mp) {
        uint32_t r[4];  // tokens 0-7 / 8-15 of chunk 2mp, then of chunk 2mp + 1
        ldsm_x4_trans(vt + j * kTile + code_offset<D>(a_row, 2 * mp + a_chunk), r);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // bytes (t, e), (t, e+1), (t+1, e), (t+1, e+1) -> (t, e), (t+1, e), (t, e+1), (t+1, e+1)
          uint32_t a[4];
          e4m3x4_to_f16x2x2(__byte_perm(r[2 * half], 0u, 0x3120), a[0], a[1]);
          e4m3x4_to_f16x2x2(__byte_perm(r[2 * half + 1], 0u, 0x3120), a[2], a[3]);
          if (tail) a[0] &= keep_lo, a[1] &= keep_lo, a[2] &= keep_hi, a[3] &= keep_hi;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            Mma<__half>::run(o[2 * mp + half][nt], a, w[j][nt]);
            Mma<__half>::run(o[2 * mp + half][nt], a, rest[j][nt]);
          }
        }
      }
    }
  }

  // The sums over all lanes' tokens, in every lane of a column.
  __device__ __forceinline__ void sum_up() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][i] += __shfl_xor_sync(kFullMask, l[nt][i], off);
  }
  // Outputs in the fragments' order (16 bytes a lane and store), maxima and sums by head.
  __device__ __forceinline__ void store(float4* at, float* ms, float* ls) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (g == 0) ms[8 * nt + 2 * c + i] = m[nt][i], ls[8 * nt + 2 * c + i] = l[nt][i];
#pragma unroll
      for (int t = 0; t < kKS; ++t) at[(nt * kKS + t) * 32 + lane] = make_float4(o[t][nt][0], o[t][nt][1], o[t][nt][2], o[t][nt][3]);
    }
  }
};

// Two neighbouring outputs.
__device__ __forceinline__ void store_out(const ScaledDecodeParams& p, int64_t at, float x, float y) {
  const uint32_t w = p.bf16 ? Mma<__nv_bfloat16>::pack(x, y) : Mma<__half>::pack(x, y);
  uint16_t* out = static_cast<uint16_t*>(p.out) + at;
  if (p.o_pairs) {
    *reinterpret_cast<uint32_t*>(out) = w;
  } else {
    out[0] = static_cast<uint16_t>(w), out[1] = static_cast<uint16_t>(w >> 16);
  }
}

// A row that runs share, left to the merge by the run that has its first unit
// (0 sharers: the run leaves none).
struct SharedRow {
  int b, h, tile, sharers;
};

// What a CTA has in shared memory.
template <int D, int NT>
struct Shared {
  using S = Shape<D, NT>;
  uint8_t ring[kWarps][S::kRing];
  float4 out[kWarps][S::kOut / 4];  // the warps' outputs of the segment that has ended, in the fragments' order, ...
  float m[kWarps][S::kHeads], l[kWarps][S::kHeads];  // ... maxima and sums, ...
  int has[kWarps];                  // ... and whether there are any
  float scales[kWarps][S::kStages][S::kScales];
  uint64_t bars[kWarps][S::kStages], stored, free;
  long long sums[kWarps], first_offset;
  int first_seq, first_len;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    decode_block_scaled_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                               const ScaledDecodeParams p) {
  using S = Shape<D, NT>;
  using G = typename S::G;
  constexpr int kKS = D / 16;
  extern __shared__ __align__(1024) uint8_t raw[];  // swizzled boxes start at 1024 bytes
  Shared<D, NT>& sh = *reinterpret_cast<Shared<D, NT>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = sh.ring[warp];
  // a stage: the expected bytes of its copies, and eight lanes' copies of scales
  if (lane < S::kStages) mbar_init(smem_u32(&sh.bars[warp][lane]), 1 + S::kScales);
  if (tid == 0) {
    mbar_init(smem_u32(&sh.stored), kWarps);
    mbar_init(smem_u32(&sh.free), kWarps);
  }
  fence_mbar_init();
  if (lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
  __syncwarp();
  grid_wait();
  grid_launch_dependents();

  // --- this CTA's run of units (it leaves no shared row until it finds one)
  if (tid == 0) static_cast<SharedRow*>(p.rows)[blockIdx.x] = SharedRow{0, 0, 0, 0};
  const int rows = p.num_kv_heads * p.head_tiles;
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  long long mine = 0;
#pragma unroll 4
  for (int b = s0; b < s1; ++b) mine += (length_of(p, b) + S::kUnit - 1) / S::kUnit;
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kFullMask, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) sh.sums[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sh.sums[w];
    total += sh.sums[w];
  }
  // a run has the units of a mean row at least, up to kLeastUnits a warp: a long row in fewer pieces has fewer results to
  // merge, but a CTA with many short rows has an end for each.  One sequence of 16000 tokens, 4 kv heads of 64: 12.4 us with
  // 1 unit a warp at least, 12.5 with 4, 16.1 with 8; 96 of 4 tokens, 4 kv heads of 128: 9.6 us, 41 without the mean row
  const long long least = max(1ll, min(static_cast<long long>(kWarps * kLeastUnits), quotient(total, p.num_seqs)));
  total *= rows;
  const long long ctas = max(1ll, min(static_cast<long long>(gridDim.x), quotient(total, least)));
  const long long c_id = blockIdx.x;
  const long long u0 = c_id < ctas ? quotient(total * c_id, ctas) : total, u1 = c_id < ctas ? quotient(total * (c_id + 1), ctas) : total;
  if (u0 < u1 && (upto - mine) * rows <= u0 && u0 < upto * rows) {
    long long before = upto - mine;
    for (int b = s0; b < s1; ++b) {
      const int len = length_of(p, b), units = (len + S::kUnit - 1) / S::kUnit;
      if (u0 < (before + units) * rows) {
        sh.first_seq = b, sh.first_len = len, sh.first_offset = u0 - before * rows;
        break;
      }
      before += units;
    }
  }
  // empty sequences: zeros, and lengths out of range are recorded
  for (int i = 0; i < per; ++i) {
    const int b = s0 + i;
    const bool ours = b < s1 && static_cast<unsigned>(b) % gridDim.x == blockIdx.x;
    const int stored = ours ? p.context_lens[b] : 0;
    if (stored < 0 || stored > p.max_tokens) atomicOr(p.err, kErrLen);
    unsigned empty = __ballot_sync(kFullMask, ours && min(stored, p.max_tokens) <= 0);
    while (empty != 0u) {
      const int seq = __shfl_sync(kFullMask, b, __ffs(empty) - 1);
      empty &= empty - 1;
      for (int x = lane; x < p.num_q_heads * (D / 2); x += 32)
        store_out(p, seq * p.o_sb + (x / (D / 2)) * p.o_sh + (x % (D / 2)) * 2, 0.f, 0.f);
    }
  }
  __syncthreads();
  if (u0 >= u1) return;

  // --- copies: a cursor of its own runs ahead; the next unit's table entries are asked for one unit early
  Segments<S::kUnit> ahead, seg;
  seg.start(p, sh.first_seq, sh.first_len, sh.first_offset, u1 - u0);
  ahead = seg;
  int ahead_at = ahead.first_of(warp);
  const bool two = p.log2_bs < 4;  // 8-token blocks: two 8-row boxes for 16 tokens
  const int bs_mask = (1 << p.log2_bs) - 1;
  // Table entries of up to 32 / kOctets units of one segment, a lane an octet; the
  // batch behind the current one is asked for when that begins.
  struct Batch {
    int entry;
    int t, len, h;    // first token of the first unit; of how many of the sequence; kv head
    int units;        // 0: none is left
  };
  constexpr int kBatchUnits = 32 / S::kOctets;
  auto look_up = [&](Batch& u) {  // by reference: nothing here waits for the entries
    u.units = 0;
    while (ahead_at >= ahead.count) {
      if (!ahead.next(p)) return;
      ahead_at = ahead.first_of(warp);
    }
    u.units = min(kBatchUnits, (ahead.count - ahead_at + kWarps - 1) / kWarps);
    u.t = (ahead.at + ahead_at) * S::kUnit, u.len = ahead.len, u.h = ahead.h;
    const int t = u.t + (lane / S::kOctets) * (kWarps * S::kUnit) + 8 * (lane % S::kOctets);
    u.entry = 0;
    if (lane < u.units * S::kOctets && t < u.len) u.entry = p.block_tables[ahead.b * p.bt_stride + (t >> p.log2_bs)];
    ahead_at += u.units * kWarps;
  };
  Batch batch{}, later{};
  int in_batch = 0;
  auto copy = [&](int stage) {  // the next unit's
    if (in_batch == batch.units) {
      if (later.units == 0) return;
      batch = later, in_batch = 0;
      if (batch.entry < 0 || batch.entry >= p.num_blocks) {
        atomicOr(p.err, kErrBlock);
        batch.entry = 0;
      }
      look_up(later);
    }
    const int from = in_batch * S::kOctets, unit_t = batch.t + in_batch * (kWarps * S::kUnit);
    ++in_batch;
    const uint32_t bar = smem_u32(&sh.bars[warp][stage]), dst = smem_u32(ring + stage * S::kStage);
    // one box a lane: K or V, column box, 16 tokens (or 8)
    const int x = two ? lane >> 1 : lane, octet_in = two ? lane & 1 : 0;
    const int kv = x & 1, col = (x >> 1) % G::kColBoxes, tile = (x >> 1) / G::kColBoxes;
    const int octet = 2 * tile + octet_in, t = unit_t + 8 * octet;
    const int phys = __shfl_sync(kFullMask, batch.entry, from + (octet & (S::kOctets - 1)));
    const bool box = tile < S::kSub && t < batch.len;
    const uint32_t box_bytes = 128u * (G::kPairRows || two ? 8u : 16u);
    const uint32_t bytes = unit_t + S::kUnit <= batch.len ? static_cast<uint32_t>(S::kStage) : box_bytes * __popc(__ballot_sync(kFullMask, box));
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    if (box) {
      const int at = (batch.h << p.log2_bs) + (t & bs_mask);
      tma_load_3d(dst + kv * S::kSide + tile * G::kTileBytes + col * 2048 + octet_in * 1024, kv ? &vmap : &kmap, bar, col * 128,
                  G::kPairRows ? at >> 1 : at, phys);
    }
    const int of = __shfl_sync(kFullMask, batch.entry, from + (lane & (S::kOctets - 1)));
    if (lane < S::kScales) {
      const int i = lane & 3;
      if (i < S::kOctets && unit_t + 8 * i < batch.len)
        copy4_async(smem_u32(&sh.scales[warp][stage][lane]),
                    (lane < 4 ? p.k_scales : p.v_scales) + int64_t(of) * p.num_kv_heads + batch.h);
      arrive_behind_copies(bar);
    }
  };
  look_up(later);

  int stage = 0;
  uint32_t phase = 0u, turn = 0u;  // of every stage, turned when the ring comes round; of the places, with every segment
  bool lost = false;
  // a wait that runs out: record it, let the copies in flight land (again with a limit), and leave
  auto give_up = [&] {
    if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
    for (int s = 0; s < S::kStages; ++s) mbar_wait_bounded(smem_u32(&sh.bars[warp][s]), s >= stage ? phase : phase ^ 1u, p.wait_limit_ns);
    lost = true;
  };
  Math<D, NT> math;
  auto ask_q = [&] {
    math.ask_q(static_cast<const uint16_t*>(p.q) + seg.b * p.q_sb + (seg.h * p.group + seg.tile * S::kHeads) * p.q_sh, p.q_sh,
               min(S::kHeads, p.group - seg.tile * S::kHeads), p.q_pairs);
  };

  // The segment that ended last: once every warp has stored its results, each
  // merges a quarter of the outputs.  It does so behind its first unit of the next
  // segment, when the others have stored theirs too, so that hardly a warp waits.
  Segments<S::kUnit> ended = seg;
  bool owed = false;
  auto settle = [&] {
    owed = false;
    if (!mbar_wait_warp(smem_u32(&sh.stored), (turn - 1u) & 1u, p.wait_limit_ns)) {
      give_up();
      return;
    }
    const int g = lane >> 2, c = lane & 3;
    const bool whole = ended.count == ended.units;
    const int heads = min(S::kHeads, p.group - ended.tile * S::kHeads);
    const int64_t out_at = ended.b * p.o_sb + (ended.h * p.group + ended.tile * S::kHeads) * p.o_sh;
    long long run_first = 0;  // of a shared row: the first run that has a unit of it
    int sharers = 1;
    float* to = nullptr;
    if (!whole) {
      const long long row_first = u1 - ended.remaining - ended.at;
      run_first = quotient((row_first + 1) * ctas - 1, total);
      sharers = static_cast<int>(quotient((row_first + ended.units) * ctas - 1, total) - run_first) + 1;
      to = p.parts + (2 * c_id + (c_id == run_first ? 1 : 0)) * S::kPart;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // this lane's two heads: their factors for each warp's outputs
      float f[kWarps][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int a = 8 * nt + 2 * c + e;
        float top = kNone, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if (sh.has[w]) top = fmaxf(top, sh.m[w][a]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w][e] = sh.has[w] ? exp2f(sh.m[w][a] - top) : 0.f;
          if (sh.has[w]) sum = fmaf(f[w][e], sh.l[w][a], sum);
        }
        if (!whole && warp == 0 && g == 0) to[S::kOut + a] = top, to[S::kOut + S::kHeads + a] = sum;
        const float by = whole ? 1.f / sum : 1.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) f[w][e] *= by;
      }
#pragma unroll
      for (int i = 0; i < kKS / kWarps; ++i) {
        const int t = warp * (kKS / kWarps) + i;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (!sh.has[w]) continue;
          const float4 x = sh.out[w][(nt * kKS + t) * 32 + lane];
          v[0] = fmaf(f[w][0], x.x, v[0]), v[1] = fmaf(f[w][1], x.y, v[1]);
          v[2] = fmaf(f[w][0], x.z, v[2]), v[3] = fmaf(f[w][1], x.w, v[3]);
        }
        if (whole) {  // entries 0, 2 and 1, 3 are neighbours of heads 2c and 2c + 1
          const int64_t at = out_at + (8 * nt + 2 * c) * p.o_sh + 16 * t + 2 * g;
          if (8 * nt + 2 * c < heads) store_out(p, at, v[0], v[2]);
          if (8 * nt + 2 * c + 1 < heads) store_out(p, at + p.o_sh, v[1], v[3]);
        } else {
          reinterpret_cast<float4*>(to)[(nt * kKS + t) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    if (!whole && c_id == run_first && warp == 0 && lane == 0)
      static_cast<SharedRow*>(p.rows)[c_id] = SharedRow{ended.b, ended.h, ended.tile, sharers};
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.free));
  };

  ask_q();
#pragma unroll 1
  for (int s = 0; s < S::kStages; ++s) copy(s);
  while (true) {
    const int columns = min(S::kHeads, p.group - seg.tile * S::kHeads);
    if (p.bf16) math.template take_q<__nv_bfloat16>(columns, p.scale_log2);
    else math.template take_q<__half>(columns, p.scale_log2);
    int i = seg.first_of(warp);
    const bool any = i < seg.count;
    for (; i < seg.count; i += kWarps) {
      if (!mbar_wait_warp(smem_u32(&sh.bars[warp][stage]), phase, p.wait_limit_ns)) {
        give_up();
        break;
      }
      math.step(smem_u32(ring + stage * S::kStage), sh.scales[warp][stage], seg.len - (seg.at + i) * S::kUnit);
      __syncwarp();  // every lane has read the stage
      copy(stage);
      if (++stage == S::kStages) stage = 0, phase ^= 1u;
      if (owed) {
        settle();
        if (lost) break;
      }
    }
    if (lost) break;
    if (owed) settle();  // no unit of this segment was this warp's
    if (lost) break;
    math.sum_up();
    ended = seg;
    const bool more_segments = seg.next(p);
    if (more_segments) ask_q();  // on its way meanwhile
    // the segment before this one has been merged by every warp
    if (turn > 0u && !mbar_wait_warp(smem_u32(&sh.free), (turn - 1u) & 1u, p.wait_limit_ns)) {
      give_up();
      break;
    }
    if (any) math.store(sh.out[warp], sh.m[warp], sh.l[warp]);
    if (lane == 0) sh.has[warp] = any;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.stored));
    owed = true;
    ++turn;
    if (!more_segments) break;
  }
  if (owed && !lost) settle();
}

// Rows that runs share: CTA i merges the row that run i has the first unit of, the
// partial results in their order.  A lane has outputs of two heads, in the
// fragments' order; each warp takes every fourth partial result.
constexpr int kMergeSplit = 4;
template <int D, int NT>
__global__ void __launch_bounds__(kMergeSplit * 32) merge_block_scaled_kernel(const ScaledDecodeParams p) {
  using S = Shape<D, NT>;
  constexpr int kKS = D / 16, kTiles = NT * kKS, kBatch = D == 64 ? 8 : D == 128 ? 4 : 2;
  __shared__ float4 outs[kMergeSplit][kTiles][32];
  __shared__ float2 ms[kMergeSplit][NT][4], ls[kMergeSplit][NT][4];
  grid_wait();
  grid_launch_dependents();
  const SharedRow row = static_cast<const SharedRow*>(p.rows)[blockIdx.x];
  if (row.sharers == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int64_t first = blockIdx.x;
#pragma unroll 1
  for (int nt = 0; nt < NT; ++nt) {
    const int a = 8 * nt + 2 * c;  // heads a and a + 1
    float top[2] = {kNone, kNone}, sum[2] = {0.f, 0.f}, v[kKS][4];
#pragma unroll
    for (int t = 0; t < kKS; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[t][e] = 0.f;
    for (int s0 = warp; s0 < row.sharers; s0 += kMergeSplit * kBatch) {
      float2 m[kBatch], l[kBatch];
      float4 x[kBatch][kKS];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int s = s0 + k * kMergeSplit;
        m[k] = make_float2(kNone, kNone);
        if (s >= row.sharers) continue;
        const float* from = p.parts + (2 * (first + s) + (s == 0 ? 1 : 0)) * S::kPart;
        m[k] = *reinterpret_cast<const float2*>(from + S::kOut + a);
        l[k] = *reinterpret_cast<const float2*>(from + S::kOut + S::kHeads + a);
#pragma unroll
        for (int t = 0; t < kKS; ++t) x[k][t] = reinterpret_cast<const float4*>(from)[(nt * kKS + t) * 32 + lane];
      }
      float higher[2] = {top[0], top[1]};
#pragma unroll
      for (int k = 0; k < kBatch; ++k) higher[0] = fmaxf(higher[0], m[k].x), higher[1] = fmaxf(higher[1], m[k].y);
      const float f0 = exp2f(top[0] - higher[0]), f1 = exp2f(top[1] - higher[1]);
      top[0] = higher[0], top[1] = higher[1];
      sum[0] *= f0, sum[1] *= f1;
#pragma unroll
      for (int t = 0; t < kKS; ++t) v[t][0] *= f0, v[t][2] *= f0, v[t][1] *= f1, v[t][3] *= f1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (s0 + k * kMergeSplit >= row.sharers) continue;
        const float fx = exp2f(m[k].x - top[0]), fy = exp2f(m[k].y - top[1]);
        sum[0] = fmaf(fx, l[k].x, sum[0]), sum[1] = fmaf(fy, l[k].y, sum[1]);
#pragma unroll
        for (int t = 0; t < kKS; ++t) {
          v[t][0] = fmaf(fx, x[k][t].x, v[t][0]), v[t][2] = fmaf(fx, x[k][t].z, v[t][2]);
          v[t][1] = fmaf(fy, x[k][t].y, v[t][1]), v[t][3] = fmaf(fy, x[k][t].w, v[t][3]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kKS; ++t) outs[warp][nt * kKS + t][lane] = make_float4(v[t][0], v[t][1], v[t][2], v[t][3]);
    if (g == 0) ms[warp][nt][c] = make_float2(top[0], top[1]), ls[warp][nt][c] = make_float2(sum[0], sum[1]);
  }
  __syncthreads();
  const int heads = min(S::kHeads, p.group - row.tile * S::kHeads);
  const int64_t out_at = row.b * p.o_sb + (row.h * p.group + row.tile * S::kHeads) * p.o_sh;
  for (int i = warp; i < kTiles; i += kMergeSplit) {
    const int nt = i / kKS, t = i - nt * kKS, a = 8 * nt + 2 * c;
    float top[2] = {kNone, kNone}, sum[2] = {0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kMergeSplit; ++w) top[0] = fmaxf(top[0], ms[w][nt][c].x), top[1] = fmaxf(top[1], ms[w][nt][c].y);
#pragma unroll
    for (int w = 0; w < kMergeSplit; ++w) {
      const float fx = exp2f(ms[w][nt][c].x - top[0]), fy = exp2f(ms[w][nt][c].y - top[1]);
      const float4 x = outs[w][i][lane];
      sum[0] = fmaf(fx, ls[w][nt][c].x, sum[0]), v[0] = fmaf(fx, x.x, v[0]), v[2] = fmaf(fx, x.z, v[2]);
      sum[1] = fmaf(fy, ls[w][nt][c].y, sum[1]), v[1] = fmaf(fy, x.y, v[1]), v[3] = fmaf(fy, x.w, v[3]);
    }
    const int64_t at = out_at + a * p.o_sh + 16 * t + 2 * g;
    const float by0 = 1.f / sum[0], by1 = 1.f / sum[1];
    if (a < heads) store_out(p, at, v[0] * by0, v[2] * by0);
    if (a + 1 < heads) store_out(p, at + p.o_sh, v[1] * by1, v[3] * by1);
  }
}

constexpr int kMostPart = 2080;  // floats of a partial result of any form

// CTAs of a launch: as many as run at once.
int ctas_of(int num_sms, int resident) { return num_sms * (resident < kMostCtas ? resident : kMostCtas); }

template <int D, int NT>
int launch_tile(const CUtensorMap& kmap, const CUtensorMap& vmap, ScaledDecodeParams p, int num_sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  constexpr int kSmem = static_cast<int>(sizeof(Shared<D, NT>));
  static_assert(S::kPart <= kMostPart, "the workspace has room for every form's partial results");
  const void* kernel = reinterpret_cast<const void*>(&decode_block_scaled_kernel<D, NT>);
  static std::atomic<int> configured[64], found[64];
  int blocks = 0, e = raise_smem_limit(configured, kernel, kSmem);
  if (e != cudaSuccess) return e;
  if ((e = resident_ctas(found, &decode_block_scaled_kernel<D, NT>, kThreads, kSmem, &blocks)) != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>(ctas_of(num_sms, blocks));
  p.rows = reinterpret_cast<uint8_t*>(p.parts) + size_t(ctas) * 2 * S::kPart * sizeof(float);
  e = launch_dependent(&decode_block_scaled_kernel<D, NT>, dim3(ctas), dim3(kThreads), kSmem, 0, stream, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_dependent(&merge_block_scaled_kernel<D, NT>, dim3(ctas), dim3(kMergeSplit * 32), 0, 0, stream, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

size_t decode_block_scaled_workspace(int num_sms) {
  return size_t(ctas_of(num_sms, kMostCtas)) * (2 * kMostPart * sizeof(float) + sizeof(SharedRow));
}

int launch_decode_block_scaled(int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap, ScaledDecodeParams p, int num_sms,
                               cudaStream_t stream) {
  // two tiles of 8 query heads share the widened codes where registers allow
  const bool wide = p.group > 8 && head_dim <= 128;
  p.head_tiles = (p.group + (wide ? 15 : 7)) / (wide ? 16 : 8);
  int e = cudaErrorInvalidValue;
  switch (head_dim) {
    case 64: e = wide ? launch_tile<64, 2>(kmap, vmap, p, num_sms, stream) : launch_tile<64, 1>(kmap, vmap, p, num_sms, stream); break;
    case 128: e = wide ? launch_tile<128, 2>(kmap, vmap, p, num_sms, stream) : launch_tile<128, 1>(kmap, vmap, p, num_sms, stream); break;
    case 256: e = launch_tile<256, 1>(kmap, vmap, p, num_sms, stream); break;
  }
  return e;
}

}  // namespace wllm
