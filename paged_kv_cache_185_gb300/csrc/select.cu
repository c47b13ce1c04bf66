// select.cu -- the blocks that a decode over a long context has to read.
//
// Mathematics.  Block j of one kv head has bounds lo_j <= k <= hi_j of its
// keys, so a query head's largest score in it is at most
// sum_d max(q_d lo_jd, q_d hi_jd).  Summed over the G query heads of the group
// that is one product with a vector that the blocks share:
//   s_j = sum_d up_d hi_jd + down_d lo_jd,
//   up = sum_h max(q_h, 0), down = sum_h min(q_h, 0).
// Kept are the first `sink` blocks, the last `recent` ones and, of the others,
// those with the largest s_j (NaN as +inf, ties to the lowest j), top in all.
//
// The scores are summed in binary32 with an error of at most
//   E = c 2^-24 sum_i |w_i b_i|,
// so blocks whose scores differ by more than 2 E are in their true order.  The
// choice between the few blocks that lie within 2 E of the border is made from
// their scores in binary64, where the products of 16-bit elements and their
// sums are exact for all but extreme exponents: as far as E holds, the selection
// is the definition's, whatever the order of the sums.
//
// 16-bit and E4M3 bounds are scored on tensor cores (mma.sync m16n8k16): 16
// blocks' bounds are the A operand and B's first three columns are the weights split into three 16-bit words whose sum has
// their 24 bits, so every product is exact.  An instruction adds 16 products to
// the running sum, and no document bounds the error of that sum: what is assumed
// is that at least 22 bits of each of its 17 terms are kept, an error of at most
// 17 * 2^-22 of the magnitudes in it.  Two instructions at a time start
// from zero and their sums are added in binary32, so those magnitudes are two
// steps' and not the whole row's: 136 2^-24 of all of them (measured over random,
// cancelling and uneven products: at most 8 2^-24, which a test keeps watch on),
// 2D/32 additions, the sum of the columns and the G additions of a weight:
// c = G + 136 + 2D/32 + 8
// (one chain over the row would need 68 for each of its 2D/16 instructions, and
// with it 6 times as many binary64 scores).  E4M3 codes are
// widened to f16, exactly; three f16 words, scaled so that the largest weight is
// near 2^14, leave off at most 2^-38 of it, which is far inside the same c.
// F32 bounds take binary32 FMA: c = G + 44 (chains of 32, 5 sums across lanes).
//
// Work split: a cluster of 1 to 8 CTAs per (sequence, kv head), each with a
// share of the blocks, so a long row is on many SMs and the selection still
// needs neither a second launch nor a workspace.  The scoring
// warps of a CTA have two halves of a turn (16 or 32 blocks' minima and their
// maxima) in shared memory each, filled by asynchronous copies, one half while
// the other is multiplied, rows with 16 bytes of padding behind them, so that
// ldmatrix reads eight blocks' chunks without a bank conflict.  The
// scores go straight to the first CTA's shared memory.  That CTA alone finds the
// border with one 1024-bin histogram between the extremes, settles the blocks at
// the border (a handful, 8 lanes each) and writes the chosen ones in ascending
// order: one barrier of the cluster in all, where every step shared by its CTAs
// would cost another (the first form had six, 10 us of them).  Bound: memory,
// the bounds are read once.  Measured, 8 sequences of 32K to 131K tokens, 8 kv
// heads of 128, bf16 (176 MB of bounds): 46.4 us, of which a row's CTAs score for
// 20 us on average and 31 us in the longest row; before that come 5 us of
// lookups, first copies and weights, after it 6 us of border and list on one CTA.  Pairing the longest row with the
// shortest in one cluster evens the scores out, but its clusters finish two rows
// after one another's scores: 47.2 us, and 1.2 us more wherever it does not apply.
// The scores' room is that of the table's width, whatever the lengths, in every
// CTA: tables of some 8,000 blocks and more leave an SM one CTA instead of two (64
// sequences over E4M3: 26.1 us at widths from 1,481 to 8,192, 33.9 from 16,384 on;
// the case above 46.4 and 58.4).
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <limits.h>

#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace wllm {
namespace {

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 1024;
constexpr int kWindow = 256;          // border blocks ranked against each other; more go through digit passes
constexpr int kMaxCluster = 8;

// Of the first CTA once the scores are there, in the place of the rings.
struct alignas(16) SelectShared {
  uint32_t hist[kBins];
  uint32_t warp_sum[kSelectWarps];
  double win_score[kWindow];
  float near_score[kWindow];          // scores around the border and their blocks
  int near_at[kWindow];
  int win_at[kWindow];                // those within the error of the border
  int near_count, win_count, sure_count;
  int found_bin, found_above;
  float border;
};

// Doubles (without NaN) to integers of the same order.
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));  // -0 is 0
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ float element(const uint8_t* base, int i, uint8_t) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(base[i], __NV_E4M3);
  return __half2float(__half(h));
}
template <typename T>
__device__ __forceinline__ float element(const uint8_t* base, int i, T) {
  return to_f32(reinterpret_cast<const T*>(base)[i]);
}

// Exclusive sum of one value a thread over the CTA; *total receives the sum.
__device__ __forceinline__ uint32_t block_scan(SelectShared& sh, uint32_t x, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t y = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t z = __shfl_up_sync(kFullMask, y, m);
    if (lane >= m) y += z;
  }
  __syncthreads();
  if (lane == 31) sh.warp_sum[warp] = y;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    const uint32_t s = sh.warp_sum[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + y - x;
}

// A candidate's score by 8 lanes, four candidates a warp at a time, as the time
// is that of their loads.  All lanes call it.  EXACT: in binary64.  Otherwise as
// the sum of two binary32 numbers: products with their rounding errors (fma),
// sums with theirs (Knuth's two-sum), the errors added up in binary32.  Those
// additions are off by at most 2^-24 of a sum of errors of at most n 2^-24 A
// each, n <= 70 of them: under 2^-35 A in all, A = sum_i |w_i b_i|.  (Binary64
// runs at a 64th of binary32's rate here: a dozen exact scores took 15 us.)
template <typename B, int D, bool EXACT>
__device__ __forceinline__ double fine_score(const uint8_t* src, const float2* w, int lane) {
  constexpr int kE = 16 / static_cast<int>(sizeof(B)), kLoads = 2 * D / (8 * kE);
  uint4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) x[i] = reinterpret_cast<const uint4*>(src)[8 * i + (lane & 7)];
  double s = 0.0;
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int k = 0; k < kE; ++k) {
      const float2 f = w[(8 * i + (lane & 7)) * kE + k];
      const float v = element(reinterpret_cast<const uint8_t*>(&x[i]), k, B());
      if constexpr (EXACT) {
        s = fma(static_cast<double>(f.x) + static_cast<double>(f.y), static_cast<double>(v), s);
      } else {
        const float prod = __fmul_rn(f.x, v), off = __fmaf_rn(f.x, v, -prod);
        const float sum = __fadd_rn(hi, prod), z = __fsub_rn(sum, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, z)), __fsub_rn(prod, z));
        lo = __fadd_rn(lo, __fadd_rn(err, __fmaf_rn(f.y, v, off)));
        hi = sum;
      }
    }
#pragma unroll
  for (int m = 4; m > 0; m >>= 1) {
    if constexpr (EXACT) {
      s += __shfl_xor_sync(kFullMask, s, m);
    } else {
      const float h = __shfl_xor_sync(kFullMask, hi, m), l = __shfl_xor_sync(kFullMask, lo, m);
      const float sum = __fadd_rn(hi, h), z = __fsub_rn(sum, hi);
      lo = __fadd_rn(__fadd_rn(lo, l), __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, z)), __fsub_rn(h, z)));
      hi = sum;
    }
  }
  if constexpr (!EXACT) return static_cast<double>(hi) + static_cast<double>(lo);
  return s != s ? static_cast<double>(INFINITY) : s;
}

// The `left`-th largest of key[j] over the set bits j of `bits`; *left becomes
// how many of the keys equal to it are among the `left` largest.
__device__ __forceinline__ uint32_t digit_cut(SelectShared& sh, const uint32_t* key, const uint32_t* bits, int words,
                                              int* left) {
  static_assert(kSelectThreads == 256, "one digit value a thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t want = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    sh.hist[tid] = 0;
    __syncthreads();
    for (int i = warp; i < words; i += kSelectWarps) {
      const uint32_t k = key[i * 32 + lane];
      if (((bits[i] >> lane) & 1u) && (shift == 24 || (k >> (shift + 8)) == (want >> (shift + 8))))
        atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    const uint32_t c = sh.hist[255 - tid];
    uint32_t total;
    const uint32_t before = block_scan(sh, c, &total);
    if (before < static_cast<uint32_t>(*left) && before + c >= static_cast<uint32_t>(*left)) {
      sh.found_bin = 255 - tid;
      sh.found_above = static_cast<int>(before);
    }
    __syncthreads();
    *left -= sh.found_above;
    want |= static_cast<uint32_t>(sh.found_bin) << shift;
  }
  return want;
}

// What a warp found out about its scores.
struct ScoreStats {
  float least = INFINITY, greatest = -INFINITY;
  float mag = 0.f;    // bound on sum_i |w_i b_ji| of every block
  bool odd = false;   // an infinite or NaN score
  __device__ __forceinline__ void add(float s) {
    least = fminf(least, s);
    greatest = fmaxf(greatest, s);
    odd |= !(fabsf(s) < INFINITY);
  }
};

// Physical block of candidate j; one outside the pool is recorded and read as block 0.
__device__ __forceinline__ int physical(const SelectParams& p, const int32_t* table, int j, int cands, bool record) {
  if (j >= cands) return 0;
  const int id = table[j];
  if (id >= 0 && id < p.num_blocks) return id;
  if (record) atomicOr(p.err, kErrBlock);
  return 0;
}

// Larger of two pairs of 16-bit integers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// d = a b with mma.sync m16n8k16.
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], const uint2& b, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
}
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], const uint2& b, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
}

// The weights in three words of type M, what is left in *rest.
template <typename M>
__device__ __forceinline__ M split_word(float x, float* rest) {
  const M y = from_f32<M>(x);
  *rest = x - to_f32(y);
  return y;
}

template <typename T, typename B, int D>
struct Scorer {  // 16-bit and E4M3 bounds
  static constexpr bool kF8 = sizeof(B) == 1;
  using M = typename std::conditional<kF8, __half, B>::type;
  static constexpr int kRow = 2 * D * static_cast<int>(sizeof(B));  // bytes of a block's bounds
  static constexpr int kWarps = kRow >= 1024 ? 4 : 8;               // that score
  static constexpr int kHalf = kRow / 2;                            // its minima or its maxima
  static constexpr int kPitch = kHalf + 16;
  static constexpr int kTiles = kRow >= 512 ? 1 : 2;                // tiles of 16 blocks in a turn
  static constexpr int kBlocks = 16 * kTiles;                       // blocks of a turn
  static constexpr int kSteps = 2 * D / 16;
  static constexpr int kFragBytes = kSteps * 8 * 4 * 8;             // [step][column][pair] two words
  static constexpr int kRing = 2 * kBlocks * kPitch;                // a warp's: minima and maxima of a turn

  int id, id_after;  // physical blocks of this lane's row (lanes 0 .. kBlocks - 1) of the turn to be copied and the next
  int copy_turn;     // the turn to be copied

  static __device__ __forceinline__ int lookup(const SelectParams& p, const int32_t* table, int cands, int turn) {
    const int lane = threadIdx.x & 31;
    return lane < kBlocks ? physical(p, table, turn * kBlocks + lane, cands, true) : 0;
  }

  // Start the copies of the turn's minima (which = 0) or maxima (1), zeros for blocks behind the last: one group of
  // copies, an empty one behind the last turn.  A warp's copy takes 512 bytes in a row: with 64 bytes of each of eight
  // rows it took 100 cycles to issue (shared-memory banks met four times).
  __device__ __forceinline__ void copy(const SelectParams& p, const int32_t* table, int h, int cands, int turns, int which,
                                       uint8_t* ring) {
    constexpr int kRows = 512 / kHalf;                      // rows of one copy
    constexpr int kLanes = 32 / kRows;                      // lanes of one row
    const int lane = threadIdx.x & 31, sub = lane / kLanes;
    if (copy_turn * kBlocks < cands) {
      const uint8_t* base = p.bounds + int64_t(h) * kRow + which * kHalf + (lane % kLanes) * 16;
      const int64_t stride = int64_t(p.num_kv_heads) * kRow;
      const uint32_t dst = smem_u32(ring) + (which * kBlocks + sub) * kPitch + (lane % kLanes) * 16;
      const int live = cands - copy_turn * kBlocks;
#pragma unroll
      for (int i = 0; i < kBlocks; i += kRows) {
        const uint8_t* src = base + __shfl_sync(kFullMask, id, i + sub) * stride;
        const uint32_t bytes = i + sub < live ? 16u : 0u;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * kPitch), "l"(src), "r"(bytes) : "memory");
      }
      if (which == 1) {
        copy_turn += turns;
        id = id_after;
        id_after = lookup(p, table, cands, copy_turn + turns);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // First copies of a scoring warp; its turns are first, first + turns, ...
  __device__ __forceinline__ void start(const SelectParams& p, const int32_t* table, int h, int cands, int first, int turns,
                                        uint8_t* ring) {
    copy_turn = first;
    id = lookup(p, table, cands, first);
    id_after = lookup(p, table, cands, first + turns);
    copy(p, table, h, cands, turns, 0, ring);
    copy(p, table, h, cands, turns, 1, ring);
  }

  // The weights' fragments: step s, column g < 3, lane c's words of k indices 2c, 2c+1 and 2c+8, 2c+9: elements 2c and
  // 2c + 8 of the step's 16 (16-bit bounds), 4c and 4c + 2 where codes are widened.  They are scaled by a power of two
  // so that the largest is near 2^14 and f16 words hold them; *unit undoes it.  Returns the sum of their magnitudes.
  static __device__ __forceinline__ float fragments(uint2* frag, const float2* w, float* unit) {
    const int lane = threadIdx.x & 31;
    float big = 0.f, sum = 0.f;
    for (int e = lane; e < 2 * D; e += 32) {
      big = fmaxf(big, fabsf(w[e].x));
      sum += fabsf(w[e].x);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      big = fmaxf(big, __shfl_xor_sync(kFullMask, big, m));
      sum += __shfl_xor_sync(kFullMask, sum, m);
    }
    // 2^(14 - e) for big in [2^(e-1), 2^e), its own exponent field read as an integer
    const int e = static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 126;
    const int k = std::is_same<M, __half>::value && big > 0.f && big < INFINITY ? min(max(14 - e, -120), 120) : 0;
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    *unit = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    uint32_t* words = reinterpret_cast<uint32_t*>(frag);
    for (int x = threadIdx.x; x < kSteps * 40; x += kSelectThreads) {  // columns 3 to 7 are zero
      const int step = x / 40, y = x - step * 40;
      words[step * 64 + 24 + y] = 0u;
    }
    for (int x = threadIdx.x; x < kSteps * 8; x += kSelectThreads) {
      const int step = x >> 3, c = (x >> 1) & 3, word = x & 1;
      const int e0 = 16 * step + (kF8 ? 4 * c + 2 * word : 2 * c + 8 * word);
      float v[2] = {w[e0].x * scale, w[e0 + 1].x * scale};
#pragma unroll
      for (int col = 0; col < 3; ++col) {
        M y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = split_word<M>(v[i], &v[i]);
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(&y[0]), hi = *reinterpret_cast<const uint16_t*>(&y[1]);
        words[step * 64 + (col * 4 + c) * 2 + word] = lo | (hi << 16);
      }
    }
    return sum;
  }

  // Half of the products of a turn's tile at shared address `at`, and the extremes of what was read: of the maxima the
  // greatest as signed, of the minima the least, which has the greatest bits.  |b| is at most the larger of the
  // greatest maximum and the least minimum's magnitude.
  template <int WHICH>
  static __device__ __forceinline__ void multiply(uint32_t at, const uint2* frag, int lane, float (&acc)[4], uint32_t (&most)[4]) {
    // four steps at a time: their chunks first, then two chains of two instructions side by side
#pragma unroll
    for (int s0 = 0; s0 < kSteps / 2; s0 += 4) {
      uint32_t af[4][4];
      uint2 bf[4];
      if constexpr (kF8) {
        uint32_t r[2][4];  // blocks 0-7 and 8-15 of a chunk, then of the next
#pragma unroll
        for (int x = 0; x < 2; ++x) ldsm_x4(at + (s0 + 2 * x) * 16, r[x]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e4m3x4_to_f16x2x2(r[i >> 1][2 * (i & 1)], af[i][0], af[i][2]);
          e4m3x4_to_f16x2x2(r[i >> 1][2 * (i & 1) + 1], af[i][1], af[i][3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) ldsm_x4(at + (s0 + i) * 32, af[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) bf[i] = frag[(WHICH * (kSteps / 2) + s0 + i) * 32 + lane];
      float part[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) mma_zero(part[x], af[2 * x], bf[2 * x], M());
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t b[2] = {bf[2 * x + 1].x, bf[2 * x + 1].y};
        Mma<M>::run(part[x], af[2 * x + 1], b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) most[k] = WHICH ? max_s16x2(most[k], af[i][k]) : max_u16x2(most[k], af[i][k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += part[0][e] + part[1][e];
    }
  }

  // Scores of a warp's turns: while the minima of one are multiplied its maxima
  // arrive, and then the next one's minima.
  __device__ __forceinline__ void run(const SelectParams& p, const uint2* frag, float unit, float wsum,
                                      const int32_t* table, int h, int cands, int first, int turns, uint8_t* ring,
                                      float* scores, ScoreStats& st) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t at = smem_u32(ring) + ((lane & 7) + (((lane >> 3) & 1) << 3)) * kPitch + (lane >> 4) * 16;
    uint32_t least[4] = {0u, 0u, 0u, 0u}, greatest[4] = {0u, 0u, 0u, 0u};
    for (int turn = first; turn * kBlocks < cands; turn += turns) {
      float acc[kTiles][4];
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();  // every lane's copies of the minima are there
#pragma unroll
      for (int t = 0; t < kTiles; ++t) multiply<0>(at + 16 * t * kPitch, frag, lane, acc[t], least);
      __syncwarp();  // every lane has read them
      // the turn that is copied next: its maxima's copies take the ids along
      copy(p, table, h, cands, turns, 0, ring);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
#pragma unroll
      for (int t = 0; t < kTiles; ++t) multiply<1>(at + (kBlocks + 16 * t) * kPitch, frag, lane, acc[t], greatest);
      __syncwarp();
      copy(p, table, h, cands, turns, 1, ring);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // columns 0 and 1 are lane c = 0's, column 2 lane c = 1's
          float x = c == 0 ? acc[t][2 * r] + acc[t][2 * r + 1] : acc[t][2 * r];
          x = (x + __shfl_xor_sync(kFullMask, x, 1)) * unit;
          const int j = turn * kBlocks + 16 * t + 8 * r + g;
          if (c == 0 && j < cands) {
            scores[j] = x;
            st.add(x);
          }
        }
    }
    least[0] = max_u16x2(max_u16x2(least[0], least[1]), max_u16x2(least[2], least[3]));
    greatest[0] = max_s16x2(max_s16x2(greatest[0], greatest[1]), max_s16x2(greatest[2], greatest[3]));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      least[0] = max_u16x2(least[0], __shfl_xor_sync(kFullMask, least[0], m));
      greatest[0] = max_s16x2(greatest[0], __shfl_xor_sync(kFullMask, greatest[0], m));
    }
    const uint16_t bits[4] = {static_cast<uint16_t>(least[0]), static_cast<uint16_t>(least[0] >> 16),
                              static_cast<uint16_t>(greatest[0]), static_cast<uint16_t>(greatest[0] >> 16)};
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(to_f32(*reinterpret_cast<const M*>(&bits[i]))));
    st.mag = most * wsum;
  }
  static __device__ __forceinline__ float chain() { return 136.f + kSteps / 2 + 8.f; }
};

template <int D>
struct Scorer<float, float, D> {  // binary32 FMA: D/16 lanes a block, 32 elements each
  static constexpr int kLanes = D / 16, kPer = 32 / kLanes, kLoads = 8, kDeep = 2;
  static constexpr int kFragBytes = 0, kRing = 0;
  static constexpr int kWarps = kSelectWarps;
  static constexpr int kBlocks = kPer * kDeep;

  static __device__ __forceinline__ float fragments(uint2*, const float2* w, float* unit) {
    float sum = 0.f;
    for (int e = threadIdx.x & 31; e < 2 * D; e += 32) sum += fabsf(w[e].x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
    *unit = 1.f;
    return sum;
  }

  int ids[kDeep];
  __device__ __forceinline__ void lookup(const SelectParams& p, const int32_t* table, int cands, int turn) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < kDeep; ++t)
      ids[t] = physical(p, table, (turn * kDeep + t) * kPer + lane / kLanes, cands, lane % kLanes == 0);
  }

  __device__ __forceinline__ void start(const SelectParams& p, const int32_t* table, int, int cands, int first, int, uint8_t*) {
    lookup(p, table, cands, first);
  }

  __device__ __forceinline__ void run(const SelectParams& p, const float2* w, float wsum, const int32_t* table, int h,
                                      int cands, int first, int turns, float* scores, ScoreStats& st) {
    const int lane = threadIdx.x & 31, gl = lane % kLanes, gi = lane / kLanes;
    float wr[32], most = 0.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) wr[4 * i + e] = w[(gl + kLanes * i) * 4 + e].x;
    for (int turn = first; turn * kBlocks < cands; turn += turns) {
      float4 x[kDeep][kLoads];
#pragma unroll
      for (int t = 0; t < kDeep; ++t)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          x[t][i] = (turn * kDeep + t) * kPer + gi < cands
                        ? reinterpret_cast<const float4*>(p.bounds)[(int64_t(ids[t]) * p.num_kv_heads + h) * (D / 2) + gl + kLanes * i]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      lookup(p, table, cands, turn + turns);
#pragma unroll
      for (int t = 0; t < kDeep; ++t) {
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const float f[4] = {x[t][i].x, x[t][i].y, x[t][i].z, x[t][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc = fmaf(wr[4 * i + e], f[e], acc);
            most = fmaxf(most, fabsf(f[e]));
          }
        }
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) acc += __shfl_xor_sync(kFullMask, acc, m);
        const int j = (turn * kDeep + t) * kPer + gi;
        if (j < cands) {
          if (gl == 0) scores[j] = acc;
          st.add(acc);
        }
      }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, m));
    st.mag = most * wsum;
  }
  static __device__ __forceinline__ float chain() { return 44.f; }
};

constexpr int kStatBytes = kMaxCluster * kSelectWarps * 16;
constexpr int kSelectMaxBlocks = 30 * 1024;

template <typename T, typename B, int D>
struct SelectSize {  // bytes of shared memory besides the scores and their two bits
  static constexpr int kAll = Scorer<T, B, D>::kWarps * Scorer<T, B, D>::kRing;
  static constexpr int kRings = kAll > static_cast<int>(sizeof(SelectShared)) ? kAll : static_cast<int>(sizeof(SelectShared));
  static constexpr int kFixed = kStatBytes + 2 * D * 8 + Scorer<T, B, D>::kFragBytes + kRings;
};

template <typename T, typename B, int D>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const SelectParams p) {
  grid_wait();
  grid_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t row = static_cast<int64_t>(blockIdx.x) / ctas;
  int b = static_cast<int>(row / p.num_kv_heads);
  const int h = static_cast<int>(row - int64_t(b) * p.num_kv_heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  using Score = Scorer<T, B, D>;
  extern __shared__ __align__(16) uint8_t raw[];
  float* stat = reinterpret_cast<float*>(raw);                    // [CTA][warp][4]: least score, greatest, magnitudes, flag
  float2* w = reinterpret_cast<float2*>(raw + kStatBytes);        // [2D]: down, up
  uint2* frag = reinterpret_cast<uint2*>(w + 2 * D);              // weights for the tensor cores
  uint8_t* rings = reinterpret_cast<uint8_t*>(frag) + Score::kFragBytes;
  SelectShared& sh = *reinterpret_cast<SelectShared*>(rings);
  static_assert(Score::kFragBytes % 16 == 0 && Score::kRing % 16 == 0 && sizeof(SelectShared) % 16 == 0, "scores are read four at a time");
  float* score = reinterpret_cast<float*>(rings + SelectSize<T, B, D>::kRings);  // [room], of the first CTA
  uint32_t* sure_bits = reinterpret_cast<uint32_t*>(score + p.room);         // [room / 32]
  uint32_t* win_bits = sure_bits + p.room / 32;
  if (p.longest_first) {  // CTAs start in launch order: the b-th longest sequence, equal ones in order
    const int mine = lane < p.num_seqs ? p.context_lens[lane] : INT_MIN;
    int before = 0;
    for (int i = 0; i < p.num_seqs; ++i) {
      const int other = __shfl_sync(kFullMask, mine, i);
      before += other > mine || (other == mine && i < lane);
    }
    b = __ffs(__ballot_sync(kFullMask, lane < p.num_seqs && before == b)) - 1;
  }
  int32_t* out = p.selected + b * p.sel_sb + h * p.sel_sh;
  int len = p.context_lens[b];
  // the first 8 heads' elements, asked for together with the length
  const T* q = static_cast<const T*>(p.q) + b * p.q_sb + int64_t(h) * p.group * p.q_sh;
  T q8[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) q8[g] = tid < D && g < p.group ? q[g * p.q_sh + tid] : from_f32<T>(0.f);
  if (len < 0 || len > p.max_tokens) {
    if (tid == 0 && rank == 0) atomicOr(p.err, kErrLen);
    len = len < 0 ? 0 : p.max_tokens;
  }
  const int n = (len + (1 << p.log2_bs) - 1) >> p.log2_bs;
  const int need = p.top - p.sink - p.recent;  // of the scored blocks
  if (n <= p.top || need == 0) {               // all of them, or the fixed ones alone: no scores
    for (int i = rank * kSelectThreads + tid; i < p.top; i += ctas * kSelectThreads) {
      if (n <= p.top)
        out[i] = i < n ? i : -1;
      else
        out[i] = i < p.sink ? i : n - p.top + i;
    }
    return;
  }
  auto started = cluster.barrier_arrive();  // waited for before the first store to the first CTA's shared memory

  // --- scores of the candidates sink .. n - recent - 1 ---
  const int cands = n - p.sink - p.recent;
  const int32_t* table = p.block_tables + b * p.bt_stride + p.sink;
  constexpr int64_t head_bytes = 2 * D * sizeof(B);
  const int first = rank * Score::kWarps + warp, turns = ctas * Score::kWarps;
  const bool scores_here = warp < Score::kWarps;
  uint8_t* ring = rings + warp * Score::kRing;
  Score scorer;
  if (scores_here) scorer.start(p, table, h, cands, first, turns, ring);

  // the weights, sums over the group's heads in two binary32 words each (the
  // rounding error of every addition is kept in the second)
  auto sums = [&](float unit) {
    bool big = false;
    static_assert(D <= kSelectThreads, "an element a thread");
    if (tid < D) {
      const int d = tid;
      float hi[2] = {0.f, 0.f}, lo[2] = {0.f, 0.f};
      for (int g0 = 0; g0 < p.group; g0 += 8) {
        float x[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) x[g] = g0 == 0 ? to_f32(q8[g]) * unit : g0 + g < p.group ? to_f32(q[(g0 + g) * p.q_sh + d]) * unit : 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          big |= fabsf(x[g]) > 1e30f && fabsf(x[g]) < INFINITY;
          const float part[2] = {x[g] > 0.f ? 0.f : x[g], x[g] < 0.f ? 0.f : x[g]};  // a NaN goes into both
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float s = __fadd_rn(hi[i], part[i]), z = __fsub_rn(s, hi[i]);
            lo[i] = __fadd_rn(lo[i], __fadd_rn(__fsub_rn(hi[i], __fsub_rn(s, z)), __fsub_rn(part[i], z)));
            hi[i] = s;
          }
        }
      }
      // an infinite sum leaves NaN behind as its error: the sum alone counts
      w[d] = make_float2(hi[0], fabsf(hi[0]) < INFINITY ? lo[0] : 0.f);
      w[D + d] = make_float2(hi[1], fabsf(hi[1]) < INFINITY ? lo[1] : 0.f);
    }
    return __syncthreads_or(big);
  };
  // sums that could leave binary32's range are taken of the queries times 2^-60
  if (sums(1.f)) sums(8.6736174e-19f);

  float unit;
  const float wsum = Score::fragments(frag, w, &unit);
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  ScoreStats st;
  if (scores_here) {
    float* scores = cluster.map_shared_rank(score, 0);
    if constexpr (sizeof(B) == 4) {
      scorer.run(p, w, wsum, table, h, cands, first, turns, scores, st);
    } else {
      scorer.run(p, frag, unit, wsum, table, h, cands, first, turns, ring, scores, st);
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    st.least = fminf(st.least, __shfl_xor_sync(kFullMask, st.least, m));
    st.greatest = fmaxf(st.greatest, __shfl_xor_sync(kFullMask, st.greatest, m));
  }
  st.odd = __any_sync(kFullMask, st.odd || !(st.mag < 1e37f));
  if (lane == 0)
    *reinterpret_cast<float4*>(cluster.map_shared_rank(stat + (rank * kSelectWarps + warp) * 4, 0)) =
        make_float4(st.least, st.greatest, st.mag, st.odd ? 1.f : 0.f);
  cluster.sync();
  if (rank != 0) return;  // nothing of this CTA is accessed any more
  for (int i = tid; i < kBins; i += kSelectThreads) sh.hist[i] = 0;
  if (tid == 0) sh.near_count = sh.win_count = sh.sure_count = 0;
  __syncthreads();

  // --- the first CTA: the bin that holds the border ---
  float smin = INFINITY, smax = -INFINITY, mag = 0.f, flag = 0.f;
  for (int r = lane; r < ctas * kSelectWarps; r += 32) {
    smin = fminf(smin, stat[4 * r]), smax = fmaxf(smax, stat[4 * r + 1]);
    mag = fmaxf(mag, stat[4 * r + 2]), flag = fmaxf(flag, stat[4 * r + 3]);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    smin = fminf(smin, __shfl_xor_sync(kFullMask, smin, m)), smax = fmaxf(smax, __shfl_xor_sync(kFullMask, smax, m));
    mag = fmaxf(mag, __shfl_xor_sync(kFullMask, mag, m)), flag = fmaxf(flag, __shfl_xor_sync(kFullMask, flag, m));
  }
  // two errors of a score; 1e-37 covers products below the smallest binary32 number
  const float err2 = 2.f * ((static_cast<float>(p.group) + Score::chain()) * 5.9604645e-8f * 1.01f * mag + 1e-37f);
  // scores that overflowed, infinite or NaN bounds: every candidate is settled in binary64
  const bool all = flag != 0.f;
  const int words = (cands + 31) / 32, quads = (cands + 3) / 4;
  for (int i = tid; i < words; i += kSelectThreads) sure_bits[i] = win_bits[i] = 0u;
  float above = INFINITY, below = -INFINITY;  // scores over `above` are in, scores under `below` are not
  if (!all) {
    const float per = smax > smin ? static_cast<float>(kBins) / (smax - smin) : 0.f;
#pragma unroll 4
    for (int i = tid; i < quads; i += kSelectThreads) {
      const float4 s = reinterpret_cast<const float4*>(score)[i];
      const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * i + e < cands)
          atomicAdd(&sh.hist[static_cast<int>(fminf(fmaxf((v[e] - smin) * per, 0.f), kBins - 1.f))], 1u);
    }
    __syncthreads();
    constexpr int kMine = kBins / kSelectThreads;
    uint32_t c[kMine], sum = 0, total;
    const int at = kBins - kMine * (tid + 1);  // thread 0 holds the highest bins
#pragma unroll
    for (int i = 0; i < kMine; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&sh.hist[at + kMine - 4 - i]);
      c[i] = x.w, c[i + 1] = x.z, c[i + 2] = x.y, c[i + 3] = x.x;
      sum += x.x + x.y + x.z + x.w;
    }
    uint32_t before = block_scan(sh, sum, &total);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (before < static_cast<uint32_t>(need) && before + c[i] >= static_cast<uint32_t>(need))
        sh.found_bin = at + kMine - 1 - i;
      before += c[i];
    }
    __syncthreads();
    // The border score is in the found bin; its edges, with the roundings of the
    // bin's number (a few 2^-24 of the extremes), moved out by two errors.
    if (per > 0.f && per < INFINITY) {
      const float slack = err2 + 16.f * 5.9604645e-8f * (fabsf(smin) + fabsf(smax));
      above = smin + static_cast<float>(sh.found_bin + 1) / per + slack;
      below = smin + static_cast<float>(sh.found_bin) / per - slack;
    }
  } else {
    __syncthreads();
  }

  // --- blocks above the border for certain, and those to be settled ---
#pragma unroll 4
  for (int i = tid; i < quads; i += kSelectThreads) {
    const float4 s = reinterpret_cast<const float4*>(score)[i];
    const float v[4] = {s.x, s.y, s.z, s.w};
    uint32_t in = 0, open = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool here = 4 * i + e < cands, over = !all && v[e] > above;
      in |= here && over ? 1u << e : 0u;
      open |= here && !over && (all || v[e] >= below) ? 1u << e : 0u;
    }
    const int shift = (4 * i) & 31;
    if (in) {
      atomicOr(&sure_bits[i >> 3], in << shift);
      atomicAdd(&sh.sure_count, __popc(in));
    }
    if (open) {
      atomicOr(&win_bits[i >> 3], open << shift);
      int at = atomicAdd(&sh.near_count, __popc(open));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((open >> e) & 1u) {
          if (at < kWindow) {
            sh.near_at[at] = 4 * i + e;
            sh.near_score[at] = v[e];
          }
          ++at;
        }
    }
  }
  __syncthreads();
  int window = sh.near_count;
  int left = need - sh.sure_count;  // of the near blocks: 1 .. window
  if (!all && window <= kWindow && window > left) {
    // the border is the left-th of them; what is more than two errors above it is in
    for (int i = tid; i < window; i += kSelectThreads) {
      const float s = sh.near_score[i];
      const int at = sh.near_at[i];
      int better = 0;
      for (int o = 0; o < window; ++o) better += sh.near_score[o] > s || (sh.near_score[o] == s && sh.near_at[o] < at);
      if (better == left - 1) sh.border = s;
    }
    __syncthreads();
    const float border = sh.border;
    for (int i = tid; i < window; i += kSelectThreads) {
      const float s = sh.near_score[i];
      const int at = sh.near_at[i];
      const bool in = s - border > err2;
      if (in || border - s > err2) {
        atomicAnd(&win_bits[at >> 5], ~(1u << (at & 31)));
        if (in) {
          atomicOr(&sure_bits[at >> 5], 1u << (at & 31));
          atomicAdd(&sh.sure_count, 1);
        }
      } else {
        sh.win_at[atomicAdd(&sh.win_count, 1)] = at;
      }
    }
    __syncthreads();
    window = sh.win_count;
    left = need - sh.sure_count;
  } else if (window <= kWindow) {
    for (int i = tid; i < window; i += kSelectThreads) sh.win_at[i] = sh.near_at[i];
    __syncthreads();
  }
  auto bounds_of = [&](int j) {
    int id = table[j];
    if (id < 0 || id >= p.num_blocks) id = 0;
    return p.bounds + (int64_t(id) * p.num_kv_heads + h) * head_bytes;
  };
  if (window == left) {  // all of them
    for (int i = tid; i < words; i += kSelectThreads) sure_bits[i] |= win_bits[i];
  } else if (window <= kWindow) {
    // from scores within 2^-35 of the magnitudes; where that leaves the border
    // open (or blocks alike), in binary64
    const double apart = 5.8207661e-11 * static_cast<double>(mag) + 1e-37;
    for (int exact = all ? 1 : 0; exact < 2; ++exact) {
      if (tid == 0) sh.found_above = 0;
      for (int i = tid; i < words; i += kSelectThreads) win_bits[i] = 0u;  // the list holds them; now those that are kept
      for (int i0 = warp * 4; i0 < window; i0 += kSelectWarps * 4) {
        const int i = min(i0 + (lane >> 3), window - 1);
        const double s = exact ? fine_score<B, D, true>(bounds_of(sh.win_at[i]), w, lane)
                               : fine_score<B, D, false>(bounds_of(sh.win_at[i]), w, lane);
        if ((lane & 7) == 0) sh.win_score[i] = s;
      }
      __syncthreads();
      for (int i = tid; i < window; i += kSelectThreads) {
        const double s = sh.win_score[i];
        const int at = sh.win_at[i];
        int better = 0, near = 0;
        for (int o = 0; o < window; ++o) {
          better += sh.win_score[o] > s || (sh.win_score[o] == s && sh.win_at[o] < at);
          near += sh.win_score[o] - s < apart && s - sh.win_score[o] < apart;
        }
        // the last that is kept and the first that is not may not be told apart by this
        if (better < left) atomicOr(&win_bits[at >> 5], 1u << (at & 31));
        if (!exact && (better == left - 1 || better == left) && near > 1) sh.found_above = 1;
      }
      __syncthreads();
      if (exact || sh.found_above == 0) break;
      __syncthreads();
    }
    for (int i = tid; i < words; i += kSelectThreads) sure_bits[i] |= win_bits[i];
  } else {
    // many alike: the high words of the exact scores, then the low words of those
    // that share the border's high word, then the index; the keys take the scores' place
    uint32_t* key = reinterpret_cast<uint32_t*>(score);
    for (int half = 0; half < 2; ++half) {
      for (int i = warp; i < words; i += kSelectWarps) {
        const uint32_t m = win_bits[i];
        for (int k0 = 0; k0 < 32; k0 += 4) {
          if (!((m >> k0) & 15u)) continue;
          const int j = min(i * 32 + k0 + (lane >> 3), cands - 1);
          const unsigned long long k = ordered(fine_score<B, D, true>(bounds_of(j), w, lane));
          if ((lane & 7) == 0 && i * 32 + k0 + (lane >> 3) == j) key[j] = static_cast<uint32_t>(half ? k : k >> 32);
        }
      }
      __syncthreads();
      const uint32_t want = digit_cut(sh, key, win_bits, words, &left);
      for (int i = warp; i < words; i += kSelectWarps) {
        const bool in = (win_bits[i] >> lane) & 1u;
        const uint32_t above = __ballot_sync(kFullMask, in && key[i * 32 + lane] > want);
        const uint32_t equal = __ballot_sync(kFullMask, in && key[i * 32 + lane] == want);
        if (lane == 0) {
          sure_bits[i] |= above;
          win_bits[i] = equal;
        }
      }
      __syncthreads();
    }
    // the first `left` of the equal ones
    int taken = 0;
    for (int i0 = 0; i0 < words; i0 += kSelectThreads) {
      const uint32_t m = i0 + tid < words ? win_bits[i0 + tid] : 0u;
      uint32_t total;
      int room = left - taken - static_cast<int>(block_scan(sh, __popc(m), &total));
      uint32_t keep = 0;
      for (uint32_t x = m; x && room > 0; x &= x - 1, --room) keep |= x & (~x + 1u);
      if (keep) sure_bits[i0 + tid] |= keep;
      taken += static_cast<int>(total);
    }
  }
  __syncthreads();

  // --- the chosen blocks, ascending ---
  int base = p.sink;
  for (int i0 = 0; i0 < words; i0 += kSelectThreads) {
    uint32_t m = i0 + tid < words ? sure_bits[i0 + tid] : 0u, total;
    int at = base + static_cast<int>(block_scan(sh, __popc(m), &total));
    for (; m; m &= m - 1, ++at)
      if (at < p.top) out[at] = p.sink + (i0 + tid) * 32 + __ffs(m) - 1;
    base += static_cast<int>(total);
  }
  for (int i = tid; i < p.sink + p.recent; i += kSelectThreads) {
    if (i < p.sink)
      out[i] = i;
    else
      out[p.top - p.recent + (i - p.sink)] = n - p.recent + (i - p.sink);
  }
}

size_t select_smem(int fixed, int room) {  // scores and two bits a block behind what the kernel always has
  return size_t(fixed) + size_t(room) * 4 + size_t(room / 32) * 8;
}

template <typename T, typename B, int D>
int launch_one(SelectParams p, int max_blocks, int num_sms, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  static_assert(SelectSize<T, B, D>::kFixed + kSelectMaxBlocks * 4 + kSelectMaxBlocks / 4 <= 226 * 1024, "scores of the widest table fit");
  p.room = (max_blocks + 31) / 32 * 32;
  const size_t smem = select_smem(SelectSize<T, B, D>::kFixed, p.room);
  // CTAs of a row: as many as run at once, so that the work of every CTA besides
  // the scores (weights, barrier, the first copies' latency) is paid once, and
  // none with less than a turn of its warps.  Measured, us for 1, 2, 4 and 8 CTAs
  // a row: 64 rows of up to 8192 blocks 94.7, 58.9, 46.4 and 46.7; 256 of up to
  // 1500 26.9, 32.5, 41.0 and 62.0; 4 of 1000 11.6, 9.2, 8.0 and 8.2.
  const int64_t rows = int64_t(p.num_seqs) * p.num_kv_heads;
  const int64_t resident = int64_t(num_sms) * std::max<int64_t>(1, std::min<int64_t>(2, 227 * 1024 / (smem + 1024)));
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas * 2 <= resident && max_blocks / (2 * ctas) >= Scorer<T, B, D>::kBlocks * Scorer<T, B, D>::kWarps / 2)
    ctas *= 2;
  // batches of more than one wave start the longest rows first
  p.longest_first = rows * ctas > resident && p.num_seqs > 1 && p.num_seqs <= 32;
  const void* func = reinterpret_cast<const void*>(&select_kernel<T, B, D>);
  int e = raise_smem_limit(configured, func, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_dependent(&select_kernel<T, B, D>, dim3(static_cast<unsigned>(int64_t(p.num_seqs) * p.num_kv_heads * ctas)),
                          dim3(kSelectThreads), smem, ctas, stream, p);
}

template <typename T, typename B>
int launch_dim(const SelectParams& p, int head_dim, int max_blocks, int num_sms, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_one<T, B, 64>(p, max_blocks, num_sms, stream);
    case 128: return launch_one<T, B, 128>(p, max_blocks, num_sms, stream);
    case 256: return launch_one<T, B, 256>(p, max_blocks, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Most blocks a table row may have: their scores have to fit one CTA's shared
// memory beside the rings (85 KB with everything else).
int select_max_blocks() { return kSelectMaxBlocks; }

int launch_select(int dtype, int bounds_dtype, int head_dim, const SelectParams& p, int max_blocks, int num_sms,
                  cudaStream_t stream) {
  int e = cudaErrorInvalidValue;
  if (dtype == 0 && bounds_dtype == 0) e = launch_dim<float, float>(p, head_dim, max_blocks, num_sms, stream);
  if (dtype == 1 && bounds_dtype == 1) e = launch_dim<__half, __half>(p, head_dim, max_blocks, num_sms, stream);
  if (dtype == 2 && bounds_dtype == 2) e = launch_dim<__nv_bfloat16, __nv_bfloat16>(p, head_dim, max_blocks, num_sms, stream);
  if (dtype == 1 && bounds_dtype == 5) e = launch_dim<__half, uint8_t>(p, head_dim, max_blocks, num_sms, stream);
  if (dtype == 2 && bounds_dtype == 5) e = launch_dim<__nv_bfloat16, uint8_t>(p, head_dim, max_blocks, num_sms, stream);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
