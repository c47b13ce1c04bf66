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
// divided out, so bf16 rows of any size do.  Weights are rounded to f16 times 2^14
// (normal numbers down to 2^-28 of the largest): 2^-11 relative each, which is
// averaged over the tokens and stays below the output's own rounding.
//
// Work split: all units, ordered by sequence, kv head and head tile, are cut into
// as many equal runs as CTAs fit the GPU, so that rows of any length fill it
// evenly; a CTA's warps take its units in turn.  At the end of a row the warps'
// results meet in the stages they have just left, while the next row's copies go
// on.  A row that several CTAs share is written as partial results (two at most a
// CTA: the row it begins in and the row it ends in), and the CTA that counts in
// last merges them in their order: nobody waits, and the result does not depend
// on who was last.
#include <atomic>

#include "decode_kernel.cuh"
#include "launch.h"
#include "mma_e4m3.cuh"
#include "wllm.h"

namespace wllm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kWeightShift = 14.f;
constexpr int kMostCtas = 4;      // of an SM
constexpr int kLeastUnits = 2;    // of a warp, before another CTA takes part

template <int D, int NT>
struct Shape {
  using G = Geom<uint8_t, D>;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kSub = D == 256 ? 1 : 2;          // 16-token tiles of a unit
  static constexpr int kUnit = 16 * kSub;                // its tokens
  static constexpr int kOctets = 2 * kSub;               // runs of 8 tokens, each of one block
  static constexpr int kSide = kSub * G::kTileBytes;     // a unit's K (or V)
  static constexpr int kStage = 2 * kSide;
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kRing = kStages * kStage;         // a warp's
  static constexpr int kScales = 8;                      // of a stage: K's octets at 0, V's at 4
  static constexpr int kSmem = 1024 + kWarps * kRing;
  static constexpr int kPart = kHeads * D + 2 * kHeads;  // floats of a partial result: outputs, maxima, sums
  static_assert(kHeads * D * 4 <= kStage, "a warp's outputs take a stage's place");
};

__device__ __forceinline__ void copy4_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
// One of the barrier's arrivals, once this thread's asynchronous copies have landed.
__device__ __forceinline__ void arrive_behind_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float scale_in_range(float s) {
  constexpr float kLeast = 1.f / (1ull << -kLeastScaleExp), kMost = static_cast<float>(1ull << kMostScaleExp);
  return fminf(fmaxf(s, kLeast), kMost);  // a NaN counts as the least
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int length_of(const ScaledDecodeParams& p, int b) {
  return min(max(p.context_lens[b], 0), p.max_tokens);
}

// A CTA's run of units as segments: the units of one row (sequence, kv head, head
// tile) that are in it.  The same in every lane.
template <int UNIT>
struct Segments {
  long long remaining;  // units of the run from this segment on
  int b, row, rows;     // sequence; row of it, of how many
  int len, units;       // the sequence's
  int at, count;        // the segment: units at .. at + count - 1 of the row
  int turn;             // the run's units before it, modulo the warps
  int window, lens;     // lengths of sequences window .. window + 31, a lane each

  __device__ __forceinline__ int length(const ScaledDecodeParams& p, int i) {
    if ((i & ~31) != window) {
      window = i & ~31;
      const int mine = window + (threadIdx.x & 31);
      lens = mine < p.num_seqs ? length_of(p, mine) : 0;
    }
    return __shfl_sync(kFullMask, lens, i & 31);
  }
  __device__ __forceinline__ void start(const ScaledDecodeParams& p, int first, long long offset, long long run, int rows_) {
    window = -1, rows = rows_, b = first, turn = 0, remaining = run;
    len = length(p, b);
    units = (len + UNIT - 1) / UNIT;
    row = static_cast<int>(offset / units);
    at = static_cast<int>(offset - static_cast<long long>(row) * units);
    count = static_cast<int>(min(static_cast<long long>(units - at), remaining));
  }
  __device__ __forceinline__ bool next(const ScaledDecodeParams& p) {
    remaining -= count;
    turn = (turn + count) & (kWarps - 1);
    if (remaining <= 0) return false;
    at = 0;
    if (++row == rows) {
      row = 0;
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

  // Heads 0 .. heads-1 from `src` on, rows `sh` elements apart.
  template <typename T>
  __device__ __forceinline__ void load_q(const T* src, int64_t sh, int heads, bool pairs, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool valid = 8 * nt + g < heads;
      const T* at = src + (valid ? 8 * nt + g : 0) * sh;
      uint32_t raw[kKS][2], most = 0u;
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const T* d = at + 16 * s + 4 * c + 2 * e;
          uint32_t x;
          if (pairs) {
            x = *reinterpret_cast<const uint32_t*>(d);
          } else {
            x = *reinterpret_cast<const uint16_t*>(d) | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(d + 1)) << 16;
          }
          raw[s][e] = valid ? x : 0u;
          most = max(most, max(raw[s][e] & 0x7fffu, (raw[s][e] >> 16) & 0x7fffu));  // magnitudes' order is their bits'
        }
      most = max(most, __shfl_xor_sync(kFullMask, most, 1));
      most = max(most, __shfl_xor_sync(kFullMask, most, 2));
      // largest magnitude to 2^14 .. 2^15; exponent fields of binary32
      const uint16_t top_bits = static_cast<uint16_t>(most);
      const float top = to_f32(*reinterpret_cast<const T*>(&top_bits));
      const int field = min(max(127 + 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
      const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * scale_log2;
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const T* x = reinterpret_cast<const T*>(&raw[s][e]);
          q[nt][s][e] = Mma<__half>::pack(to_f32(x[0]) * up, to_f32(x[1]) * up);
        }
      factor[nt][0] = __shfl_sync(kFullMask, down, 8 * c);
      factor[nt][1] = __shfl_sync(kFullMask, down, 8 * c + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = -INFINITY, l[nt][i] = 0.f;
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
      inv[i] = __frcp_rn(vs);
    }
    uint32_t w[S::kSub][NT][2];
    float alpha[NT][2];
    bool moved = false;
    const bool full = live >= S::kUnit;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < S::kSub; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 2 * j + (e >> 1);
          const float x = fmaf(s[j][nt][e], factor[nt][e & 1] * ks[i], add[i]);
          s[j][nt][e] = full || 8 * i + g < live ? x : -INFINITY;
          top[e & 1] = fmaxf(top[e & 1], s[j][nt][e]);
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(kFullMask, top[i], off));
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[nt][i], top[i]);
        alpha[nt][i] = m[nt][i] == -INFINITY ? 0.f : exp2f(m[nt][i] - mn);
        moved |= mn > m[nt][i];
        m[nt][i] = mn;
        base[i] = (mn == -INFINITY ? 0.f : mn) - kWeightShift;
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
        w[j][nt][0] = movmatrix_trans(Mma<__half>::pack(e[0], e[1]));
        w[j][nt][1] = movmatrix_trans(Mma<__half>::pack(e[2], e[3]));
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
          for (int nt = 0; nt < NT; ++nt) Mma<__half>::run(o[2 * mp + half][nt], a, w[j][nt]);
        }
      }
    }
  }

  // Outputs [heads][D] to `at`, maxima and sums to `ms` and `ls`.
  __device__ __forceinline__ void store(float* at, float* ms, float* ls) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[nt][i];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(kFullMask, x, off);
        if (g == 0) ms[8 * nt + 2 * c + i] = m[nt][i], ls[8 * nt + 2 * c + i] = x;
      }
#pragma unroll
      for (int t = 0; t < kKS; ++t) {  // rows g and g + 8 are elements 16t + 2g and 16t + 2g + 1
        const int d = 16 * t + 2 * g;
        *reinterpret_cast<float2*>(at + (8 * nt + 2 * c) * D + d) = make_float2(o[t][nt][0], o[t][nt][2]);
        *reinterpret_cast<float2*>(at + (8 * nt + 2 * c + 1) * D + d) = make_float2(o[t][nt][1], o[t][nt][3]);
      }
    }
  }
};

// Four outputs of a row.
__device__ __forceinline__ void store_out(const ScaledDecodeParams& p, int64_t at, float4 v) {
  uint32_t lo, hi;
  if (p.bf16) {
    lo = Mma<__nv_bfloat16>::pack(v.x, v.y), hi = Mma<__nv_bfloat16>::pack(v.z, v.w);
  } else {
    lo = Mma<__half>::pack(v.x, v.y), hi = Mma<__half>::pack(v.z, v.w);
  }
  uint16_t* out = static_cast<uint16_t*>(p.out) + at;
  if (p.o_pairs) {
    reinterpret_cast<uint32_t*>(out)[0] = lo, reinterpret_cast<uint32_t*>(out)[1] = hi;
  } else {
    out[0] = static_cast<uint16_t>(lo), out[1] = static_cast<uint16_t>(lo >> 16);
    out[2] = static_cast<uint16_t>(hi), out[3] = static_cast<uint16_t>(hi >> 16);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads)
    decode_block_scaled_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                               const ScaledDecodeParams p) {
  using S = Shape<D, NT>;
  using G = typename S::G;
  extern __shared__ __align__(16) uint8_t unaligned[];
  __shared__ uint64_t bars[kWarps][S::kStages];
  __shared__ float scales[kWarps][S::kStages][S::kScales];
  __shared__ float part_m[kWarps][S::kHeads], part_l[kWarps][S::kHeads];
  __shared__ int part_stage[kWarps];
  __shared__ long long sums[kWarps], first_offset;
  __shared__ int first_seq, last_in;
  uint8_t* raw = unaligned + ((1024 - (smem_u32(unaligned) & 1023)) & 1023);  // swizzled boxes start at 1024 bytes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = raw + warp * S::kRing;
  // a stage: the expected bytes of its copies, and eight lanes' copies of scales
  if (lane < S::kStages) mbar_init(smem_u32(&bars[warp][lane]), 1 + S::kScales);
  fence_mbar_init();
  if (lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
  __syncwarp();
  grid_wait();
  grid_launch_dependents();

  // --- this CTA's run of units
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
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sums[w];
    total += sums[w];
  }
  total *= rows;
  const long long ctas = max(1ll, min(static_cast<long long>(gridDim.x), total / (kWarps * kLeastUnits)));
  const long long c = blockIdx.x;
  const long long u0 = c < ctas ? total * c / ctas : total, u1 = c < ctas ? total * (c + 1) / ctas : total;
  if (u0 < u1 && (upto - mine) * rows <= u0 && u0 < upto * rows) {
    long long before = upto - mine;
    for (int b = s0; b < s1; ++b) {
      const int units = (length_of(p, b) + S::kUnit - 1) / S::kUnit;
      if (u0 < (before + units) * rows) {
        first_seq = b, first_offset = u0 - before * rows;
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
      for (int x = lane; x < p.num_q_heads * (D / 4); x += 32)
        store_out(p, seq * p.o_sb + (x / (D / 4)) * p.o_sh + (x % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  __syncthreads();
  if (u0 >= u1) return;

  // --- copies: a cursor of its own runs ahead; the next unit's table entries are asked for one unit early
  Segments<S::kUnit> ahead, seg;
  seg.start(p, first_seq, first_offset, u1 - u0, rows);
  ahead = seg;
  int ahead_at = ahead.first_of(warp), entry = 0, next_t = 0, next_len = 0, next_h = 0;
  bool more = true;
  const bool two = p.log2_bs < 4;  // 8-token blocks: two 8-row boxes for 16 tokens
  const int bs_mask = (1 << p.log2_bs) - 1;
  auto look_up = [&] {  // the cursor's unit, which becomes the next to be copied
    while (more && ahead_at >= ahead.count) {
      more = ahead.next(p);
      ahead_at = ahead.first_of(warp);
    }
    if (!more) return;
    next_t = (ahead.at + ahead_at) * S::kUnit, next_len = ahead.len, next_h = ahead.row / p.head_tiles;
    const int t = next_t + 8 * lane;
    if (lane < S::kOctets && t < next_len) entry = p.block_tables[ahead.b * p.bt_stride + (t >> p.log2_bs)];
    ahead_at += kWarps;
  };
  auto refill = [&](int stage) {
    if (!more) return;
    if (lane < S::kOctets && next_t + 8 * lane < next_len && (entry < 0 || entry >= p.num_blocks)) {
      atomicOr(p.err, kErrBlock);
      entry = 0;
    }
    const uint32_t bar = smem_u32(&bars[warp][stage]), dst = smem_u32(ring + stage * S::kStage);
    // one box a lane: K or V, column box, 16 tokens (or 8)
    const int x = two ? lane >> 1 : lane, octet_in = two ? lane & 1 : 0;
    const int kv = x & 1, col = (x >> 1) % G::kColBoxes, tile = (x >> 1) / G::kColBoxes;
    const int octet = 2 * tile + octet_in, t = next_t + 8 * octet;
    const int phys = __shfl_sync(kFullMask, entry, octet & (S::kOctets - 1));
    const bool box = tile < S::kSub && t < next_len;
    const uint32_t box_bytes = 128u * (G::kPairRows || two ? 8u : 16u);
    const uint32_t bytes = box_bytes * __popc(__ballot_sync(kFullMask, box));
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    if (box) {
      const int at = (next_h << p.log2_bs) + (t & bs_mask);
      tma_load_3d(dst + kv * S::kSide + tile * G::kTileBytes + col * 2048 + octet_in * 1024, kv ? &vmap : &kmap, bar, col * 128,
                  G::kPairRows ? at >> 1 : at, phys);
    }
    const int of = __shfl_sync(kFullMask, entry, lane & 3 & (S::kOctets - 1));
    if (lane < S::kScales) {
      const int i = lane & 3;
      if (i < S::kOctets && next_t + 8 * i < next_len)
        copy4_async(smem_u32(&scales[warp][stage][lane]), (lane < 4 ? p.k_scales : p.v_scales) + int64_t(of) * p.num_kv_heads + next_h);
      arrive_behind_copies(bar);
    }
    look_up();
  };
  look_up();
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) refill(s);

  int stage = 0;
  uint32_t phase = 0u;  // of every stage, turned when the ring comes round
  bool lost = false;
  Math<D, NT> math;
  while (true) {
    const int h = seg.row / p.head_tiles, tile = seg.row - h * p.head_tiles;
    const int heads = min(S::kHeads, p.group - tile * S::kHeads);
    const int head0 = h * p.group + tile * S::kHeads;
    const int64_t q_at = seg.b * p.q_sb + head0 * p.q_sh;
    if (p.bf16) math.load_q(static_cast<const __nv_bfloat16*>(p.q) + q_at, p.q_sh, heads, p.q_pairs, p.scale_log2);
    else math.load_q(static_cast<const __half*>(p.q) + q_at, p.q_sh, heads, p.q_pairs, p.scale_log2);

    int left = -1;  // the stage that this warp's last unit of the segment leaves
    for (int i = seg.first_of(warp); i < seg.count && !lost; i += kWarps) {
      if (!mbar_wait_warp(smem_u32(&bars[warp][stage]), phase, p.wait_limit_ns)) {
        // give up: record it, let what is in flight land (again with a limit), and take no more units
        if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
        for (int s = 0; s < S::kStages; ++s) mbar_wait_bounded(smem_u32(&bars[warp][s]), s >= stage ? phase : phase ^ 1u, p.wait_limit_ns);
        lost = true;
        break;
      }
      math.step(smem_u32(ring + stage * S::kStage), scales[warp][stage], seg.len - (seg.at + i) * S::kUnit);
      __syncwarp();  // every lane has read the stage
      if (i + kWarps < seg.count) refill(stage); else left = stage;
      if (++stage == S::kStages) stage = 0, phase ^= 1u;
    }

    // --- the segment's end: the warps' results meet
    if (left >= 0) math.store(reinterpret_cast<float*>(ring + left * S::kStage), part_m[warp], part_l[warp]);
    if (lane == 0) part_stage[warp] = lost ? -1 : left;
    fence_async_smem();  // the stage is written by copies again
    __syncthreads();
    const bool whole = seg.count == seg.units;
    long long row_first = 0, cta_first = 0;  // of a shared row: its first unit, the first CTA that has one
    int sharers = 1;
    float* to = nullptr;
    if (!whole) {
      row_first = u1 - seg.remaining - seg.at;
      cta_first = ((row_first + 1) * ctas - 1) / total;
      sharers = static_cast<int>(((row_first + seg.units) * ctas - 1) / total - cta_first) + 1;
      to = p.parts + (2 * c + (c == cta_first ? 1 : 0)) * S::kPart;
    }
    for (int i = tid; i < S::kHeads * (D / 4); i += kThreads) {
      const int a = i / (D / 4), d = (i - a * (D / 4)) * 4;
      float top = -INFINITY, f[kWarps], sum = 0.f;
      int at[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        at[w] = part_stage[w];
        if (at[w] >= 0) top = fmaxf(top, part_m[w][a]);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (at[w] < 0) continue;
        f[w] = part_m[w][a] == -INFINITY ? 0.f : exp2f(part_m[w][a] - top);
        sum = fmaf(f[w], part_l[w][a], sum);
        const float4 x = *reinterpret_cast<const float4*>(raw + w * S::kRing + at[w] * S::kStage + (a * D + d) * 4);
        v.x = fmaf(f[w], x.x, v.x), v.y = fmaf(f[w], x.y, v.y), v.z = fmaf(f[w], x.z, v.z), v.w = fmaf(f[w], x.w, v.w);
      }
      if (whole) {
        if (a < heads) {
          const float by = 1.f / sum;
          store_out(p, seg.b * p.o_sb + (head0 + a) * p.o_sh + d, make_float4(v.x * by, v.y * by, v.z * by, v.w * by));
        }
      } else {
        *reinterpret_cast<float4*>(to + a * D + d) = v;
        if (d == 0) to[S::kHeads * D + a] = top, to[S::kHeads * D + S::kHeads + a] = sum;
      }
    }
    fence_async_smem();
    __syncthreads();
    if (!whole) {
      if (tid == 0) {
        __threadfence();
        const int before = atomicAdd(p.counters + cta_first, 1);
        last_in = before == sharers - 1;
        if (last_in) p.counters[cta_first] = 0;
        __threadfence();
      }
      __syncthreads();
      if (last_in) {
        // the row's partial results in their order, eight at a time
        for (int i = tid; i < heads * (D / 4); i += kThreads) {
          const int a = i / (D / 4), d = (i - a * (D / 4)) * 4;
          float top = -INFINITY, sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s0 = 0; s0 < sharers; s0 += 8) {
            float ms[8], ls[8];
            float4 x[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              if (s0 + s >= sharers) continue;
              const float* from = p.parts + (2 * (cta_first + s0 + s) + (s0 + s == 0 ? 1 : 0)) * S::kPart;
              ms[s] = __ldcg(from + S::kHeads * D + a);
              ls[s] = __ldcg(from + S::kHeads * D + S::kHeads + a);
              x[s] = __ldcg(reinterpret_cast<const float4*>(from + a * D + d));
            }
            float higher = top;
#pragma unroll
            for (int s = 0; s < 8; ++s)
              if (s0 + s < sharers) higher = fmaxf(higher, ms[s]);
            const float f0 = top == -INFINITY ? 0.f : exp2f(top - higher);
            top = higher;
            sum *= f0, v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              if (s0 + s >= sharers) continue;
              const float f = ms[s] == -INFINITY ? 0.f : exp2f(ms[s] - top);
              sum = fmaf(f, ls[s], sum);
              v.x = fmaf(f, x[s].x, v.x), v.y = fmaf(f, x[s].y, v.y), v.z = fmaf(f, x[s].z, v.z), v.w = fmaf(f, x[s].w, v.w);
            }
          }
          const float by = 1.f / sum;
          store_out(p, seg.b * p.o_sb + (head0 + a) * p.o_sh + d, make_float4(v.x * by, v.y * by, v.z * by, v.w * by));
        }
      }
    }
    if (left >= 0 && !lost) refill(left);
    if (!seg.next(p)) break;
  }
}

constexpr int kMostPart = 2080;  // floats of a partial result of any form

// CTAs of a launch: as many as run at once, and have a counter.
int ctas_of(int num_sms, int resident) {
  const int most = WLLM_BLOCK_SCALED_COUNTER_BYTES / static_cast<int>(sizeof(int));
  const int ctas = num_sms * (resident < kMostCtas ? resident : kMostCtas);
  return ctas < most ? ctas : most;
}

template <int D, int NT>
int launch_tile(const CUtensorMap& kmap, const CUtensorMap& vmap, const ScaledDecodeParams& p, int num_sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  const void* kernel = reinterpret_cast<const void*>(&decode_block_scaled_kernel<D, NT>);
  static std::atomic<int> configured[64], found{0};
  const int e = raise_smem_limit(configured, kernel, S::kSmem);
  if (e != cudaSuccess) return e;
  int blocks = found.load(std::memory_order_relaxed);
  if (blocks == 0) {
    const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, &decode_block_scaled_kernel<D, NT>, kThreads, S::kSmem);
    if (err != cudaSuccess) return err;
    found.store(blocks, std::memory_order_relaxed);
  }
  static_assert(S::kPart <= kMostPart, "the workspace has room for every form's partial results");
  return launch_dependent(&decode_block_scaled_kernel<D, NT>, dim3(static_cast<unsigned>(ctas_of(num_sms, blocks))), dim3(kThreads),
                          S::kSmem, 0, stream, kmap, vmap, p);
}

}  // namespace

size_t decode_block_scaled_workspace(int num_sms) {
  return WLLM_BLOCK_SCALED_COUNTER_BYTES + size_t(ctas_of(num_sms, kMostCtas)) * 2 * kMostPart * sizeof(float);
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
  if (e == cudaSuccess) note_launch();
  return e;
}
}  // namespace wllm
