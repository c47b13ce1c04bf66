// sparse_decode.cu -- single-query attention over the selected blocks of each
// sequence and kv head.
//
// Mathematics: over the tokens t of the blocks listed for (b, kv head) that lie
// below the context length,
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t,
// one pass with a running maximum m and sum l per query head (log2 units):
//   O <- O 2^(m - m') + sum_t 2^(s_t - m') v_t.
//
// Tensor-core kernel (f16/bf16 and E4M3 caches).  A warp takes 16 tokens at a
// time; its K and V rows come by TMA (128-byte swizzle) into the warp's own ring
// of shared-memory stages, the next units' copies in flight while one is
// multiplied with mma.sync m16n8k16:
//   S[heads x tokens] = Q K^T: K rows by ldmatrix are the B operand, Q's heads
//     the A operand in registers (a tile of 8 heads leaves its lower half zero:
//     the instructions are not what bounds this);
//   O^T[dims x heads] += V^T P^T: V by ldmatrix.trans is the A operand, and S's
//     accumulator, in two 16-bit words (what the first leaves off is the
//     second), is already P^T's fragment.  Tensor cores take 16-bit weights; one
//     word alone, as the dense decode takes it, put 2^-9 (bf16) of a weight into
//     the output, which is as much as the output's own rounding.  The second
//     product costs nothing where memory sets the pace (256 sequences over E4M3
//     72.0 us without and 73.7 with it, 8 long ones 15.8 and 15.7) and 8 % where
//     two head tiles share a fragment of E4M3 codes (30.7 and 33.3).
// E4M3 codes are widened to f16 in registers, which is exact, with the head_dim
// order of the fp8 decode; bf16 queries are rounded to f16 for that product.
//
// Work split: the list of a (sequence, kv head, tile of up to 8 or 16 query
// heads) is divided over the warps of a cluster of 1 to 8 CTAs; warps meet in
// shared memory and CTAs in distributed shared memory, so short batches fill
// the GPU with neither a second launch nor a workspace, and in a fixed order.
// Bound: memory, each selected K and V byte is read once per head tile.  256
// sequences with 96 listed blocks, 28/4 heads of 128, E4M3 (401 MB): 73.6 us,
// 0.80 of the measured copy rate; 8 sequences with 128 blocks, 32/8 heads, bf16
// (67 MB): 15.8 us, 0.63, the rest lookups, the rings' filling and the merge.
//
// F32 caches keep the same split and rings with binary32 FMA (no tensor cores).
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

#include "decode_kernel.cuh"
#include "launch.h"
#include "mma_e4m3.cuh"

namespace cg = cooperative_groups;

namespace wllm {
namespace {

constexpr int kMaxSparseCluster = 8;

// Warps of a CTA and stages of a warp's ring.  Eight warps instead of four: 256
// sequences over an fp8 cache 76.4 instead of 73.7 us, one sequence 4.8 instead of 5.1.
// f32 units are bound by their FMA and take more warps with a stage each.
// DEEP: a stage more, for launches that leave the shared memory to it (launch_tile).
template <typename B, int D, bool DEEP>
struct SparseTuning {
  static constexpr int kStage = Geom<B, D>::kStageBytes;  // 16 tokens' K and V rows
  static constexpr bool kF32 = sizeof(B) == 4;
  static constexpr int kWarps = kStage >= 32768 || (kStage >= 16384 && !kF32) ? 2 : 4;
  static constexpr int kStages = (kF32 && kStage >= 16384 ? 1 : kStage >= 8192 ? 2 : kStage >= 4096 ? 3 : 6) + (DEEP ? 1 : 0);
  static constexpr bool kDeeper = sizeof(B) == 2 && kStage >= 8192;  // whether there is a deep form
  static constexpr int kRing = kStages * kStage;          // a warp's
};

// A unit of up to 16 listed tokens of one block: its physical block, its first
// row's offset in it, and how many of its rows are below the context length.
// Lanes look up 32 units at a time (the caller broadcasts).  Entries that are
// negative are padding; others outside the sequence are recorded and skipped.
struct Unit {
  int phys, off, live;
};

__device__ __forceinline__ Unit find_unit(const SparseParams& p, const int32_t* list, const int32_t* table,
                                          const int32_t* len_at, int64_t unit) {
  Unit u{0, 0, 0};
  const int log2_units = max(0, p.log2_bs - 4);  // units of a block
  const int64_t e = unit >> log2_units;
  if (e >= p.top) return u;
  // the length and the entry together, then the table: two round trips, not three
  const int stored = *len_at, id = list[e];
  const int max_blocks = p.max_tokens >> p.log2_bs;
  const int phys = id >= 0 && id < max_blocks ? table[id] : -1;
  const int len = min(max(stored, 0), p.max_tokens);
  if (id < 0 || len == 0) return u;
  if (id > (len - 1) >> p.log2_bs || phys < 0 || phys >= p.num_blocks) {
    atomicOr(p.err, kErrBlock);
    return u;
  }
  u.phys = phys;
  u.off = static_cast<int>(unit & ((1 << log2_units) - 1)) << 4;
  u.live = max(0, min(min(16, 1 << p.log2_bs), len - ((id << p.log2_bs) + u.off)));
  return u;
}

// Units of one list.
__device__ __forceinline__ int64_t units_of(const SparseParams& p) {
  return static_cast<int64_t>(p.top) << max(0, p.log2_bs - 4);
}

// Partial results of one warp or CTA in shared memory: [HT heads][D] outputs,
// then maxima and sums.
template <int D, int HT>
struct Partial {
  float o[HT][D];
  float m[HT];
  float l[HT];
};

// Merge of the warps' partials (one every `stride` bytes from `raw` on) and of
// the cluster's CTAs.  A partial's factor 2^(m_i - m) is computed once a head, by
// a warp with a lane a partial, into `scratch` [HT][parts]; then four
// neighbouring outputs are summed by a thread.  The warps' merge takes the first
// warp's partial's place; the CTAs' merge is shared by the cluster's ranks.
template <typename T, int D, int HT, int WARPS>
__device__ __forceinline__ void merge_and_store(const SparseParams& p, cg::cluster_group& cluster, uint8_t* raw, int stride,
                                                float* scratch, T* out, int heads) {
  constexpr int kThreads = WARPS * 32, kQuads = D / 4;
  static_assert(WARPS <= 8 && kMaxSparseCluster <= 8, "a factor a lane of 8");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  auto part = [&](int w) { return reinterpret_cast<Partial<D, HT>*>(raw + w * stride); };
  // 8 lanes a head: lane i of them has partial i's maximum and sum; returns the
  // merged ones and leaves the factors in scratch
  auto factors = [&](int h, bool have, float m_i, float l_i, float* m, float* l) {
    *m = have ? m_i : -INFINITY;
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) *m = fmaxf(*m, __shfl_xor_sync(kFullMask, *m, x));
    const float f = !have || m_i == -INFINITY ? 0.f : exp2f(m_i - *m);
    *l = have ? f * l_i : 0.f;
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) *l += __shfl_xor_sync(kFullMask, *l, x);
    return f;
  };
  __syncthreads();
  float m_cta = 0.f, l_cta = 0.f;
  for (int h0 = warp * 4; h0 < HT; h0 += WARPS * 4) {
    const int h = min(h0 + (lane >> 3), HT - 1), i = lane & 7;
    const bool have = i < WARPS;
    const Partial<D, HT>* x = part(have ? i : 0);
    const float f = factors(h, have, x->m[h], x->l[h], &m_cta, &l_cta);
    // with one CTA the division is part of the factor
    if (have) scratch[h * 8 + i] = ctas > 1 ? f : l_cta == 0.f ? 0.f : f * (p.v_scale / l_cta);
    __syncwarp();  // every lane has read the partials' maxima
    if (i == 0) part(0)->m[h] = m_cta, part(0)->l[h] = l_cta;
  }
  __syncthreads();
  for (int i = tid; i < heads * kQuads; i += kThreads) {
    const int h = i / kQuads, d = (i - h * kQuads) * 4;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(&part(w)->o[h][d]);
      const float f = scratch[h * 8 + w];
      o[0] = fmaf(f, v.x, o[0]), o[1] = fmaf(f, v.y, o[1]), o[2] = fmaf(f, v.z, o[2]), o[3] = fmaf(f, v.w, o[3]);
    }
    if (ctas > 1) {
      *reinterpret_cast<float4*>(&part(0)->o[h][d]) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[h * p.o_sh + d + e] = from_f32<T>(o[e]);
    }
  }
  if (ctas == 1) return;
  cluster.sync();
  for (int h0 = warp * 4; h0 < HT; h0 += WARPS * 4) {
    const int h = min(h0 + (lane >> 3), HT - 1), i = lane & 7;
    const bool have = i < ctas;
    const Partial<D, HT>* x = cluster.map_shared_rank(part(0), have ? i : 0);
    float m, l;
    const float f = factors(h, have, x->m[h], x->l[h], &m, &l);
    if (have) scratch[h * 8 + i] = l == 0.f ? 0.f : f * (p.v_scale / l);
  }
  __syncthreads();
  for (int i = rank * kThreads + tid; i < heads * kQuads; i += ctas * kThreads) {
    const int h = i / kQuads, d = (i - h * kQuads) * 4;
    float4 v[kMaxSparseCluster];
#pragma unroll
    for (int r = 0; r < kMaxSparseCluster; ++r)
      if (r < ctas) v[r] = *reinterpret_cast<const float4*>(&cluster.map_shared_rank(part(0), r)->o[h][d]);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kMaxSparseCluster; ++r) {
      if (r < ctas) {
        const float f = scratch[h * 8 + r];
        o[0] = fmaf(f, v[r].x, o[0]), o[1] = fmaf(f, v[r].y, o[1]), o[2] = fmaf(f, v[r].z, o[2]), o[3] = fmaf(f, v[r].w, o[3]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) out[h * p.o_sh + d + e] = from_f32<T>(o[e]);
  }
  cluster.sync();  // a CTA's shared memory outlives its peers' reads
}

// First words of two weights: below them, so that what is left for the second
// word is positive and an infinite value comes out infinite (a second word of 0
// would make it NaN, a negative one too).  Cut off to the 16-bit type: the second
// word holds the rest within 2^-15 (bf16) or 2^-21 (f16) of the weight.
__device__ __forceinline__ uint32_t first_words(float w0, float w1, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(w1 * 0.99999237f), "f"(w0 * 0.99999237f));  // 1 - 2^-17
  return r;
}
__device__ __forceinline__ uint32_t first_words(float w0, float w1, __half) {
  uint32_t r;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(w1 * 0.99975586f), "f"(w0 * 0.99975586f));  // 1 - 2^-12
  return r;
}

// The products of one warp on tensor cores.
template <typename T, bool F8, int D, int HT>
struct MmaMath {
  using M = typename std::conditional<F8, __half, T>::type;
  static constexpr int kNT = HT / 8;  // tiles of 8 heads
  static constexpr int kKS = D / 16;  // k16 steps over head_dim
  static constexpr int kQueryBytes = 0;
  // weights and their sum are taken times 2^14 in f16: second words are normal numbers then down to weights of 2^-16
  static constexpr float kWeightShift = std::is_same<M, __half>::value ? 14.f : 0.f;
  uint32_t qf[kNT][kKS][2];
  float m[kNT], l[kNT], o[kKS][kNT][4];

  __device__ __forceinline__ void load_q(const SparseParams& p, float*, int b, int head0, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // Q fragments: head 8a + g; elements 16s + 2c (+8) of 16-bit rows, 16s + 4c (+2) where codes are widened
#pragma unroll
    for (int a = 0; a < kNT; ++a)
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t x = 0u;
          if (8 * a + g < heads) {
            const int d = F8 ? 16 * s + 4 * c + 2 * e : 16 * s + 2 * c + 8 * e;
            const T* q = static_cast<const T*>(p.q) + b * p.q_sb + (head0 + 8 * a + g) * p.q_sh + d;
            if (p.q_pairs) {
              x = *reinterpret_cast<const uint32_t*>(q);
            } else {
              const uint16_t lo = *reinterpret_cast<const uint16_t*>(q), hi = *reinterpret_cast<const uint16_t*>(q + 1);
              x = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
            }
            if constexpr (F8) x = to_f16x2<T>(x);
          }
          qf[a][s][e] = x;
        }
#pragma unroll
    for (int a = 0; a < kNT; ++a) m[a] = -INFINITY, l[a] = 0.f;
#pragma unroll
    for (int t = 0; t < kKS; ++t)
#pragma unroll
      for (int a = 0; a < kNT; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][a][e] = 0.f;
  }

  // 16 tokens whose K rows are at shared address kt and V rows at vt, the first `live` of them.
  __device__ __forceinline__ void step(uint32_t kt, uint32_t vt, int live, float scale_log2) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    // S = Q K^T, tokens 0-7 and 8-15
    float s[2][4];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[half][e] = 0.f;
    // chunks of four steps first, then their products
    constexpr int kGroup = kKS < 4 ? kKS : 4;
#pragma unroll
    for (int s0 = 0; s0 < kKS; s0 += kGroup) {
      uint32_t bf[kGroup][2][2];  // [step][half]
      if constexpr (F8) {
        const int k_row = (lane & 7) + (((lane >> 3) & 1) << 3), k_chunk = lane >> 4;
        uint32_t r[kGroup / 2][4];  // tokens 0-7 and 8-15 of a chunk, then of the next
#pragma unroll
        for (int x = 0; x < kGroup / 2; ++x) ldsm_x4(kt + code_offset<D>(k_row, s0 + 2 * x + k_chunk), r[x]);
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) e4m3x4_to_f16x2x2(r[i >> 1][2 * (i & 1) + half], bf[i][half][0], bf[i][half][1]);
      } else {
        const int k_row = (lane & 7) + ((lane >> 4) << 3), k_chunk = (lane >> 3) & 1;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          uint32_t r[4];  // chunks 2 step and 2 step + 1 of tokens 0-7, then of tokens 8-15
          ldsm_x4(kt + tile_offset(k_row, 2 * (s0 + i) + k_chunk), r);
          bf[i][0][0] = r[0], bf[i][0][1] = r[1], bf[i][1][0] = r[2], bf[i][1][1] = r[3];
        }
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const uint32_t af[4] = {qf[0][s0 + i][0], kNT > 1 ? qf[kNT - 1][s0 + i][0] : 0u, qf[0][s0 + i][1],
                                kNT > 1 ? qf[kNT - 1][s0 + i][1] : 0u};
        Mma<M>::run(s[0], af, bf[i][0]);
        Mma<M>::run(s[1], af, bf[i][1]);
      }
    }
    // weights: head 8a + g, tokens 2c, 2c + 1 of both halves
    uint32_t pf[kNT][2], pr[kNT][2];
#pragma unroll
    for (int a = 0; a < kNT; ++a) {
      float x[4];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[2 * half + e] = 8 * half + 2 * c + e < live ? s[half][2 * a + e] * scale_log2 : -INFINITY;
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      const float mn = fmaxf(m[a], top);
      if (__any_sync(kFullMask, mn > m[a])) {
        const float f = m[a] == -INFINITY ? 0.f : exp2f(m[a] - mn);
        l[a] *= f;
        m[a] = mn;
        const float f0 = __shfl_sync(kFullMask, f, 8 * c), f1 = __shfl_sync(kFullMask, f, 8 * c + 4);
#pragma unroll
        for (int t = 0; t < kKS; ++t) {
          o[t][a][0] *= f0, o[t][a][1] *= f1, o[t][a][2] *= f0, o[t][a][3] *= f1;
        }
      }
      const float base = (m[a] == -INFINITY ? 0.f : m[a]) - kWeightShift;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float w0 = ex2_approx(x[2 * half] - base), w1 = ex2_approx(x[2 * half + 1] - base);
        pf[a][half] = first_words(w0, w1, M());
        const M* w = reinterpret_cast<const M*>(&pf[a][half]);
        pr[a][half] = Mma<M>::pack(w0 - to_f32(w[0]), w1 - to_f32(w[1]));
        l[a] += w0 + w1;
      }
    }
    // O^T += V^T P^T; V rows behind the context are zeroed (they may hold anything)
    const bool tail = live < 16;
    const uint32_t keep_lo = (2 * c < live ? 0x0000ffffu : 0u) | (2 * c + 1 < live ? 0xffff0000u : 0u);
    const uint32_t keep_hi = (2 * c + 8 < live ? 0x0000ffffu : 0u) | (2 * c + 9 < live ? 0xffff0000u : 0u);
    const int v_row = F8 ? (lane & 7) + (((lane >> 3) & 1) << 3) : (lane & 7) + ((lane >> 4) << 3);
    const int v_chunk = F8 ? lane >> 4 : (lane >> 3) & 1;
#pragma unroll
    for (int t0 = 0; t0 < kKS; t0 += kGroup) {
      uint32_t af[kGroup][4];
      if constexpr (F8) {
        uint32_t r[kGroup / 2][4];  // tokens 0-7 and 8-15 of a chunk, then of the next
#pragma unroll
        for (int x = 0; x < kGroup / 2; ++x) ldsm_x4_trans(vt + code_offset<D>(v_row, t0 + 2 * x + v_chunk), r[x]);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          // bytes (t, e), (t, e+1), (t+1, e), (t+1, e+1) -> (t, e), (t+1, e), (t, e+1), (t+1, e+1)
          e4m3x4_to_f16x2x2(__byte_perm(r[i >> 1][2 * (i & 1)], 0u, 0x3120), af[i][0], af[i][1]);
          e4m3x4_to_f16x2x2(__byte_perm(r[i >> 1][2 * (i & 1) + 1], 0u, 0x3120), af[i][2], af[i][3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) ldsm_x4_trans(vt + tile_offset(v_row, 2 * (t0 + i) + v_chunk), af[i]);
      }
      if (tail) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) af[i][0] &= keep_lo, af[i][1] &= keep_lo, af[i][2] &= keep_hi, af[i][3] &= keep_hi;
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
#pragma unroll
        for (int a = 0; a < kNT; ++a) {
          Mma<M>::run(o[t0 + i][a], af[i], pf[a]);
          Mma<M>::run(o[t0 + i][a], af[i], pr[a]);
        }
    }
  }

  __device__ __forceinline__ void store(Partial<D, HT>& out, int) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int a = 0; a < kNT; ++a) {
      l[a] += __shfl_xor_sync(kFullMask, l[a], 1);
      l[a] += __shfl_xor_sync(kFullMask, l[a], 2);
      if (c == 0) {
        out.m[8 * a + g] = m[a];
        out.l[8 * a + g] = l[a];
      }
#pragma unroll
      for (int t = 0; t < kKS; ++t) {
        if constexpr (F8) {  // rows g and g + 8 are elements 16t + 2g and 16t + 2g + 1
          const int d = 16 * t + 2 * g;
          *reinterpret_cast<float2*>(&out.o[8 * a + 2 * c][d]) = make_float2(o[t][a][0], o[t][a][2]);
          *reinterpret_cast<float2*>(&out.o[8 * a + 2 * c + 1][d]) = make_float2(o[t][a][1], o[t][a][3]);
        } else {
          const int d = 16 * t + g;
          out.o[8 * a + 2 * c][d] = o[t][a][0];
          out.o[8 * a + 2 * c + 1][d] = o[t][a][1];
          out.o[8 * a + 2 * c][d + 8] = o[t][a][2];
          out.o[8 * a + 2 * c + 1][d + 8] = o[t][a][3];
        }
      }
    }
  }
};

// The same in binary32 FMA.  Scores: lane (token t of 8, quarter of the 16-byte
// chunks) has tokens t and t + 8, so a query chunk, the same for the 8 lanes of a
// quarter, serves 8 products and K's chunks meet no bank twice; the quarters are
// summed by shuffles.  Outputs: D/32 columns a lane, weights from shared memory.
template <int D, int HT>
struct FmaMath {
  static constexpr int kCols = D / 32, kPs = 16 * HT;
  static constexpr int kQueryBytes = (HT * D + 4 * kPs) * 4;  // queries, then a warp's weights for up to 4 warps
  float m[HT], l[HT], o[HT][kCols];
  const float* qs;
  float* ps;

  __device__ __forceinline__ void load_q(const SparseParams& p, float* queries, int b, int head0, int heads) {
    for (int i = threadIdx.x; i < HT * D; i += blockDim.x) {
      const int a = i / D, d = i - a * D;
      queries[i] = a < heads ? static_cast<const float*>(p.q)[b * p.q_sb + (head0 + a) * p.q_sh + d] : 0.f;
    }
    qs = queries;
    ps = queries + HT * D + (threadIdx.x >> 5) * kPs;
#pragma unroll
    for (int a = 0; a < HT; ++a) {
      m[a] = -INFINITY, l[a] = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[a][i] = 0.f;
    }
    __syncthreads();
  }

  // One token's V columns of this lane.
  static __device__ __forceinline__ void value(const uint8_t* v, int token, int lane, float (&x)[kCols]) {
    if constexpr (kCols == 2) {
      const float2 y = *reinterpret_cast<const float2*>(v + tile_offset(token, lane >> 1) + (lane & 1) * 8);
      x[0] = y.x, x[1] = y.y;
    } else {
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 y = *reinterpret_cast<const float4*>(v + tile_offset(token, lane + 32 * i));
        x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
      }
    }
  }

  __device__ __forceinline__ void step(uint32_t kt, uint32_t vt, int live, float scale_log2) {
    const uint8_t* k = static_cast<const uint8_t*>(__cvta_shared_to_generic(kt));
    const uint8_t* v = static_cast<const uint8_t*>(__cvta_shared_to_generic(vt));
    const int lane = threadIdx.x & 31, tok = lane & 7, quarter = lane >> 3;
    float s[2][HT];
#pragma unroll
    for (int a = 0; a < HT; ++a) s[0][a] = s[1][a] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 16; ++c) {
      const float4 k0 = *reinterpret_cast<const float4*>(k + tile_offset(tok, 4 * c + quarter));
      const float4 k1 = *reinterpret_cast<const float4*>(k + tile_offset(tok + 8, 4 * c + quarter));
#pragma unroll
      for (int a = 0; a < HT; ++a) {
        const float4 q = *reinterpret_cast<const float4*>(qs + a * D + (4 * c + quarter) * 4);
        s[0][a] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[0][a]))));
        s[1][a] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[1][a]))));
      }
    }
    bool moved = false;
    float f[HT];
#pragma unroll
    for (int a = 0; a < HT; ++a) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        s[x][a] += __shfl_xor_sync(kFullMask, s[x][a], 8);
        s[x][a] += __shfl_xor_sync(kFullMask, s[x][a], 16);
        s[x][a] = tok + 8 * x < live ? s[x][a] * scale_log2 : -INFINITY;
      }
      float top = fmaxf(s[0][a], s[1][a]);
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
      const float mn = fmaxf(m[a], top);
      f[a] = m[a] == -INFINITY ? 0.f : exp2f(m[a] - mn);
      moved |= mn > m[a];
      m[a] = mn;
      const float base = mn == -INFINITY ? 0.f : mn;
      s[0][a] = exp2f(s[0][a] - base);
      s[1][a] = exp2f(s[1][a] - base);
      l[a] = fmaf(l[a], f[a], s[0][a] + s[1][a]);
    }
    if (moved) {  // the same in every lane
#pragma unroll
      for (int a = 0; a < HT; ++a)
#pragma unroll
        for (int i = 0; i < kCols; ++i) o[a][i] *= f[a];
    }
    __syncwarp();
    if (quarter < 2) {  // each writes one of its lanes' two tokens
#pragma unroll
      for (int a = 0; a < HT; ++a) ps[(tok + 8 * quarter) * HT + a] = quarter ? s[1][a] : s[0][a];
    }
    __syncwarp();
    auto add = [&](int t) {
      float x[kCols], w[HT];
      value(v, t, lane, x);
      if constexpr (HT % 4 == 0) {
#pragma unroll
        for (int a = 0; a < HT; a += 4) {
          const float4 y = *reinterpret_cast<const float4*>(ps + t * HT + a);
          w[a] = y.x, w[a + 1] = y.y, w[a + 2] = y.z, w[a + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int a = 0; a < HT; ++a) w[a] = ps[t * HT + a];
      }
#pragma unroll
      for (int a = 0; a < HT; ++a)
#pragma unroll
        for (int i = 0; i < kCols; ++i) o[a][i] = fmaf(w[a], x[i], o[a][i]);
    };
    if (live == 16) {
#pragma unroll 8
      for (int t = 0; t < 16; ++t) add(t);
    } else {
      for (int t = 0; t < live; ++t) add(t);  // rows behind the context may hold anything
    }
  }

  __device__ __forceinline__ void store(Partial<D, HT>& out, int) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int a = 0; a < HT; ++a) {
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) l[a] += __shfl_xor_sync(kFullMask, l[a], x);
      if (lane == 0) out.m[a] = m[a], out.l[a] = l[a];
#pragma unroll
      for (int i = 0; i < kCols; ++i) out.o[a][kCols == 2 ? lane * 2 + i : (lane + 32 * (i >> 2)) * 4 + (i & 3)] = o[a][i];
    }
  }
};

template <typename T, bool F8, int D, int HT>
struct SparseMath {
  using type = MmaMath<T, F8, D, HT>;
};
template <int D, int HT>
struct SparseMath<float, false, D, HT> {
  using type = FmaMath<D, HT>;
};

// --- the kernel -------------------------------------------------------------------
// T: query and output type; F8: the caches hold E4M3 codes.
template <typename T, bool F8, int D, int HT, bool DEEP>
__global__ void __launch_bounds__((SparseTuning<typename std::conditional<F8, uint8_t, T>::type, D, DEEP>::kWarps * 32))
    sparse_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const SparseParams p) {
  using B = typename std::conditional<F8, uint8_t, T>::type;
  using G = Geom<B, D>;
  using Tune = SparseTuning<B, D, DEEP>;
  using Math = typename SparseMath<T, F8, D, HT>::type;
  constexpr int kWarps = Tune::kWarps, kStages = Tune::kStages;
  static_assert(sizeof(Partial<D, HT>) <= Tune::kRing, "a warp's partial takes its ring's place");

  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  int64_t row = static_cast<int64_t>(blockIdx.x) / ctas;
  const int tile = static_cast<int>(row % p.num_head_tiles);
  row /= p.num_head_tiles;
  const int h = static_cast<int>(row % p.num_kv_heads), b = static_cast<int>(row / p.num_kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = min(HT, p.group - tile * HT);
  const int head0 = h * p.group + tile * HT;

  extern __shared__ __align__(16) uint8_t unaligned[];
  uint8_t* raw = unaligned + ((1024 - (smem_u32(unaligned) & 1023)) & 1023);  // swizzled boxes start at 1024 bytes
  uint8_t* ring = raw + warp * Tune::kRing;
  float* scratch = reinterpret_cast<float*>(raw + kWarps * Tune::kRing);  // [HT][8]
  float* queries = scratch + HT * 8;
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(queries) + Math::kQueryBytes) + warp * kStages;
  if (lane < kStages) mbar_init(smem_u32(&bars[lane]), 1);
  fence_mbar_init();
  if (lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
  __syncwarp();
  grid_wait();
  grid_launch_dependents();

  const int32_t* len_at = p.context_lens + b;
  const int32_t* list = p.selected + b * p.sel_sb + h * p.sel_sh;
  const int32_t* table = p.block_tables + b * p.bt_stride;
  const int64_t units = units_of(p);
  const int stride = ctas * kWarps;

  // 32 units of this warp, a lane each; those with tokens
  Unit mine{0, 0, 0};
  int64_t u0 = rank * kWarps + warp;
  auto find = [&]() -> unsigned {
    mine.live = 0;
    if (u0 + int64_t(lane) * stride < units) mine = find_unit(p, list, table, len_at, u0 + int64_t(lane) * stride);
    return __ballot_sync(kFullMask, mine.live > 0);
  };
  unsigned to_use = u0 < units ? find() : 0u, to_copy = to_use;
  int next_stage = 0;  // of the copies; the uses follow in the same order
  const uint32_t box_bytes = 128u * (G::kPairRows ? 8u : static_cast<uint32_t>(min(16, 1 << p.log2_bs)));
  auto copy = [&] {  // the next unit's K and V rows, one box a lane
    const int from = __ffs(to_copy) - 1;
    to_copy &= to_copy - 1;
    const int phys = __shfl_sync(kFullMask, mine.phys, from), off = __shfl_sync(kFullMask, mine.off, from);
    const uint32_t bar = smem_u32(&bars[next_stage]), dst = smem_u32(ring + next_stage * Tune::kStage);
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * G::kColBoxes * box_bytes);
    __syncwarp();
    if (lane < 2 * G::kColBoxes) {
      const bool is_v = lane >= G::kColBoxes;
      const int box = lane - (is_v ? G::kColBoxes : 0);
      const int at = (h << p.log2_bs) + off;
      tma_load_3d(dst + (is_v ? G::kTileBytes : 0) + box * 2048, is_v ? &vmap : &kmap, bar, box * G::kBoxCols,
                  G::kPairRows ? at >> 1 : at, phys);
    }
    next_stage = next_stage + 1 == kStages ? 0 : next_stage + 1;
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s)
    if (to_copy) copy();

  Math math;
  math.load_q(p, queries, b, head0, heads);

  int stage = 0;
  uint32_t phase = 0u;  // of every stage, turned when the ring comes round
  bool lost = false;
  while (u0 < units && !lost) {
    while (to_use) {
      const int from = __ffs(to_use) - 1;
      to_use &= to_use - 1;
      const int live = __shfl_sync(kFullMask, mine.live, from);
      if (!mbar_wait_warp(smem_u32(&bars[stage]), phase, p.wait_limit_ns)) {
        // give up: record it, let what is in flight land (again with a limit), and take no more units
        if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
        for (int s = 0; s < kStages; ++s) mbar_wait_bounded(smem_u32(&bars[s]), s >= stage ? phase : phase ^ 1u, p.wait_limit_ns);
        lost = true;
        break;
      }
      const uint32_t kt = smem_u32(ring + stage * Tune::kStage), vt = kt + G::kTileBytes;
      math.step(kt, vt, live, p.scale_log2);
      __syncwarp();  // every lane has read the stage
      if (to_copy) copy();
      if (++stage == kStages) stage = 0, phase ^= 1u;
    }
    if (lost) break;
    u0 += 32LL * stride;
    if (u0 >= units) break;
    to_use = to_copy = find();
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (to_copy) copy();
  }

  math.store(*reinterpret_cast<Partial<D, HT>*>(ring), lane);  // in the place of the ring
  if (threadIdx.x == 0 && rank == 0 && h == 0 && tile == 0 && (*len_at < 0 || *len_at > p.max_tokens))
    atomicOr(p.err, kErrLen);
  merge_and_store<T, D, HT, kWarps>(p, cluster, raw, Tune::kRing, scratch, static_cast<T*>(p.out) + b * p.o_sb + head0 * p.o_sh,
                                    heads);
}

// CTAs of a list: as many as run at once (`resident` an SM), but no warp under
// one unit.  Measured, us for 1, 2, 4 and 8 CTAs a list: 64 lists of 128 blocks
// (bf16, two stages) 23.3, 17.7, 16.5, 22.0; 1024 of 96 (fp8) 73.7, 84.5, 107, 161; 4 of 64
// (f16, head_dim 64) 10.2, 7.7, 5.9, 5.1.
int cluster_size(const SparseParams& p, int warps, int resident, int num_sms) {
  const int64_t rows = int64_t(p.num_seqs) * p.num_kv_heads * p.num_head_tiles;
  const int64_t units = int64_t(p.top) << (p.log2_bs > 4 ? p.log2_bs - 4 : 0);
  int ctas = 1;
  while (ctas < kMaxSparseCluster && rows * ctas * 2 <= int64_t(num_sms) * resident && units >= 2 * ctas * warps) ctas *= 2;
  return ctas;
}

dim3 grid_of(const SparseParams& p, int ctas) {
  return dim3(static_cast<unsigned>(int64_t(p.num_seqs) * p.num_kv_heads * p.num_head_tiles * ctas));
}

// One form of the kernel: its shared memory, and how many CTAs of it an SM holds.
template <typename T, bool F8, int D, int HT, bool DEEP>
struct SparseForm {
  using Tune = SparseTuning<typename std::conditional<F8, uint8_t, T>::type, D, DEEP>;
  static constexpr size_t kSmem = 1024 + Tune::kWarps * (Tune::kRing + Tune::kStages * sizeof(uint64_t)) +
                                  HT * 8 * sizeof(float) + SparseMath<T, F8, D, HT>::type::kQueryBytes;

  static int resident(int* blocks) {
    static std::atomic<int> configured[64], found{0};
    const int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&sparse_kernel<T, F8, D, HT, DEEP>),
                                   static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    *blocks = found.load(std::memory_order_relaxed);
    if (*blocks == 0) {
      const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, &sparse_kernel<T, F8, D, HT, DEEP>,
                                                                            Tune::kWarps * 32, kSmem);
      if (err != cudaSuccess) return err;
      found.store(*blocks, std::memory_order_relaxed);
    }
    return cudaSuccess;
  }

  static int launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const SparseParams& p, int ctas, cudaStream_t stream) {
    return launch_dependent(&sparse_kernel<T, F8, D, HT, DEEP>, grid_of(p, ctas), dim3(Tune::kWarps * 32), kSmem, ctas,
                            stream, kmap, vmap, p);
  }
};

template <typename T, bool F8, int D, int HT>
int launch_tile(const CUtensorMap& kmap, const CUtensorMap& vmap, const SparseParams& p, int num_sms, cudaStream_t stream) {
  using Form = SparseForm<T, F8, D, HT, false>;
  int blocks = 0;
  int e = Form::resident(&blocks);
  if (e != cudaSuccess) return e;
  const int ctas = cluster_size(p, Form::Tune::kWarps, blocks, num_sms);
  if constexpr (Form::Tune::kDeeper) {
    // The deep form where all its CTAs run at once too.  Measured, us with 2 and 3 stages: 64 lists of 128 blocks (bf16)
    // 17.0 and 15.6, 256 of 64 27.3 and 24.6, 32 of 64 with head_dim 256 12.0 and 10.8; behind a fill 19.6 and 19.5, 27.3
    // and 24.6, 15.1 and 14.8.  Not so for E4M3 codes: 1024 lists 73.7 and 85.3 (3 and 4), 256 18.3 and 18.3.
    using Deep = SparseForm<T, F8, D, HT, true>;
    if ((e = Deep::resident(&blocks)) != cudaSuccess) return e;
    if (int64_t(grid_of(p, ctas).x) <= int64_t(num_sms) * blocks) return Deep::launch(kmap, vmap, p, ctas, stream);
  }
  return Form::launch(kmap, vmap, p, ctas, stream);
}

template <int HT>
int launch_f32(const CUtensorMap& kmap, const CUtensorMap& vmap, const SparseParams& p, int head_dim, int num_sms,
               cudaStream_t stream) {
  if (head_dim == 64) return launch_tile<float, false, 64, HT>(kmap, vmap, p, num_sms, stream);
  if (head_dim == 128) return launch_tile<float, false, 128, HT>(kmap, vmap, p, num_sms, stream);
  if (head_dim == 256) return launch_tile<float, false, 256, HT>(kmap, vmap, p, num_sms, stream);
  return cudaErrorInvalidValue;
}

template <typename T, bool F8>
int launch_dim(const CUtensorMap& kmap, const CUtensorMap& vmap, const SparseParams& p, int head_dim, int head_tile,
               int num_sms, cudaStream_t stream) {
  if (head_dim == 64)
    return head_tile == 16 ? launch_tile<T, F8, 64, 16>(kmap, vmap, p, num_sms, stream)
                           : launch_tile<T, F8, 64, 8>(kmap, vmap, p, num_sms, stream);
  if (head_dim == 128)
    return head_tile == 16 ? launch_tile<T, F8, 128, 16>(kmap, vmap, p, num_sms, stream)
                           : launch_tile<T, F8, 128, 8>(kmap, vmap, p, num_sms, stream);
  if (head_dim == 256) return launch_tile<T, F8, 256, 8>(kmap, vmap, p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

int launch_sparse_decode(int dtype, bool kv_fp8, int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         SparseParams p, int num_sms, cudaStream_t stream) {
  // two tiles of 8 query heads share the K/V fragments where registers allow;
  // binary32 products are not made for heads that are not there
  const int head_tile = dtype == 0 ? (p.group == 1 ? 1 : p.group <= 4 ? 4 : 8) : p.group > 8 && head_dim <= 128 ? 16 : 8;
  p.num_head_tiles = (p.group + head_tile - 1) / head_tile;
  int e = cudaErrorInvalidValue;
  if (dtype == 0 && !kv_fp8) {
    e = head_tile == 1   ? launch_f32<1>(kmap, vmap, p, head_dim, num_sms, stream)
        : head_tile == 4 ? launch_f32<4>(kmap, vmap, p, head_dim, num_sms, stream)
                         : launch_f32<8>(kmap, vmap, p, head_dim, num_sms, stream);
  } else if (dtype == 1) {
    e = kv_fp8 ? launch_dim<__half, true>(kmap, vmap, p, head_dim, head_tile, num_sms, stream)
               : launch_dim<__half, false>(kmap, vmap, p, head_dim, head_tile, num_sms, stream);
  } else if (dtype == 2) {
    e = kv_fp8 ? launch_dim<__nv_bfloat16, true>(kmap, vmap, p, head_dim, head_tile, num_sms, stream)
               : launch_dim<__nv_bfloat16, false>(kmap, vmap, p, head_dim, head_tile, num_sms, stream);
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
