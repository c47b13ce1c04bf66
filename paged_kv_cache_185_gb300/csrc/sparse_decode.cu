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
// time straight from global memory into mma.sync m16n8k16 fragments, without a
// stage in shared memory:
//   S[heads x tokens] = Q K^T: a lane (g = lane/4, c = lane%4) loads 16 bytes
//     of token row g at chunk 4i + c.  Its elements serve as k indices
//     2c, 2c+1, 2c+8, 2c+9 of consecutive k16 steps; the sum over head_dim
//     takes any order, so Q's fragment takes the same one.
//   O^T[dims x heads] += V^T P^T: a lane loads chunk g (+8i) of the rows
//     2c, 2c+1, 2c+8, 2c+9; one byte permute pairs two rows' element, which is
//     a word of the A fragment with row g = element 2i and row g+8 = element
//     2i+1 of the lane's chunk.  P^T's fragment is S's accumulator, rounded to
//     the 16-bit type (tensor cores take 16-bit weights; the sum l adds the
//     rounded weights, so numerator and denominator agree).
// Every 16-byte load is part of a whole 64- or 128-byte run.  E4M3 codes are
// widened to f16 in registers, which is exact; bf16 queries are rounded to f16
// for that product, as in the decode over an fp8 cache.
//
// Work split: the list of a (sequence, kv head, tile of up to 8 or 16 query
// heads) is divided over the warps of a cluster of 1 to 8 CTAs; warps meet in
// shared memory and CTAs in distributed shared memory, so short batches fill
// the GPU with neither a second launch nor a workspace, and in a fixed order.
// Bound: memory, each selected K and V byte is read once per head tile.
//
// The f32 kernel keeps the same split with binary32 FMA (no tensor cores).
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace wllm {
namespace {

constexpr int kSparseWarps = 4;
constexpr int kSparseThreads = kSparseWarps * 32;
constexpr int kMaxSparseCluster = 8;

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Where a warp's next 16 tokens are: for each half of 8 rows the byte offset
// of its first row and how many of its rows are below the context length.
struct UnitRows {
  int64_t at[2];
  int live[2];
};

// Units of 16 listed tokens; unit u covers list positions 16u .. 16u+15.
// Lanes look up 32 units at a time (the caller broadcasts).  Entries that are
// negative are padding; others outside the sequence are recorded and skipped.
struct UnitLookup {
  int64_t at[2];
  int live[2];
  __device__ __forceinline__ void fetch(const SparseParams& p, const int32_t* list, const int32_t* table, int len, int h,
                                        int row_bytes, int64_t unit) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t pos = unit * 16 + half * 8;
      at[half] = 0;
      live[half] = 0;
      if (half == 1 && p.log2_bs > 3) {  // both halves lie in one block
        at[1] = at[0] + 8 * row_bytes;
        live[1] = max(0, live[0] - 8);
        live[0] = min(8, live[0]);
        continue;
      }
      const int64_t e = pos >> p.log2_bs;
      if (e >= p.top || len == 0) continue;
      const int id = __ldg(list + e);
      if (id < 0) continue;
      const int off = static_cast<int>(pos) & ((1 << p.log2_bs) - 1);
      if (id > (len - 1) >> p.log2_bs) {
        atomicOr(p.err, kErrBlock);
        continue;
      }
      const int phys = __ldg(table + id);
      if (phys < 0 || phys >= p.num_blocks) {
        atomicOr(p.err, kErrBlock);
        continue;
      }
      at[half] = (((static_cast<int64_t>(phys) * p.num_kv_heads + h) << p.log2_bs) + off) * row_bytes;
      live[half] = max(0, min(p.log2_bs > 3 ? 16 : 8, len - ((id << p.log2_bs) + off)));
    }
  }
};

// Partial results of one warp or CTA in shared memory: [HT heads][D] outputs,
// then maxima and sums.
template <int D, int HT>
struct Partial {
  float o[HT][D];
  float m[HT];
  float l[HT];
};

// Merge of the warps' partials (in `part`, one a warp) and of the cluster's
// CTAs; the cluster's ranks share the output elements of the tile.
template <typename T, int D, int HT>
__device__ __forceinline__ void merge_and_store(const SparseParams& p, cg::cluster_group& cluster, Partial<D, HT>* part,
                                                T* out, int heads) {
  const int tid = threadIdx.x, ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  __syncthreads();
  if (ctas == 1) {
    for (int i = tid; i < heads * D; i += kSparseThreads) {
      const int h = i / D, d = i - h * D;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSparseWarps; ++w) m = fmaxf(m, part[w].m[h]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kSparseWarps; ++w) {
        const float f = part[w].m[h] == -INFINITY ? 0.f : exp2f(part[w].m[h] - m);
        l = fmaf(f, part[w].l[h], l);
        o = fmaf(f, part[w].o[h][d], o);
      }
      out[h * p.o_sh + d] = from_f32<T>(l == 0.f ? 0.f : o / l * p.v_scale);
    }
    return;
  }
  // this CTA's merge, in place of its first warp's partial
  float mc[kSparseWarps];
  for (int i = tid; i < heads * D; i += kSparseThreads) {
    const int h = i / D, d = i - h * D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) m = fmaxf(m, part[w].m[h]);
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
      mc[w] = part[w].m[h] == -INFINITY ? 0.f : exp2f(part[w].m[h] - m);
      o = fmaf(mc[w], part[w].o[h][d], o);
    }
    part[0].o[h][d] = o;
  }
  __syncthreads();
  if (tid < heads) {
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) m = fmaxf(m, part[w].m[tid]);
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
      const float f = part[w].m[tid] == -INFINITY ? 0.f : exp2f(part[w].m[tid] - m);
      l = fmaf(f, part[w].l[tid], l);
    }
    part[0].m[tid] = m;
    part[0].l[tid] = l;
  }
  cluster.sync();
  for (int i = rank * kSparseThreads + tid; i < heads * D; i += ctas * kSparseThreads) {
    const int h = i / D, d = i - h * D;
    float ms[kMaxSparseCluster], ls[kMaxSparseCluster], os[kMaxSparseCluster];
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < kMaxSparseCluster; ++r) {
      if (r < ctas) {
        const Partial<D, HT>* peer = cluster.map_shared_rank(part, r);
        ms[r] = peer->m[h], ls[r] = peer->l[h], os[r] = peer->o[h][d];
        m = fmaxf(m, ms[r]);
      }
    }
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxSparseCluster; ++r) {
      if (r < ctas) {
        const float f = ms[r] == -INFINITY ? 0.f : exp2f(ms[r] - m);
        l = fmaf(f, ls[r], l);
        o = fmaf(f, os[r], o);
      }
    }
    out[h * p.o_sh + d] = from_f32<T>(l == 0.f ? 0.f : o / l * p.v_scale);
  }
  cluster.sync();  // a CTA's shared memory outlives its peers' reads
}

template <typename T>
__device__ __forceinline__ uint32_t as_pair(const uint8_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

// --- tensor-core kernel --------------------------------------------------------
// T: query and output type; F8: the caches hold E4M3 codes (M is then f16).
template <typename T, bool F8, int D, int HT>
__global__ void __launch_bounds__(kSparseThreads) sparse_mma_kernel(const SparseParams p) {
  using M = typename std::conditional<F8, __half, T>::type;
  constexpr int kElt = F8 ? 1 : 2;
  constexpr int kRow = D * kElt;                        // bytes of a token row
  constexpr int kNT = HT / 8;                           // head tiles of 8
  constexpr int kKLoads = kRow / 64;                    // 16-byte K loads of a lane and row
  constexpr int kVBytes = kRow / 8 < 16 ? 8 : 16;       // bytes of one V load
  constexpr int kVLoads = kRow / (8 * kVBytes);
  constexpr int kVWords = kVBytes / 4;                  // 32-bit words of one V load
  constexpr int kMT = F8 ? 2 * kVWords : kVWords;       // m16 tiles of one V load (2 elements a lane each)
  constexpr int kSteps = F8 ? 4 : 2;                    // k16 steps of one K load

  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  int64_t row = static_cast<int64_t>(blockIdx.x) / ctas;
  const int tile = static_cast<int>(row % p.num_head_tiles);
  row /= p.num_head_tiles;
  const int h = static_cast<int>(row % p.num_kv_heads), b = static_cast<int>(row / p.num_kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int heads = min(HT, p.group - tile * HT);
  const int head0 = h * p.group + tile * HT;

  extern __shared__ __align__(16) uint8_t raw[];
  Partial<D, HT>* part = reinterpret_cast<Partial<D, HT>*>(raw);

  int len = p.context_lens[b];
  if (len < 0 || len > p.max_tokens) {
    if (threadIdx.x == 0 && rank == 0 && h == 0 && tile == 0) atomicOr(p.err, kErrLen);
    len = len < 0 ? 0 : p.max_tokens;
  }
  const int32_t* list = p.selected + b * p.sel_sb + h * p.sel_sh;
  const int32_t* table = p.block_tables + b * p.bt_stride;

  // Q fragments: heads 8a + g, the elements that this lane's K loads bring
  uint32_t qf[kNT][kKLoads][kSteps][2];
#pragma unroll
  for (int a = 0; a < kNT; ++a)
#pragma unroll
    for (int i = 0; i < kKLoads; ++i)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t x = 0u;
          if (8 * a + g < heads) {
            constexpr int kPer = 16 / kElt;  // elements of one K load
            const int d = (4 * i + c) * kPer + 4 * s + 2 * e;
            const T* q = static_cast<const T*>(p.q) + b * p.q_sb + (head0 + 8 * a + g) * p.q_sh + d;
            if constexpr (std::is_same<T, M>::value) {
              const uint16_t lo = *reinterpret_cast<const uint16_t*>(q), hi = *reinterpret_cast<const uint16_t*>(q + 1);
              x = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
            } else {
              x = Mma<M>::pack(to_f32(q[0]), to_f32(q[1]));
            }
          }
          qf[a][i][s][e] = x;
        }

  float m[kNT], l[kNT];
  float o[kVLoads][kMT][kNT][4];
#pragma unroll
  for (int a = 0; a < kNT; ++a) m[a] = -INFINITY, l[a] = 0.f;
#pragma unroll
  for (int i = 0; i < kVLoads; ++i)
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int a = 0; a < kNT; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][a][e] = 0.f;

  const int64_t units = ((static_cast<int64_t>(p.top) << p.log2_bs) + 15) / 16;
  const int stride = ctas * kSparseWarps;
  for (int64_t u0 = rank * kSparseWarps + warp; u0 < units; u0 += 32LL * stride) {
    UnitLookup look;
    look.at[0] = look.at[1] = 0;
    look.live[0] = look.live[1] = 0;
    if (u0 + int64_t(lane) * stride < units)
      look.fetch(p, list, table, len, h, kRow, u0 + int64_t(lane) * stride);
    unsigned todo = __ballot_sync(kFullMask, look.live[0] + look.live[1] > 0);
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      UnitRows r;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        r.at[half] = __shfl_sync(kFullMask, look.at[half], from);
        r.live[half] = __shfl_sync(kFullMask, look.live[half], from);
      }
      // K rows g of both halves, V rows 2c, 2c+1 of both halves
      uint4 kx[2][kKLoads];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < kKLoads; ++i)
          kx[half][i] = g < r.live[half] ? load16(p.k_cache + r.at[half] + g * kRow + (4 * i + c) * 16)
                                         : make_uint4(0u, 0u, 0u, 0u);
      uint32_t vx[4][kVLoads][kVWords];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int half = n >> 1, tok = 2 * c + (n & 1);
        const uint8_t* src = p.v_cache + r.at[half] + tok * kRow + g * kVBytes;
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
          if constexpr (kVBytes == 16) {
            const uint4 x = tok < r.live[half] ? load16(src + i * 8 * kVBytes) : make_uint4(0u, 0u, 0u, 0u);
            vx[n][i][0] = x.x, vx[n][i][1] = x.y, vx[n][i][2] = x.z, vx[n][i][3] = x.w;
          } else {
            const uint2 x = tok < r.live[half] ? __ldg(reinterpret_cast<const uint2*>(src + i * 8 * kVBytes)) : make_uint2(0u, 0u);
            vx[n][i][0] = x.x, vx[n][i][1] = x.y;
          }
        }
      }
      // S = Q K^T
      float s[2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[half][e] = 0.f;
#pragma unroll
        for (int i = 0; i < kKLoads; ++i) {
          const uint32_t w[4] = {kx[half][i].x, kx[half][i].y, kx[half][i].z, kx[half][i].w};
#pragma unroll
          for (int t = 0; t < kSteps; ++t) {
            uint32_t bf[2];
            if constexpr (F8) {
              e4m3x4_to_f16x2x2(w[t], bf[0], bf[1]);
            } else {
              bf[0] = w[2 * t], bf[1] = w[2 * t + 1];
            }
            const uint32_t af[4] = {qf[0][i][t][0], kNT > 1 ? qf[kNT - 1][i][t][0] : 0u, qf[0][i][t][1],
                                    kNT > 1 ? qf[kNT - 1][i][t][1] : 0u};
            Mma<M>::run(s[half], af, bf);
          }
        }
      }
      // weights: head 8a + g, tokens 2c, 2c+1 of both halves
      uint32_t pf[kNT][2];
#pragma unroll
      for (int a = 0; a < kNT; ++a) {
        float x[4];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x[2 * half + e] = 2 * c + e < r.live[half] ? s[half][2 * a + e] * p.scale_log2 : -INFINITY;
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        const float mn = fmaxf(m[a], top);
        const bool moved = mn > m[a];
        if (__any_sync(kFullMask, moved)) {
          const float f = m[a] == -INFINITY ? 0.f : exp2f(m[a] - mn);
          l[a] *= f;
          m[a] = mn;
          const float f0 = __shfl_sync(kFullMask, f, 8 * c), f1 = __shfl_sync(kFullMask, f, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < kVLoads; ++i)
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
              o[i][t][a][0] *= f0, o[i][t][a][1] *= f1, o[i][t][a][2] *= f0, o[i][t][a][3] *= f1;
            }
        }
        const float base = m[a] == -INFINITY ? 0.f : m[a];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          pf[a][half] = Mma<M>::pack(ex2_approx(x[2 * half] - base), ex2_approx(x[2 * half + 1] - base));
          const M* w = reinterpret_cast<const M*>(&pf[a][half]);
          l[a] += to_f32(w[0]) + to_f32(w[1]);
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < kVLoads; ++i)
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
          if constexpr (F8) {
            uint32_t y[4][2];
#pragma unroll
            for (int n = 0; n < 4; ++n) e4m3x4_to_f16x2x2(vx[n][i][w], y[n][0], y[n][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t af[4] = {__byte_perm(y[0][e], y[1][e], 0x5410), __byte_perm(y[0][e], y[1][e], 0x7632),
                                      __byte_perm(y[2][e], y[3][e], 0x5410), __byte_perm(y[2][e], y[3][e], 0x7632)};
#pragma unroll
              for (int a = 0; a < kNT; ++a) Mma<M>::run(o[i][2 * w + e][a], af, pf[a]);
            }
          } else {
            const uint32_t af[4] = {
                __byte_perm(vx[0][i][w], vx[1][i][w], 0x5410), __byte_perm(vx[0][i][w], vx[1][i][w], 0x7632),
                __byte_perm(vx[2][i][w], vx[3][i][w], 0x5410), __byte_perm(vx[2][i][w], vx[3][i][w], 0x7632)};
#pragma unroll
            for (int a = 0; a < kNT; ++a) Mma<M>::run(o[i][w][a], af, pf[a]);
          }
        }
    }
  }

  // this warp's partial: heads 8a + 2c, 8a + 2c + 1, elements (8i + g) * 2 kMT + 2t, + 1
  Partial<D, HT>& mine = part[warp];
#pragma unroll
  for (int a = 0; a < kNT; ++a) {
    l[a] += __shfl_xor_sync(kFullMask, l[a], 1);
    l[a] += __shfl_xor_sync(kFullMask, l[a], 2);
    if (c == 0) {
      mine.m[8 * a + g] = m[a];
      mine.l[8 * a + g] = l[a];
    }
#pragma unroll
    for (int i = 0; i < kVLoads; ++i)
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        const int d = (8 * i + g) * 2 * kMT + 2 * t;
        *reinterpret_cast<float2*>(&mine.o[8 * a + 2 * c][d]) = make_float2(o[i][t][a][0], o[i][t][a][2]);
        *reinterpret_cast<float2*>(&mine.o[8 * a + 2 * c + 1][d]) = make_float2(o[i][t][a][1], o[i][t][a][3]);
      }
  }
  merge_and_store<T, D, HT>(p, cluster, part, static_cast<T*>(p.out) + b * p.o_sb + head0 * p.o_sh, heads);
}

// --- f32 kernel ------------------------------------------------------------------
// A warp takes 8 tokens (half a unit) at a time: lane (g, c) holds row g's
// chunks 4i + c for the products with the tile's 8 query heads (in shared
// memory), the four lanes of a row sum; then lane owns dims lane + 32i of V.
template <int D>
__global__ void __launch_bounds__(kSparseThreads) sparse_f32_kernel(const SparseParams p) {
  constexpr int HT = 8, kRow = D * 4, kChunks = D / 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  int64_t row = static_cast<int64_t>(blockIdx.x) / ctas;
  const int tile = static_cast<int>(row % p.num_head_tiles);
  row /= p.num_head_tiles;
  const int h = static_cast<int>(row % p.num_kv_heads), b = static_cast<int>(row / p.num_kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int heads = min(HT, p.group - tile * HT);
  const int head0 = h * p.group + tile * HT;

  extern __shared__ __align__(16) uint8_t raw[];
  Partial<D, HT>* part = reinterpret_cast<Partial<D, HT>*>(raw);
  float* qs = reinterpret_cast<float*>(part + kSparseWarps);             // [HT][D]
  float* ps = qs + HT * D + warp * 64;                                   // [8 tokens][HT] weights of this warp

  int len = p.context_lens[b];
  if (len < 0 || len > p.max_tokens) {
    if (threadIdx.x == 0 && rank == 0 && h == 0 && tile == 0) atomicOr(p.err, kErrLen);
    len = len < 0 ? 0 : p.max_tokens;
  }
  const int32_t* list = p.selected + b * p.sel_sb + h * p.sel_sh;
  const int32_t* table = p.block_tables + b * p.bt_stride;
  for (int i = threadIdx.x; i < HT * D; i += kSparseThreads) {
    const int a = i / D, d = i - a * D;
    qs[i] = a < heads ? static_cast<const float*>(p.q)[b * p.q_sb + (head0 + a) * p.q_sh + d] : 0.f;
  }
  __syncthreads();

  float m[HT], l[HT], o[HT][D / 32];
#pragma unroll
  for (int a = 0; a < HT; ++a) {
    m[a] = -INFINITY, l[a] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[a][i] = 0.f;
  }
  const int64_t units = ((static_cast<int64_t>(p.top) << p.log2_bs) + 15) / 16;
  const int stride = ctas * kSparseWarps;
  for (int64_t u0 = rank * kSparseWarps + warp; u0 < units; u0 += 32LL * stride) {
    UnitLookup look;
    look.at[0] = look.at[1] = 0;
    look.live[0] = look.live[1] = 0;
    if (u0 + int64_t(lane) * stride < units)
      look.fetch(p, list, table, len, h, kRow, u0 + int64_t(lane) * stride);
    unsigned todo = __ballot_sync(kFullMask, look.live[0] + look.live[1] > 0);
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t at = __shfl_sync(kFullMask, look.at[half], from);
        const int live = __shfl_sync(kFullMask, look.live[half], from);
        if (live == 0) continue;
        float4 kx[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          kx[i] = g < live ? __ldg(reinterpret_cast<const float4*>(p.k_cache + at + g * kRow + (4 * i + c) * 16))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        float s[HT];
#pragma unroll
        for (int a = 0; a < HT; ++a) {
          float x = 0.f;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(qs + a * D + (4 * i + c) * 4);
            x = fmaf(q.x, kx[i].x, fmaf(q.y, kx[i].y, fmaf(q.z, kx[i].z, fmaf(q.w, kx[i].w, x))));
          }
          x += __shfl_xor_sync(kFullMask, x, 1);
          x += __shfl_xor_sync(kFullMask, x, 2);
          s[a] = g < live ? x * p.scale_log2 : -INFINITY;
        }
#pragma unroll
        for (int a = 0; a < HT; ++a) {
          float top = s[a];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, k));
          const float mn = fmaxf(m[a], top);
          const float f = m[a] == -INFINITY ? 0.f : exp2f(m[a] - mn);
          m[a] = mn;
          l[a] *= f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) o[a][i] *= f;
          s[a] = exp2f(s[a] - (mn == -INFINITY ? 0.f : mn));
          if (c == 0) l[a] += s[a];
        }
        __syncwarp();
        if (c == 0) {
#pragma unroll
          for (int a = 0; a < HT; ++a) ps[g * HT + a] = s[a];
        }
        __syncwarp();
#pragma unroll 4
        for (int t = 0; t < 8; ++t) {
          if (t >= live) break;
          float w[HT];
#pragma unroll
          for (int a = 0; a < HT; a += 4) {
            const float4 x = *reinterpret_cast<const float4*>(ps + t * HT + a);
            w[a] = x.x, w[a + 1] = x.y, w[a + 2] = x.z, w[a + 3] = x.w;
          }
          const float* src = reinterpret_cast<const float*>(p.v_cache + at + t * kRow);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const float v = __ldg(src + lane + 32 * i);
#pragma unroll
            for (int a = 0; a < HT; ++a) o[a][i] = fmaf(w[a], v, o[a][i]);
          }
        }
      }
    }
  }
  Partial<D, HT>& mine = part[warp];
#pragma unroll
  for (int a = 0; a < HT; ++a) {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) l[a] += __shfl_xor_sync(kFullMask, l[a], k);
    if (lane == 0) {
      mine.m[a] = m[a];
      mine.l[a] = l[a];
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) mine.o[a][lane + 32 * i] = o[a][i];
  }
  merge_and_store<float, D, HT>(p, cluster, part, static_cast<float*>(p.out) + b * p.o_sb + head0 * p.o_sh, heads);
}

template <typename K>
int launch_cluster(K kernel, const SparseParams& p, size_t smem, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(p.num_seqs) * p.num_kv_heads * p.num_head_tiles * ctas));
  cfg.blockDim = dim3(kSparseThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, bool F8, int D, int HT>
int launch_mma(const SparseParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  constexpr size_t smem = sizeof(Partial<D, HT>) * kSparseWarps;
  const int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&sparse_mma_kernel<T, F8, D, HT>),
                                 static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_cluster(&sparse_mma_kernel<T, F8, D, HT>, p, smem, ctas, stream);
}

template <int D>
int launch_f32(const SparseParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  constexpr size_t smem = sizeof(Partial<D, 8>) * kSparseWarps + (8 * D + 64 * kSparseWarps) * sizeof(float);
  const int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&sparse_f32_kernel<D>), static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_cluster(&sparse_f32_kernel<D>, p, smem, ctas, stream);
}

template <typename T, bool F8>
int launch_dim(const SparseParams& p, int head_dim, int head_tile, int ctas, cudaStream_t stream) {
  if (head_dim == 64) return head_tile == 16 ? launch_mma<T, F8, 64, 16>(p, ctas, stream) : launch_mma<T, F8, 64, 8>(p, ctas, stream);
  if (head_dim == 128)
    return head_tile == 16 ? launch_mma<T, F8, 128, 16>(p, ctas, stream) : launch_mma<T, F8, 128, 8>(p, ctas, stream);
  if (head_dim == 256) return launch_mma<T, F8, 256, 8>(p, ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

int launch_sparse_decode(int dtype, bool kv_fp8, int head_dim, SparseParams p, int num_sms, cudaStream_t stream) {
  // two tiles of 8 query heads share the K/V fragments where registers allow
  const int head_tile = dtype != 0 && p.group > 8 && head_dim <= 128 ? 16 : 8;
  p.num_head_tiles = (p.group + head_tile - 1) / head_tile;
  // CTAs of a list: enough that all lists together give every SM four, but no
  // warp under one unit of 16 tokens
  const int64_t rows = int64_t(p.num_seqs) * p.num_kv_heads * p.num_head_tiles;
  const int64_t units = ((int64_t(p.top) << p.log2_bs) + 15) / 16;
  int ctas = 1;
  while (ctas < kMaxSparseCluster && rows * ctas < int64_t(num_sms) * 4 && units >= 2 * ctas * kSparseWarps) ctas *= 2;
  int e = cudaErrorInvalidValue;
  if (dtype == 0 && !kv_fp8) {
    e = head_dim == 64 ? launch_f32<64>(p, ctas, stream) : head_dim == 128 ? launch_f32<128>(p, ctas, stream)
                                                           : launch_f32<256>(p, ctas, stream);
  } else if (dtype == 1) {
    e = kv_fp8 ? launch_dim<__half, true>(p, head_dim, head_tile, ctas, stream)
               : launch_dim<__half, false>(p, head_dim, head_tile, ctas, stream);
  } else if (dtype == 2) {
    e = kv_fp8 ? launch_dim<__nv_bfloat16, true>(p, head_dim, head_tile, ctas, stream)
               : launch_dim<__nv_bfloat16, false>(p, head_dim, head_tile, ctas, stream);
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
