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
// The scores are summed in binary32, each with an error of at most
//   E = c u sum_i |w_i b_i|,  u = 2^-24, c = G + 44
// (G - 1 roundings in w, a chain of 32 fused products, at most 5 sums across
// lanes, some spare), so blocks whose scores differ by more than 2 E are in
// their true order.  The choice between the few blocks that lie within 2 E of
// the border is made from their scores in binary64, where the products of
// 16-bit elements and their sums are exact for all but extreme exponents: the
// selection is the definition's, whatever the order of the sums.
//
// Work split: a cluster of up to 8 CTAs per (sequence, kv head), each with a
// contiguous share of the blocks, so a long row is on many SMs and the
// selection still needs neither a second launch nor a workspace.  D/16 lanes
// read a block's 2D bounds, 16 bytes a lane and load, with their 32 weights in
// registers.  The cluster then finds the border with one 1024-bin histogram
// of the scores between their extremes, settles the border bin in binary64,
// and writes the chosen blocks in ascending order.  Bound: memory, the bounds
// are read once.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

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
constexpr int kWindow = 512;          // border blocks ranked in one CTA; more go through the digit passes
constexpr int kMaxCluster = 8;

struct SelectShared {
  float stat[kMaxCluster][4];         // per CTA: smallest score, largest, bound on the sum of magnitudes, flag
  uint32_t hist[kBins];
  uint32_t digits[2][256];
  uint32_t warp_sum[kSelectWarps];
  float warp_stat[kSelectWarps][4];
  unsigned long long win_key[kWindow];
  int win_at[kWindow];
  int win_count;                      // rank 0: border blocks of the cluster
  int sure_count;                     // rank 0: blocks above the border
  int my_sure, my_win;
  unsigned long long cut_key;         // last border block that is kept: its key and index
  int cut_at;
  int found_bin, found_above, found_count;
  int picked[kMaxCluster];            // per CTA, for the offsets of the output
};

// Doubles (without NaN) to integers of the same order.
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));  // -0 is 0
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// 16 bytes of bounds as floats.
template <typename T>
struct Bounds16;
template <>
struct Bounds16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void open(const uint4& x, float (&f)[4], float& most) {
    f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y), f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(f[i]));
  }
};
template <>
struct Bounds16<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void open(const uint4& x, float (&f)[8], float& most) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __half2 m = __float2half2_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
      const float2 v = __half22float2(h);
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
      m = __hmax2(m, __habs2(h));
    }
    most = fmaxf(most, fmaxf(__low2float(m), __high2float(m)));
  }
};
template <>
struct Bounds16<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void open(const uint4& x, float (&f)[8], float& most) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    }
    most = fmaxf(most, fmaxf(__low2float(m), __high2float(m)));
  }
};
template <>
struct Bounds16<uint8_t> {
  static constexpr int kN = 16;
  static __device__ __forceinline__ void open(const uint4& x, float (&f)[16], float& most) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __half2 m = __float2half2_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y[2];
      e4m3x4_to_f16x2x2(w[i], y[0], y[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2 h = *reinterpret_cast<const __half2*>(&y[e]);
        const float2 v = __half22float2(h);
        f[4 * i + 2 * e] = v.x, f[4 * i + 2 * e + 1] = v.y;
        m = __hmax2(m, __habs2(h));
      }
    }
    most = fmaxf(most, fmaxf(__low2float(m), __high2float(m)));
  }
};

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

template <typename T, typename B, int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t row = static_cast<int64_t>(blockIdx.x) / ctas;
  const int b = static_cast<int>(row / p.num_kv_heads), h = static_cast<int>(row - int64_t(b) * p.num_kv_heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.selected + b * p.sel_sb + h * p.sel_sh;

  int len = p.context_lens[b];
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

  extern __shared__ __align__(16) uint8_t raw[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(raw);
  double* w64 = reinterpret_cast<double*>(raw + ((sizeof(SelectShared) + 15) / 16) * 16);  // [2D]: down, up
  float* w32 = reinterpret_cast<float*>(w64 + 2 * D);
  unsigned long long* key = reinterpret_cast<unsigned long long*>(w32 + 2 * D);            // [share]
  float* score = reinterpret_cast<float*>(key + p.share);                                  // [share]

  for (int i = tid; i < kBins; i += kSelectThreads) sh.hist[i] = 0;
  if (tid == 0) sh.win_count = sh.sure_count = sh.my_sure = sh.my_win = 0;
  const T* q = static_cast<const T*>(p.q) + b * p.q_sb + int64_t(h) * p.group * p.q_sh;
  for (int d = tid; d < D; d += kSelectThreads) {
    double up = 0.0, down = 0.0;
    float up32 = 0.f, down32 = 0.f;
    for (int g = 0; g < p.group; ++g) {
      const float x = to_f32(q[g * p.q_sh + d]);
      // a NaN goes into both sums
      const float a = x < 0.f ? 0.f : x, c = x > 0.f ? 0.f : x;
      up += a, down += c;
      up32 += a, down32 += c;
    }
    w64[d] = down, w64[D + d] = up;
    w32[d] = down32, w32[D + d] = up32;
  }
  auto started = cluster.barrier_arrive();  // waited for before the first access to a peer's shared memory
  __syncthreads();

  // --- scores of this CTA's share of the candidates sink .. n - recent - 1 ---
  const int cands = n - p.sink - p.recent;
  const int lo = static_cast<int>(int64_t(cands) * rank / ctas), hi = static_cast<int>(int64_t(cands) * (rank + 1) / ctas);
  const int mine = hi - lo, first = p.sink + lo;
  const int32_t* table = p.block_tables + b * p.bt_stride;
  constexpr int kLanes = D / 16;                       // lanes of one block
  constexpr int kPer = 32 / kLanes;                    // blocks of one step
  constexpr int kN = Bounds16<B>::kN, kLoads = 32 / kN;
  const int gl = lane % kLanes, gi = lane / kLanes;
  float w[32];
  float wsum = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      w[i * kN + e] = w32[(gl + kLanes * i) * kN + e];
      wsum += fabsf(w[i * kN + e]);
    }
  const int64_t head_bytes = 2 * D * sizeof(B);
  float smin = INFINITY, smax = -INFINITY, most = 0.f;
  bool odd = false;
  for (int j0 = warp * 32; j0 < mine; j0 += kSelectWarps * 32) {
    int id = 0;
    if (j0 + lane < mine) {
      id = table[first + j0 + lane];
      if (id < 0 || id >= p.num_blocks) {
        atomicOr(p.err, kErrBlock);
        id = 0;
      }
    }
    const int count = min(32, mine - j0);
#pragma unroll 2
    for (int s = 0; s < count; s += kPer) {
      const int jj = s + gi;
      const int phys = __shfl_sync(kFullMask, id, jj & 31);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.bounds + (int64_t(phys) * p.num_kv_heads + h) * head_bytes) + gl;
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = jj < count ? __ldg(src + kLanes * i) : make_uint4(0u, 0u, 0u, 0u);
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float f[kN];
        Bounds16<B>::open(x[i], f, most);
#pragma unroll
        for (int e = 0; e < kN; ++e) acc = fmaf(w[i * kN + e], f[e], acc);
      }
#pragma unroll
      for (int m = 1; m < kLanes; m <<= 1) acc += __shfl_xor_sync(kFullMask, acc, m);
      if (gl == 0 && jj < count) {
        score[j0 + jj] = acc;
        odd |= !(fabsf(acc) < INFINITY);
        smin = fminf(smin, acc);
        smax = fmaxf(smax, acc);
      }
    }
  }
  {  // sum_i |w_i b_ji| <= sum over lanes of (its largest |b|) (its sum of |w|), for every j
    float mag = most * wsum;
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) mag += __shfl_xor_sync(kFullMask, mag, m);
#pragma unroll
    for (int m = kLanes; m < 32; m <<= 1) mag = fmaxf(mag, __shfl_xor_sync(kFullMask, mag, m));
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      smin = fminf(smin, __shfl_xor_sync(kFullMask, smin, m));
      smax = fmaxf(smax, __shfl_xor_sync(kFullMask, smax, m));
    }
    odd = __any_sync(kFullMask, odd || !(mag < 1e37f));
    if (lane == 0) {
      sh.warp_stat[warp][0] = smin, sh.warp_stat[warp][1] = smax, sh.warp_stat[warp][2] = mag;
      sh.warp_stat[warp][3] = odd ? 1.f : 0.f;
    }
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (tid < ctas) {  // this CTA's extremes, to every CTA of the cluster
    float a = INFINITY, c = -INFINITY, m = 0.f, o = 0.f;
#pragma unroll
    for (int i = 0; i < kSelectWarps; ++i) {
      a = fminf(a, sh.warp_stat[i][0]), c = fmaxf(c, sh.warp_stat[i][1]);
      m = fmaxf(m, sh.warp_stat[i][2]), o = fmaxf(o, sh.warp_stat[i][3]);
    }
    float* dst = cluster.map_shared_rank(&sh.stat[rank][0], tid);
    dst[0] = a, dst[1] = c, dst[2] = m, dst[3] = o;
  }
  cluster.sync();
  smin = INFINITY, smax = -INFINITY;
  float mag = 0.f, flag = 0.f;
  for (int r = 0; r < ctas; ++r) {
    smin = fminf(smin, sh.stat[r][0]), smax = fmaxf(smax, sh.stat[r][1]);
    mag = fmaxf(mag, sh.stat[r][2]), flag = fmaxf(flag, sh.stat[r][3]);
  }
  // two errors of a score; 1e-37 covers products below the smallest binary32 number
  const float err2 = 2.f * (static_cast<float>(p.group + 44) * 5.9604645e-8f * 1.01f * mag + 1e-37f);
  // scores that overflowed, infinite or NaN bounds: every candidate is settled in binary64
  const bool all = flag != 0.f;
  const float per = smax > smin ? static_cast<float>(kBins) / (smax - smin) : 0.f;
  auto bin = [&](float x) { return static_cast<int>(fminf(fmaxf((x - smin) * per, 0.f), kBins - 1.f)); };

  // --- the bin that holds the border ---
  int border = 0;
  if (!all) {
    for (int j = tid; j < mine; j += kSelectThreads) atomicAdd(&sh.hist[bin(score[j])], 1u);
    cluster.sync();
    uint32_t c[4] = {0, 0, 0, 0};
    const int at = kBins - 4 - 4 * tid;  // thread 0 holds the highest bins
    for (int r = 0; r < ctas; ++r) {
      const uint4 x = *cluster.map_shared_rank(reinterpret_cast<const uint4*>(&sh.hist[at]), r);
      c[0] += x.w, c[1] += x.z, c[2] += x.y, c[3] += x.x;
    }
    uint32_t total;
    uint32_t before = block_scan(sh, c[0] + c[1] + c[2] + c[3], &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < static_cast<uint32_t>(need) && before + c[i] >= static_cast<uint32_t>(need)) sh.found_bin = at + 3 - i;
      before += c[i];
    }
    __syncthreads();
    border = sh.found_bin;
  }
  // 2: above the border for certain, 1: to be settled, 0: below for certain
  auto place = [&](float s) {
    if (all) return 1;
    return bin(s - err2) > border ? 2 : bin(s + err2) < border ? 0 : 1;
  };

  // --- border blocks in binary64, a warp each ---
  SelectShared* head = cluster.map_shared_rank(&sh, 0);
  int sure = 0;
  for (int j0 = warp * 32; j0 < mine; j0 += kSelectWarps * 32) {
    const int what = j0 + lane < mine ? place(score[j0 + lane]) : 0;
    sure += __popc(__ballot_sync(kFullMask, what == 2));
    unsigned todo = __ballot_sync(kFullMask, what == 1);
    while (todo) {
      const int j = j0 + __ffs(todo) - 1;
      todo &= todo - 1;
      int phys = table[first + j];
      if (phys < 0 || phys >= p.num_blocks) phys = 0;
      const uint8_t* src = p.bounds + (int64_t(phys) * p.num_kv_heads + h) * head_bytes;
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < 2 * D / 32; ++i) {
        const int e = lane + 32 * i;
        s = fma(w64[e], static_cast<double>(element(src, e, B())), s);
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(kFullMask, s, m);
      if (lane == 0) {
        const unsigned long long k = ordered(s != s ? static_cast<double>(INFINITY) : s);
        key[j] = k;
        const int at = atomicAdd(&head->win_count, 1);
        if (at < kWindow) {
          head->win_key[at] = k;
          head->win_at[at] = first + j;
        }
      }
    }
  }
  if (lane == 0 && sure > 0) atomicAdd(&head->sure_count, sure);
  cluster.sync();
  const int window = head->win_count;
  int left = need - head->sure_count;  // border blocks to keep: 1 .. window
  if (window <= kWindow) {
    if (rank == 0) {
      for (int i = tid; i < window; i += kSelectThreads) {
        const unsigned long long k = sh.win_key[i];
        const int at = sh.win_at[i];
        int better = 0;
        for (int o = 0; o < window; ++o) better += sh.win_key[o] > k || (sh.win_key[o] == k && sh.win_at[o] < at);
        if (better == left - 1) {
          for (int r = 0; r < ctas; ++r) {
            SelectShared* peer = cluster.map_shared_rank(&sh, r);
            peer->cut_key = k;
            peer->cut_at = at;
          }
        }
      }
    }
    cluster.sync();
  } else {
    // the digits of (key, complement of the index), 8 bits at a time from the top
    unsigned long long want = 0;
    uint32_t want_at = 0;
    for (int pass = 0; pass < 12; ++pass) {
      uint32_t* dig = sh.digits[pass & 1];
      dig[tid] = 0;
      __syncthreads();
      const int shift = pass < 8 ? 56 - 8 * pass : 24 - 8 * (pass - 8);
      for (int j = tid; j < mine; j += kSelectThreads) {
        if (place(score[j]) != 1) continue;
        const unsigned long long k = key[j];
        const uint32_t a = ~static_cast<uint32_t>(first + j);
        bool in;
        uint32_t d;
        if (pass < 8) {
          in = pass == 0 || (k >> (shift + 8)) == (want >> (shift + 8));
          d = static_cast<uint32_t>(k >> shift) & 255u;
        } else {
          in = k == want && (pass == 8 || (a >> (shift + 8)) == (want_at >> (shift + 8)));
          d = (a >> shift) & 255u;
        }
        if (in) atomicAdd(&dig[d], 1u);
      }
      cluster.sync();
      uint32_t c = 0, total;
      const int at = 255 - tid;
      for (int r = 0; r < ctas; ++r) c += *cluster.map_shared_rank(&dig[at], r);
      const uint32_t before = block_scan(sh, c, &total);
      if (before < static_cast<uint32_t>(left) && before + c >= static_cast<uint32_t>(left)) {
        sh.found_bin = at;
        sh.found_above = static_cast<int>(before);
      }
      __syncthreads();
      left -= sh.found_above;
      if (pass < 8)
        want |= static_cast<unsigned long long>(sh.found_bin) << shift;
      else
        want_at |= static_cast<uint32_t>(sh.found_bin) << shift;
    }
    if (tid == 0) {
      sh.cut_key = want;
      sh.cut_at = static_cast<int>(~want_at);
    }
    __syncthreads();
  }
  const unsigned long long cut_key = sh.cut_key;
  const int cut_at = sh.cut_at;
  auto kept = [&](int j) {
    const int what = place(score[j]);
    return what == 2 || (what == 1 && (key[j] > cut_key || (key[j] == cut_key && first + j <= cut_at)));
  };

  // --- the chosen blocks, ascending ---
  int count = 0;
  for (int j = tid; j < mine; j += kSelectThreads) count += kept(j);
  uint32_t total;
  block_scan(sh, static_cast<uint32_t>(count), &total);
  if (tid < ctas) *cluster.map_shared_rank(&sh.picked[rank], tid) = static_cast<int>(total);
  cluster.sync();  // the last access to another CTA's shared memory
  int base = p.sink;
  for (int r = 0; r < rank; ++r) base += sh.picked[r];
  for (int j0 = 0; j0 < mine; j0 += kSelectThreads) {
    const int j = j0 + tid;
    const bool in = j < mine && kept(j);
    uint32_t all_in;
    const uint32_t before = block_scan(sh, in, &all_in);
    if (in && base + static_cast<int>(before) < p.top) out[base + before] = first + j;
    base += static_cast<int>(all_in);
  }
  for (int i = rank * kSelectThreads + tid; i < p.sink + p.recent; i += ctas * kSelectThreads) {
    if (i < p.sink)
      out[i] = i;
    else
      out[p.top - p.recent + (i - p.sink)] = n - p.recent + (i - p.sink);
  }
}

size_t select_smem(int head_dim, int share) {
  return (sizeof(SelectShared) + 15) / 16 * 16 + size_t(2 * head_dim) * 12 + size_t(share) * 12;
}

template <typename T, typename B, int D>
int launch_one(const SelectParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  const size_t smem = select_smem(D, p.share);
  int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&select_kernel<T, B, D>), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(p.num_seqs) * p.num_kv_heads * ctas));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<T, B, D>, p);
}

template <typename T, typename B>
int launch_dim(const SelectParams& p, int head_dim, int ctas, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_one<T, B, 64>(p, ctas, stream);
    case 128: return launch_one<T, B, 128>(p, ctas, stream);
    case 256: return launch_one<T, B, 256>(p, ctas, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Most blocks a table row may have: the largest cluster's shares have to fit
// its CTAs' shared memory.
int select_max_blocks(int head_dim) {
  const size_t room = 200 * 1024 - select_smem(head_dim, 0);
  return static_cast<int>(room / 12) * kMaxCluster;
}

int launch_select(int dtype, int bounds_dtype, int head_dim, SelectParams p, int max_blocks, int num_sms,
                  cudaStream_t stream) {
  // CTAs of a row: enough that all rows together give every SM four, but no
  // CTA under 64 blocks; and as many as the scores' share needs
  const int64_t rows = int64_t(p.num_seqs) * p.num_kv_heads;
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas < int64_t(num_sms) * 4 && max_blocks / (2 * ctas) >= 64) ctas *= 2;
  while (ctas < kMaxCluster && select_smem(head_dim, (max_blocks + ctas - 1) / ctas) > 100 * 1024) ctas *= 2;
  p.share = ((max_blocks + ctas - 1) / ctas + 1) / 2 * 2;
  int e = cudaErrorInvalidValue;
  if (dtype == 0 && bounds_dtype == 0) e = launch_dim<float, float>(p, head_dim, ctas, stream);
  if (dtype == 1 && bounds_dtype == 1) e = launch_dim<__half, __half>(p, head_dim, ctas, stream);
  if (dtype == 2 && bounds_dtype == 2) e = launch_dim<__nv_bfloat16, __nv_bfloat16>(p, head_dim, ctas, stream);
  if (dtype == 1 && bounds_dtype == 5) e = launch_dim<__half, uint8_t>(p, head_dim, ctas, stream);
  if (dtype == 2 && bounds_dtype == 5) e = launch_dim<__nv_bfloat16, uint8_t>(p, head_dim, ctas, stream);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
