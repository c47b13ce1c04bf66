// append_block_scaled.cu -- the KV append into E4M3 caches that have a scale for
// each block and kv head, found from what is stored.
//
// Mathematics: for a block that gets new tokens, a head, and K or V, with m the
// largest finite magnitude of the new elements,
//   need = 2^e, the least e in [-40, 40] with m <= 448 2^e,
//   scale = need where the block's first token is new, else max(need, old scale),
//   code = E4M3(x * (1 / scale)),
// and where the scale has risen, the block's earlier codes are stored again times
// old / scale.  A power of two keeps codes exact through a rise, but for those that
// fall below 2^-6; a floating-point code gains nothing from a closer scale.
//
// Work split: a warp (block_size * head_dim up to 4096 elements, and always for
// one token a sequence) or a CTA of 2 or 4 warps per (sequence's block, head, K or
// V).  A warp holds 2048 elements in registers, 16 bytes a lane and load, all in
// flight together; the maximum is taken in the elements' own type, met by shuffles
// (and in shared memory), and the same registers are then stored as codes.  What is
// more is read twice, the second time from L2.  Which blocks there are is found on the
// device from the packed starts; while a unit's elements are on their way the warp
// looks up its next one.  Every CTA also looks at all the packed starts before it
// writes, so that nothing is written where they decrease (16 chunks 17.9 us with and
// 18.1 without; one token each of 1024 sequences, 4 heads of 128, 13.0 and 12.6, of
// 16384, 1 head of 64, 48.2 and 45.6).
//
// Bound: memory, each element is read once and its code written.  16 chunks of up to
// 1024 tokens, 8 heads of 128, bf16, block_size 16 (86 MB): 17.9 us, 0.72 of the
// measured copy rate, the rest launch, first look-ups and the last round of units; 256
// sequences with a token each 3.1 us, 8 2.4, both latency.  Warps a unit, measured with
// 16 chunks of 1024 in blocks of 4096 elements: one 19.8 us, two 19.8, four 27.6; of
// 8192: one 23.9, two 21.9, four 21.2; of 16384: one 24.9, two 22.5, four 22.4.
#include "common.cuh"
#include "launch.h"

namespace wllm {
namespace {

constexpr int kAppendWarps = 4;        // of a CTA whose warps work by themselves
constexpr int kWarpElements = 2048;    // that a warp holds

// 16 bytes of elements: their largest magnitude so far (bits of f32 or packed
// pairs; NaN never wins), and their values.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) {
    return __float_as_uint(fmaxf(__uint_as_float(m), fabsf(__uint_as_float(w))));
  }
  static __device__ __forceinline__ float widest(uint32_t m) { return __uint_as_float(m); }
  static __device__ __forceinline__ uint32_t finite(uint32_t w) { return (w & 0x7fffffffu) < 0x7f800000u ? w : 0u; }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
    return r;
  }
  static __device__ __forceinline__ float widest(uint32_t m) {
    const __half2 h = *reinterpret_cast<const __half2*>(&m);
    return fmaxf(__low2float(h), __high2float(h));
  }
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    return ((w & 0x7fffu) < 0x7c00u ? w & 0xffffu : 0u) | ((w & 0x7fff0000u) < 0x7c000000u ? w & 0xffff0000u : 0u);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
    return r;
  }
  static __device__ __forceinline__ float widest(uint32_t m) {
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    return ((w & 0x7fffu) < 0x7f80u ? w & 0xffffu : 0u) | ((w & 0x7fff0000u) < 0x7f800000u ? w & 0xffff0000u : 0u);
  }
};

// Codes of 16 bytes of elements times `inv`.
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint4& x, float inv, float) {
  const uint32_t c = f32x2_to_e4m3x2(__uint_as_float(x.y) * inv, __uint_as_float(x.x) * inv) |
                     f32x2_to_e4m3x2(__uint_as_float(x.w) * inv, __uint_as_float(x.z) * inv) << 16;
  *reinterpret_cast<uint32_t*>(dst) = c;
}
__device__ __forceinline__ float2 pair(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ float2 pair(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint4& x, float inv, T) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = pair(w[i], T());
    c[i] = f32x2_to_e4m3x2(f.y * inv, f.x * inv);
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// 2^e for the least e in the scales' range with m <= 448 2^e; 448 = 1.75 2^8.
__device__ __forceinline__ float scale_for(float m) {
  const int e = static_cast<int>((__float_as_uint(m) + 0x1fffffu) >> 23) - 127 - 8;
  return __uint_as_float(static_cast<uint32_t>(127 + min(max(e, kLeastScaleExp), kMostScaleExp)) << 23);
}

// Four codes times f, rounded again.
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(codes, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return f32x2_to_e4m3x2(a.y * f, a.x * f) | f32x2_to_e4m3x2(b.y * f, b.x * f) << 16;
}

constexpr int append_threads(int wpu) { return 32 * (wpu == 1 ? kAppendWarps : wpu); }
// that run at once; the registers of 20 warps (96 a thread) are enough for one warp a unit
constexpr int append_warps_per_sm(int wpu) { return wpu == 1 ? 20 : 16; }

// Sequence b, whose new tokens are packed rows r = qsl[b] - qsl[0] .. qsl[b+1] -
// qsl[0], owns the unit numbers from floor(r / bs) + 2 b on: n tokens touch at most
// floor(n / bs) + 2 blocks, which is no more than the distance to the next
// sequence's first unit.
// WPU: warps of a unit (1: a CTA's warps have units of their own).
template <typename T, int D, int WPU>
__global__ void __launch_bounds__(append_threads(WPU), append_warps_per_sm(WPU) * 32 / append_threads(WPU))
    append_block_scaled_kernel(const ScaledAppendParams p) {
  constexpr int kVecs = D / Vec<T>::kN;                          // 16-byte vectors of a row
  constexpr int kLoads = kWarpElements / Vec<T>::kN / 32;        // a lane's
  constexpr int kRows = kWarpElements / D;                       // rows that a warp holds
  constexpr int kUnitsPerCta = WPU == 1 ? kAppendWarps : 1;
  __shared__ float met[2][4];
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = WPU == 1 ? 0 : warp;  // of the unit
  const bool speaker = lane == 0 && part == 0;
  const int bs = 1 << p.log2_bs;
  int64_t slots = p.num_seqs;  // of every head, K and V
  int row_first = 0;
  bool falls = false;  // a start that decreases
  if (p.query_start_loc != nullptr) {
    constexpr int kThreads = 32 * (WPU == 1 ? kAppendWarps : WPU), kStarts = 4;  // of a thread, asked for together
    for (int i0 = threadIdx.x; i0 < p.num_seqs; i0 += kStarts * kThreads) {
      int here[kStarts], behind[kStarts];
#pragma unroll
      for (int k = 0; k < kStarts; ++k) {
        const int i = min(i0 + k * kThreads, p.num_seqs - 1);
        here[k] = p.query_start_loc[i], behind[k] = p.query_start_loc[i + 1];
      }
#pragma unroll
      for (int k = 0; k < kStarts; ++k) falls |= behind[k] < here[k];
    }
    row_first = p.query_start_loc[0];
    const int64_t total = int64_t(p.query_start_loc[p.num_seqs]) - row_first;
    if (total < 0 || total > p.num_tokens || total > int64_t(p.num_seqs) * p.max_tokens) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrLen);
      return;
    }
    slots = (total >> p.log2_bs) + 2 * int64_t(p.num_seqs);
  }
  const int sides = 2 * p.num_kv_heads;
  const int64_t units = slots * sides;
  const int64_t first = int64_t(blockIdx.x) * kUnitsPerCta + (WPU == 1 ? warp : 0);
  const int64_t stride = int64_t(gridDim.x) * kUnitsPerCta;
  struct Unit {
    const T* src;    // first new element
    uint8_t* codes;  // of the block and head
    float* scale_at;
    float held;      // the scale so far, where the block has earlier tokens
    int off, count;  // first new token in the block; new tokens in it (0: nothing to do)
    int kv;
  };
  const auto locate = [&](int64_t unit, Unit& u) {
    const int slot = static_cast<int>(unit / sides), side = static_cast<int>(unit - int64_t(slot) * sides);
    const int h = side >> 1;
    u.kv = side & 1;
    u.count = 0;
    int b = slot, n = 1, j = 0, row = slot;
    if (p.query_start_loc != nullptr) {
      // largest b whose first unit is not behind this one: 32 probes at a time
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool before = at <= hi && ((p.query_start_loc[at] - row_first) >> p.log2_bs) + 2 * at <= slot;
        const int k = __popc(__ballot_sync(kFullMask, before));
        hi = min(hi, lo + (k + 1) * step - 1);
        lo += k * step;
      }
      b = lo;
      row = p.query_start_loc[b];
      n = p.query_start_loc[b + 1] - row;
      j = slot - (((row - row_first) >> p.log2_bs) + 2 * b);
    }
    const int len = p.context_lens[b];
    if (p.query_start_loc == nullptr && len == 0) return;  // an empty sequence of the one-token form has no new token
    if (n < 0 || n > len || len > p.max_tokens || j < 0 || row < 0 || n > p.num_tokens - row) {
      if (speaker) atomicOr(p.err, kErrLen);
      return;
    }
    if (n == 0) return;
    const int begin = len - n;                        // position of the first new token
    const int at = (begin >> p.log2_bs) + j;          // this unit's block of the sequence
    if (at > (len - 1) >> p.log2_bs) return;
    const int id = p.block_tables[b * p.bt_stride + at];
    if (id < 0 || id >= p.num_blocks) {
      if (speaker) atomicOr(p.err, kErrBlock);
      return;
    }
    u.off = max(0, begin - (at << p.log2_bs));
    u.count = min(bs, len - (at << p.log2_bs)) - u.off;
    u.src = static_cast<const T*>(p.src[u.kv]) + (row + ((at << p.log2_bs) + u.off - begin)) * p.src_st[u.kv] + h * p.src_sh[u.kv];
    const int64_t run = int64_t(id) * p.num_kv_heads + h;
    u.codes = p.cache[u.kv] + run * bs * D;
    u.scale_at = p.scales[u.kv] + run;
    u.held = 0.f;
    if (u.off > 0) u.held = *u.scale_at;
  };

  int turn = 0;
  Unit u, next{};
  if (first < units) locate(first, next);
  // every CTA looks at all the starts, so that none writes where they are not what they have to be
  if (p.query_start_loc != nullptr && __syncthreads_or(falls)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrLen);
    return;
  }
  for (int64_t unit = first; unit < units; unit += stride) {
    u = next;
    // the new elements: into registers, or through them where there are more
    const int64_t st = p.src_st[u.kv];
    uint4 x[kLoads];
    uint32_t most = 0u;
    const auto row_of = [&](int i) { return (i * 32 + lane) / kVecs; };  // of load i, among the rows that a warp holds
    auto load = [&](int r0) {
      const T* base = u.src + (r0 + lane / kVecs) * st + (lane % kVecs) * Vec<T>::kN;
      const auto piece = [&](int i) { return base + i * 32 / kVecs * st + i * 32 % kVecs * Vec<T>::kN; };
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.vec) {  // a loop for each kind of load: a choice inside it would wait for every load
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (r0 + row_of(i) < u.count) x[i] = *reinterpret_cast<const uint4*>(piece(i));
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (r0 + row_of(i) < u.count) {
            const T* from = piece(i);
            T* e = reinterpret_cast<T*>(&x[i]);
#pragma unroll
            for (int k = 0; k < Vec<T>::kN; ++k) e[k] = from[k];
          }
      }
    };
    load(part * kRows);
    // the next unit is looked up while these are on their way
    next.count = 0;
    if (unit + stride < units) locate(unit + stride, next);
    if (u.count == 0) continue;
    auto measure = [&](bool finite_only) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) most = Vec<T>::most(most, finite_only ? Vec<T>::finite(w[e]) : w[e]);
      }
    };
    const bool once = u.count <= kRows * WPU;
    auto largest = [&](bool finite_only) {
      most = 0u;
      for (int r0 = part * kRows; r0 < u.count; r0 += kRows * WPU) {
        if (!once && (finite_only || r0 != part * kRows)) load(r0);
        measure(finite_only);
      }
      float m = Vec<T>::widest(most);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, d));
      if constexpr (WPU > 1) {
        if (lane == 0) met[turn & 1][warp] = m;
        __syncthreads();  // the room of the turn before last is free: every warp has passed the last turn's
#pragma unroll
        for (int w = 0; w < WPU; ++w) m = fmaxf(m, met[turn & 1][w]);
        ++turn;
      }
      return m;
    };
    float m = largest(false);
    if (m == INFINITY) m = largest(true);  // infinities do not count (the same for all the unit's warps)
    const float need = scale_for(m), old = scale_in_range(u.held);
    const float scale = u.off > 0 ? fmaxf(need, old) : need;
    const float inv = 1.f / scale;
    for (int r0 = part * kRows; r0 < u.count; r0 += kRows * WPU) {
      if (!once) load(r0);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int v = i * 32 + lane, r = r0 + row_of(i);
        if (r < u.count) store_codes(u.codes + (u.off + r) * D + (v % kVecs) * Vec<T>::kN, x[i], inv, T());
      }
    }
    if (u.off > 0 && scale > old) {
      const float f = old * inv;
      uint4* again = reinterpret_cast<uint4*>(u.codes);
      for (int v = part * 32 + lane; v < u.off * (D / 16); v += 32 * WPU) {
        const uint4 c = again[v];
        again[v] = make_uint4(rescaled(c.x, f), rescaled(c.y, f), rescaled(c.z, f), rescaled(c.w, f));
      }
    }
    if (speaker) *u.scale_at = scale;
  }
}

template <typename T, int D, int WPU>
int launch_one(const ScaledAppendParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kThreads = append_threads(WPU), kUnits = WPU == 1 ? kAppendWarps : 1;
  // packed: how many blocks the chunks touch is on the device; as many CTAs as that can be, or as run at once
  const int64_t slots = p.query_start_loc == nullptr ? p.num_seqs : (int64_t(p.num_tokens) >> p.log2_bs) + 2 * int64_t(p.num_seqs);
  const int64_t units = slots * 2 * p.num_kv_heads, resident = int64_t(num_sms) * (append_warps_per_sm(WPU) * 32 / kThreads);
  int64_t ctas = (units + kUnits - 1) / kUnits;
  if (ctas > resident) ctas = resident;
  return launch_dependent(&append_block_scaled_kernel<T, D, WPU>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, 0,
                          stream, p);
}

template <typename T, int D>
int launch_dim(const ScaledAppendParams& p, int num_sms, cudaStream_t stream) {
  const int warps = p.query_start_loc == nullptr ? 1 : (D << p.log2_bs) / (2 * kWarpElements);
  if (warps <= 1) return launch_one<T, D, 1>(p, num_sms, stream);
  if (warps == 2) return launch_one<T, D, 2>(p, num_sms, stream);
  return launch_one<T, D, 4>(p, num_sms, stream);
}

template <typename T>
int launch_type(const ScaledAppendParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_dim<T, 64>(p, num_sms, stream);
    case 128: return launch_dim<T, 128>(p, num_sms, stream);
    case 256: return launch_dim<T, 256>(p, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int launch_append_block_scaled(int dtype, int head_dim, const ScaledAppendParams& p, int num_sms, cudaStream_t stream) {
  int e;
  switch (dtype) {
    case 0: e = launch_type<float>(p, head_dim, num_sms, stream); break;
    case 1: e = launch_type<__half>(p, head_dim, num_sms, stream); break;
    case 2: e = launch_type<__nv_bfloat16>(p, head_dim, num_sms, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
