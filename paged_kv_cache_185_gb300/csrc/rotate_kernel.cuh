// rotate_kernel.cuh -- the rotary append: per-head norms of query and key, rotary
// positions, the query written out and key and value written to their cache
// slots, one pass over a fused projection's output.
//
// Mathematics, for every row x (one head of one token) of query or key:
//   y = x * rsqrt(mean(x^2) + eps) * w              (where a weight is given)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
// for every pair p < R/2 of elements (a, b) = (p, p + R/2) or (2p, 2p + 1),
// with (cos, sin) = (cos_sin[pos][p], cos_sin[pos][R/2 + p]) and pos the
// position on the axis that pair p belongs to.  All of it in binary32; the one
// rounding to the output or cache type is the store.  Value rows are copied
// bit for bit (or stored as E4M3 codes).
//
// Work split: D/16 lanes share a row, each with 16 elements that are 8 whole
// pairs (8-element chunks c and c + R/16 of a row whose halves pair, chunks 2c
// and 2c + 1 otherwise), so a turn needs no exchange between lanes and the sum
// of squares log2(D/16) shuffles.  A warp holds 32 / (D/16) rows at a time.
// Many tokens: CTAs of two or four warps stay resident and the next token's rows and
// table rows come by bulk copies into the other of two buffers meanwhile; a
// token's factors (cos, sin, weights) are computed once for its rows.  Few
// tokens: their rows are spread over warps, a step or two each.  The bound is
// memory, every value is read once and written once; 8192 tokens of 28/4 heads
// of 128, bf16, norms, three axes (155 MB): 27.6 us, 0.83 of the measured copy
// rate; the same in f32 (306 MB): 56.8 us, 0.80.  Instructions decide, not the
// copies: with lanes and bounds known only at run time, weights read from global memory for every token and the step loop not
// unrolled, the same copies took 33.5 us.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace wllm {
namespace {

constexpr int kRingThreads = 128;  // at most; 128 registers a thread let an SM hold 4 CTAs of as many, or 8 of half

// Eight elements of a row as floats, or moved as they are.
template <typename T, bool VEC>
struct Chunk {
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {  // plain loads: q_out may be q itself
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = p[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) set_raw(i, e[i]);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = raw(i);
    }
  }
  __device__ __forceinline__ T raw(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      return *reinterpret_cast<const T*>(&h);
    }
  }
  __device__ __forceinline__ void set_raw(int i, T x) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(x);
    } else {
      const uint32_t h = *reinterpret_cast<const uint16_t*>(&x);
      w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xffffu) | (h << 16) : h;
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // the upper half of a binary32
#pragma unroll
      for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = Mma<T>::pack(f[2 * i], f[2 * i + 1]);
    }
  }
};

// E4M3 codes of x * inv: the product rounded to binary32, then to the nearest
// code (ties to even), saturating at +-448; eight bytes at an 8-byte boundary.
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = f32x2_to_e4m3x2(__fmul_rn(x[2 * i + 1], inv), __fmul_rn(x[2 * i], inv));
  *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void load_weight(const RotateParams& p, const void* w, int e, float (&f)[8]) {
  // weights are read once per row from L1: element-wise unless vectors fit
  if (p.weight_dtype == 0) {
    Chunk<float, true> c;
    Chunk<float, false> s;
    if (p.weight_vec) {
      c.load(static_cast<const float*>(w) + e);
      c.get(f);
    } else {
      s.load(static_cast<const float*>(w) + e);
      s.get(f);
    }
  } else if (p.weight_dtype == 1) {
    Chunk<__half, true> c;
    Chunk<__half, false> s;
    if (p.weight_vec) {
      c.load(static_cast<const __half*>(w) + e);
      c.get(f);
    } else {
      s.load(static_cast<const __half*>(w) + e);
      s.get(f);
    }
  } else {
    Chunk<__nv_bfloat16, true> c;
    Chunk<__nv_bfloat16, false> s;
    if (p.weight_vec) {
      c.load(static_cast<const __nv_bfloat16*>(w) + e);
      c.get(f);
    } else {
      s.load(static_cast<const __nv_bfloat16*>(w) + e);
      s.get(f);
    }
  }
}

// a b + c where `on`, else a b (to which -0 adds nothing, not even a sign).
__device__ __forceinline__ float product_and(bool on, float a, float b, float c) { return fmaf(a, b, on ? c : -0.f); }

// What one lane does with its 16 elements of a row: its chunks, the (cos, sin)
// of its pairs and the factors of the rows of one kind.
// LANES: lanes of a row where head_dim is 16 * LANES, 0 where they are p.row_lanes
// and some may be idle.
template <typename T, bool VEC, bool ADJACENT, int LANES>
struct RowMath {
  const RotateParams& p;
  int g, sub, c0, c1, p0;
  bool mine, turns;
  __device__ __forceinline__ int lanes() const { return LANES > 0 ? LANES : p.row_lanes; }  // a power of two
  __device__ __forceinline__ int lanes_log2() const { return __ffs(lanes()) - 1; }
  __device__ __forceinline__ int rows_per_step() const { return 32 >> lanes_log2(); }
  __device__ __forceinline__ int steps_of(int heads) const { return (heads + rows_per_step() - 1) >> (5 - lanes_log2()); }
  float cs[8], sn[8];
  // weights folded in: x' = f (fx x - gy y), y' = f (fy y + gx x), f the row's norm
  float fx[8], fy[8], gx[8], gy[8];

  __device__ __forceinline__ RowMath(const RotateParams& params, int lane) : p(params) {
    g = lane & (lanes() - 1), sub = lane >> lanes_log2();
    mine = LANES > 0 || g < p.head_dim / 16;
    p0 = 8 * g;                              // this lane's first pair
    turns = mine && p0 < p.rot_dim / 2;
    if (ADJACENT || !turns) {
      c0 = 2 * g;                            // behind the rotated part, chunks as they come
      c1 = c0 + 1;
    } else {
      c0 = g;
      c1 = g + p.rot_dim / 16;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  }

  // (cos, sin) of this lane's pairs; row(axis) is the table row of an axis.
  template <typename Row>
  __device__ __forceinline__ void angles(Row row) {
    if (!turns) return;
    const int pairs = p.rot_dim / 2;
    int axis = 0;
    while (axis < p.num_axes - 1 && p0 >= p.section_end[axis]) ++axis;
    if (p.table_vec && p0 + 8 <= p.section_end[axis]) {
      const float* tab = row(axis) + p0;
      Chunk<float, true> c;
      c.load(tab);
      c.get(cs);
      c.load(tab + pairs);
      c.get(sn);
    } else {  // a section ends inside this lane's pairs, or rows without vector alignment
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        while (axis < p.num_axes - 1 && p0 + i >= p.section_end[axis]) ++axis;
        const float* tab = row(axis) + p0 + i;
        cs[i] = tab[0];
        sn[i] = tab[pairs];
      }
    }
  }

  // Factors of the rows with a weight (null: none), from global memory.
  __device__ __forceinline__ void factors(const void* weight) {
    factors(weight != nullptr, [&](int e, float (&w)[8]) { load_weight(p, weight, e, w); });
  }

  template <typename Load>
  __device__ __forceinline__ void factors(bool weighted, Load load) {
    float wx[8], wy[8];
    if (weighted && mine) {
      float wa[8], wb[8];
      load(8 * c0, wa);
      load(8 * c1, wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wx[i] = ADJACENT ? (i < 4 ? wa[(2 * i) & 7] : wb[(2 * i) & 7]) : wa[i];
        wy[i] = ADJACENT ? (i < 4 ? wa[(2 * i + 1) & 7] : wb[(2 * i + 1) & 7]) : wb[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) wx[i] = wy[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      fx[i] = wx[i] * cs[i], gx[i] = wx[i] * sn[i];
      fy[i] = wy[i] * cs[i], gy[i] = wy[i] * sn[i];
    }
  }

  // The turned values of a row's two chunks.  All lanes of the warp call it.
  __device__ __forceinline__ void turn(const Chunk<T, VEC>& u, const Chunk<T, VEC>& v, bool norm, float (&a)[8],
                                       float (&b)[8]) {
    u.get(a);
    v.get(b);
    float f = 1.f;
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
      for (int m = lanes() >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(kFullMask, ss, m);
      f = rsqrtf(ss * p.inv_dim + p.eps);
    }
    // Behind the rotated part every element stands alone: a product of 0 with its neighbour would bring that one's infinity
    // or NaN along, so the second product of a turn is left out (by a branch around the turn 3001 tokens half turned took
    // 14.1 us instead of 13.6).  The products are those of a plain turn, in its order.
    if constexpr (ADJACENT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
        a[2 * i] = f * product_and(turns, fx[i], x, -(gy[i] * y));
        a[2 * i + 1] = f * product_and(turns, fy[i], y, gx[i] * x);
        b[2 * i] = f * product_and(turns, fx[4 + i], z, -(gy[4 + i] * w));
        b[2 * i + 1] = f * product_and(turns, fy[4 + i], w, gx[4 + i] * z);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = a[i], y = b[i];
        a[i] = f * product_and(turns, fx[i], x, -(gy[i] * y));
        b[i] = f * product_and(turns, fy[i], y, gx[i] * x);
      }
    }
  }

  // Store query row r of token t.
  __device__ __forceinline__ void store_q(int64_t t, int r, const float (&a)[8], const float (&b)[8]) const {
    if (!mine || r >= p.num_q_heads) return;
    T* dst = static_cast<T*>(p.q_out) + t * p.qo_st + r * p.qo_sh;
    Chunk<T, VEC> u, v;
    u.set(a);
    v.set(b);
    u.store(dst + 8 * c0);
    v.store(dst + 8 * c1);
  }

  // Store key row (turned values a, b) or value row (chunks u, v) r in its slot.
  template <bool F8>
  __device__ __forceinline__ void store_kv(int64_t slot, int r, bool is_k, Chunk<T, VEC> u, Chunk<T, VEC> v, float (&a)[8],
                                           float (&b)[8]) const {
    if (!mine || r >= p.num_kv_heads) return;
    const int64_t blk = slot >> p.log2_bs, off = slot & ((int64_t(1) << p.log2_bs) - 1);
    const int64_t row = (((blk * p.num_kv_heads + r) << p.log2_bs) + off) * p.head_dim;
    if constexpr (F8) {
      if (!is_k) u.get(a), v.get(b);
      uint8_t* dst = (is_k ? p.k_cache : p.v_cache) + row;
      store_codes(dst + 8 * c0, a, is_k ? p.k_inv : p.v_inv);
      store_codes(dst + 8 * c1, b, is_k ? p.k_inv : p.v_inv);
    } else {
      if (is_k) u.set(a), v.set(b);
      T* dst = reinterpret_cast<T*>(is_k ? p.k_cache : p.v_cache) + row;
      u.store(dst + 8 * c0);
      v.store(dst + 8 * c1);
    }
  }
};

__device__ __forceinline__ int64_t slot_of(const RotateParams& p, int64_t t) {
  return p.slots_are_i64 ? static_cast<const int64_t*>(p.slots)[t]
                         : static_cast<int64_t>(static_cast<const int32_t*>(p.slots)[t]);
}

__device__ __forceinline__ int64_t position_of(const RotateParams& p, int axis, int64_t t) {
  const int64_t at = axis * p.pos_sa + t;
  return p.pos_are_i64 ? static_cast<const int64_t*>(p.positions)[at]
                       : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[at]);
}

// Few tokens, or rows that bulk copies cannot take: the steps of a token's rows
// are spread over warps_per_token warps, rows straight into registers.
template <typename T, bool VEC, bool F8, bool ADJACENT>
__global__ void __launch_bounds__(kRotateWarps * 32, 4) rotate_kernel(const RotateParams p) {
  constexpr int kDeep = 2;  // steps whose rows are in flight
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const unsigned gw = blockIdx.x * kRotateWarps + (threadIdx.x >> 5), token = gw / static_cast<unsigned>(p.warps_per_token);
  const int64_t t = token;
  if (t >= p.num_tokens) return;
  const int part = static_cast<int>(gw - token * p.warps_per_token);
  RowMath<T, VEC, ADJACENT, 0> math(p, lane);
  const int rows_per_step = math.rows_per_step(), steps_q = math.steps_of(p.num_q_heads), steps_kv = math.steps_of(p.num_kv_heads);
  const int steps = steps_q + 2 * steps_kv;  // of query rows, then of key rows, then of value rows

  Chunk<T, VEC> x0[kDeep], x1[kDeep];
  auto load = [&](int s, Chunk<T, VEC>& u, Chunk<T, VEC>& v) {
    const T* src;
    bool have = math.mine && s < steps;
    if (s < steps_q) {
      const int r = s * rows_per_step + math.sub;
      have = have && r < p.num_q_heads;
      src = static_cast<const T*>(p.q) + t * p.q_st + r * p.q_sh;
    } else if (s < steps_q + steps_kv) {
      const int r = (s - steps_q) * rows_per_step + math.sub;
      have = have && r < p.num_kv_heads;
      src = static_cast<const T*>(p.key) + t * p.key_st + r * p.key_sh;
    } else {
      const int r = (s - steps_q - steps_kv) * rows_per_step + math.sub;
      have = have && r < p.num_kv_heads;
      src = static_cast<const T*>(p.value) + t * p.val_st + r * p.val_sh;
    }
    if (have) {
      u.load(src + 8 * math.c0);
      v.load(src + 8 * math.c1);
    } else {
#pragma unroll
      for (int i = 0; i < Chunk<T, VEC>::kWords; ++i) u.w[i] = v.w[i] = 0u;
    }
  };
  // slot, positions and the first rows together: one round trip to memory
  const int64_t slot = slot_of(p, t);
  int64_t pos[kMaxRotaryAxes];
#pragma unroll
  for (int a = 0; a < kMaxRotaryAxes; ++a) pos[a] = a < p.num_axes ? position_of(p, a, t) : 0;
#pragma unroll
  for (int i = 0; i < kDeep; ++i) load(part + i * p.warps_per_token, x0[i], x1[i]);

  if (slot < 0) return;  // padding token
  int bad = slot >= p.num_slots ? kErrSlot : 0;
#pragma unroll
  for (int a = 0; a < kMaxRotaryAxes; ++a)
    if (pos[a] < 0 || (a < p.num_axes && pos[a] >= p.num_positions)) bad |= kErrPosition;
  if (bad) {
    if (lane == 0 && part == 0) atomicOr(p.err, bad);
    return;
  }
  math.angles([&](int axis) {
    return p.cos_sin + (axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3]) * p.table_stride;
  });

  int kind = -1;
  for (int s0 = part; s0 < steps; s0 += kDeep * p.warps_per_token) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int s = s0 + i * p.warps_per_token;
      if (s >= steps) break;
      float a[8], b[8];
      if (s < steps_q) {
        if (kind != 0) math.factors(p.q_weight);
        kind = 0;
        math.turn(x0[i], x1[i], p.q_weight != nullptr, a, b);
        load(s + kDeep * p.warps_per_token, x0[i], x1[i]);
        math.store_q(t, s * rows_per_step + math.sub, a, b);
        continue;
      }
      const bool is_k = s < steps_q + steps_kv;
      if (is_k && kind != 1) math.factors(p.k_weight);
      kind = is_k ? 1 : 2;
      const Chunk<T, VEC> u = x0[i], v = x1[i];
      if (is_k) math.turn(u, v, p.k_weight != nullptr, a, b);
      load(s + kDeep * p.warps_per_token, x0[i], x1[i]);
      math.template store_kv<F8>(slot, (s - steps_q - (is_k ? 0 : steps_kv)) * rows_per_step + math.sub, is_k, u, v, a, b);
    }
  }
}

// Many tokens: resident CTAs walk over the tokens, and while one is turned the
// next one's rows and table rows arrive in the CTA's other buffer by bulk
// copies, so no warp waits for a chain of slot, position, table and rows.  The
// warps share a token's steps.  Buffer: query rows, key rows, value rows, one
// table row an axis.
template <typename T, bool F8, bool ADJACENT, int LANES>
__global__ void __launch_bounds__(kRingThreads, 4) rotate_ring_kernel(const RotateParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;  // 2 or 4 warps
  const uint32_t row_bytes = p.head_dim * sizeof(T), table_bytes = p.rot_dim * sizeof(float);
  const uint32_t q_bytes = p.num_q_heads * row_bytes, kv_bytes = p.num_kv_heads * row_bytes;
  const uint32_t buffer_bytes = q_bytes + 2 * kv_bytes + p.num_axes * table_bytes;
  if (threadIdx.x < 2) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
  fence_mbar_init();
  grid_wait();
  grid_launch_dependents();
  // the norms' weights in binary32, behind the buffers
  float* weights = reinterpret_cast<float*>(raw + 2 * buffer_bytes);
  for (int i = threadIdx.x; i < p.head_dim / 4; i += blockDim.x) {  // 8 elements of q's, then of k's
    const void* w = i < p.head_dim / 8 ? p.q_weight : p.k_weight;
    float f[8];
    if (w != nullptr) {
      load_weight(p, w, 8 * (i % (p.head_dim / 8)), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) weights[8 * i + e] = f[e];
    }
  }
  __syncthreads();
  auto factors_of = [&](auto& math, bool is_k) {
    math.factors((is_k ? p.k_weight : p.q_weight) != nullptr, [&](int e, float (&w)[8]) {
      Chunk<float, true> c;
      c.load(weights + (is_k ? p.head_dim : 0) + e);
      c.get(w);
    });
  };

  const int stride = gridDim.x;
  RowMath<T, true, ADJACENT, LANES> math(p, lane);
  const int rows_per_step = math.rows_per_step(), steps_q = math.steps_of(p.num_q_heads), steps_kv = math.steps_of(p.num_kv_heads);

  // slot and (lane a: axis a) position of a token
  struct Meta {
    int64_t slot, pos;
  };
  auto fetch = [&](int64_t at) {
    Meta m{-1, 0};
    if (at < p.num_tokens) {
      m.slot = slot_of(p, at);
      if (lane < p.num_axes) m.pos = position_of(p, lane, at);
    }
    return m;
  };
  // Whether token `at` has work; the first warp starts its copies into buffer `k`.
  auto start = [&](const Meta& m, int64_t at, int k) {
    if (m.slot < 0) return false;  // padding, or behind the last token
    const bool off_table = __any_sync(kFullMask, m.pos < 0 || m.pos >= p.num_positions);
    if (m.slot >= p.num_slots || off_table) {
      if (threadIdx.x == 0) atomicOr(p.err, (m.slot >= p.num_slots ? kErrSlot : 0) | (off_table ? kErrPosition : 0));
      return false;
    }
    if (warp != 0) return true;
    const uint32_t bar = smem_u32(&bars[k]), dst = smem_u32(raw + k * buffer_bytes);
    if (lane == 0) mbar_arrive_expect_tx(bar, buffer_bytes);
    __syncwarp();
    // rows of one operand that lie next to each other in one copy
    auto rows = [&](const void* base, int64_t st, int64_t sh, int heads, uint32_t to, int first_lane) {
      const T* src = static_cast<const T*>(base) + at * st;
      if (sh == p.head_dim) {
        if (lane == first_lane && heads > 0) bulk_load(to, src, heads * row_bytes, bar);
      } else {
        for (int r = lane; r < heads; r += 32) bulk_load(to + r * row_bytes, src + r * sh, row_bytes, bar);
      }
    };
    rows(p.q, p.q_st, p.q_sh, p.num_q_heads, dst, 4);
    rows(p.key, p.key_st, p.key_sh, p.num_kv_heads, dst + q_bytes, 5);
    rows(p.value, p.val_st, p.val_sh, p.num_kv_heads, dst + q_bytes + kv_bytes, 6);
    if (lane < p.num_axes)
      bulk_load(dst + q_bytes + 2 * kv_bytes + lane * table_bytes, p.cos_sin + m.pos * p.table_stride, table_bytes, bar);
    return true;
  };

  int64_t t = blockIdx.x;
  Meta now = fetch(t), next = fetch(t + stride);
  int k = 0;
  uint32_t phase = 0u;  // bit k: buffer k's
  bool live = start(now, t, 0);
  for (; t < p.num_tokens; t += stride, k ^= 1) {
    __syncthreads();  // every warp has read the buffer that the next copies go to
    const bool coming = start(next, t + stride, k ^ 1);
    const Meta after = fetch(t + 2 * stride);
    if (live) {
      const uint32_t bar = smem_u32(&bars[k]);
      if (!mbar_wait_warp(bar, (phase >> k) & 1u, p.wait_limit_ns)) {
        // give up: record it, and leave no copy in flight
        if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
        mbar_wait_bounded(bar, (phase >> k) & 1u, p.wait_limit_ns);
        if (coming) mbar_wait_bounded(smem_u32(&bars[k ^ 1]), (phase >> (k ^ 1)) & 1u, p.wait_limit_ns);
        return;
      }
      phase ^= 1u << k;
      const uint8_t* buf = raw + k * buffer_bytes;
      const float* tables = reinterpret_cast<const float*>(buf + q_bytes + 2 * kv_bytes);
      math.angles([&](int axis) { return tables + axis * p.rot_dim; });
      float a[8], b[8];
      Chunk<T, true> u, v;
      auto load = [&](const uint8_t* rows, int r, int heads) {
        const T* src = reinterpret_cast<const T*>(rows + min(r, heads - 1) * row_bytes);
        if (math.mine) {
          u.load(src + 8 * math.c0);
          v.load(src + 8 * math.c1);
        } else {
#pragma unroll
          for (int i = 0; i < Chunk<T, true>::kWords; ++i) u.w[i] = v.w[i] = 0u;
        }
      };
      factors_of(math, false);
#pragma unroll 2
      for (int s = warp; s < steps_q; s += warps) {
        const int r = s * rows_per_step + math.sub;
        load(buf, r, p.num_q_heads);
        math.turn(u, v, p.q_weight != nullptr, a, b);
        math.store_q(t, r, a, b);
      }
      bool fresh = p.k_weight == p.q_weight;
      for (int i = (warp - steps_q) & (warps - 1); i < 2 * steps_kv; i += warps) {
        const int r = (i >> 1) * rows_per_step + math.sub;
        if (i & 1) {
          load(buf + q_bytes + kv_bytes, r, p.num_kv_heads);
        } else {
          if (!fresh) factors_of(math, true);
          fresh = true;
          load(buf + q_bytes, r, p.num_kv_heads);
          math.turn(u, v, p.k_weight != nullptr, a, b);
        }
        math.template store_kv<F8>(now.slot, r, !(i & 1), u, v, a, b);
      }
    }
    now = next, next = after, live = coming;
  }
}

template <typename T, bool VEC, bool F8>
int launch_few(const RotateParams& p, unsigned blocks, cudaStream_t stream) {
  if (p.adjacent)
    return launch_dependent(&rotate_kernel<T, VEC, F8, true>, dim3(blocks), dim3(kRotateWarps * 32), 0, 0, stream, p);
  return launch_dependent(&rotate_kernel<T, VEC, F8, false>, dim3(blocks), dim3(kRotateWarps * 32), 0, 0, stream, p);
}

template <typename T, bool F8, bool ADJACENT, int LANES>
int launch_ring(const RotateParams& p, int smem, int num_sms, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  const int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&rotate_ring_kernel<T, F8, ADJACENT, LANES>), smem);
  if (e != cudaSuccess) return e;
  // CTAs of 2 warps or of 4, as many as are resident (228 KB an SM, 1 KB of it the system's in each CTA): whichever
  // takes fewer steps one after another, a token counted as one more.  Measured, us for 2 and 4 warps: 8192 tokens of
  // 28/4 heads 27.7 and 34.4 (9 steps), 3001 of 32/8 15.1 and 13.7, 1000 of 64/8 14.3 and 12.0, 830 of 4/1 4.0 and 4.7.
  const int rows_per_step = 32 / p.row_lanes;
  const int steps = (p.num_q_heads + rows_per_step - 1) / rows_per_step + 2 * ((p.num_kv_heads + rows_per_step - 1) / rows_per_step);
  const int fit = std::max(1, 228 * 1024 / (smem + 1024 + 64));
  int64_t grid = 0, least = 0;
  int warps = 0;
  for (int w = 2; w <= 4; w += 2) {
    const int64_t resident = int64_t(num_sms) * std::min(fit, 16 / w);
    const int64_t serial = (p.num_tokens + resident - 1) / resident * ((steps + w - 1) / w + 1);
    if (warps == 0 || serial < least) grid = std::min<int64_t>(resident, p.num_tokens), least = serial, warps = w;
  }
  return launch_dependent(&rotate_ring_kernel<T, F8, ADJACENT, LANES>, dim3(static_cast<unsigned>(grid)), dim3(warps * 32), smem, 0,
                          stream, p);
}

template <typename T, bool F8, bool ADJACENT>
int launch_many(const RotateParams& p, int smem, int num_sms, cudaStream_t stream) {
  switch (p.head_dim) {  // without idle lanes or runtime bounds where head_dim is 64 or 128
    case 64: return launch_ring<T, F8, ADJACENT, 4>(p, smem, num_sms, stream);
    case 128: return launch_ring<T, F8, ADJACENT, 8>(p, smem, num_sms, stream);
    default: return launch_ring<T, F8, ADJACENT, 0>(p, smem, num_sms, stream);
  }
}

// `ring_smem` > 0: the resident form with that much shared memory.
template <typename T>
int launch_rotate_typed(const RotateParams& p, unsigned blocks, int ring_smem, int num_sms, cudaStream_t stream) {
  if (ring_smem > 0) {
    if (p.adjacent)
      return p.kv_fp8 ? launch_many<T, true, true>(p, ring_smem, num_sms, stream)
                      : launch_many<T, false, true>(p, ring_smem, num_sms, stream);
    return p.kv_fp8 ? launch_many<T, true, false>(p, ring_smem, num_sms, stream)
                    : launch_many<T, false, false>(p, ring_smem, num_sms, stream);
  }
  if (p.kv_fp8) return p.vec ? launch_few<T, true, true>(p, blocks, stream) : launch_few<T, false, true>(p, blocks, stream);
  return p.vec ? launch_few<T, true, false>(p, blocks, stream) : launch_few<T, false, false>(p, blocks, stream);
}

}  // namespace
}  // namespace wllm
