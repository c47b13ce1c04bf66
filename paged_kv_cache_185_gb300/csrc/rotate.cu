// rotate.cu -- the rotary append: per-head norms of query and key, rotary
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
// of squares log2(D/16) shuffles.  A warp holds 32 / (D/16) rows at a time and
// walks over the heads of one token with the token's 8 (cos, sin) pairs in
// registers.  The token's heads are spread over more warps when there are few
// tokens.  The bound is memory: every value is read once and written once.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace wllm {
namespace {

constexpr int kRotateWarps = 4;
constexpr int kRotateBatch = 2;  // rows a lane has in flight

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
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(raw(i));
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

template <typename T, bool VEC, bool F8>
__global__ void __launch_bounds__(kRotateWarps * 32) rotate_kernel(const RotateParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kRotateWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(gw / p.warps_per_token);
  if (t >= p.num_tokens) return;
  const int part = static_cast<int>(gw - static_cast<int64_t>(t) * p.warps_per_token);
  const int g = lane & (p.row_lanes - 1), sub = lane / p.row_lanes;
  const bool mine = g < p.head_dim / 16;
  const int rows_per_step = 32 / p.row_lanes;
  const int num_rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int steps = (num_rows + rows_per_step - 1) / rows_per_step;

  const int64_t slot = p.slots_are_i64 ? static_cast<const int64_t*>(p.slots)[t]
                                       : static_cast<int64_t>(static_cast<const int32_t*>(p.slots)[t]);
  const int pairs = p.rot_dim / 2;
  const int p0 = 8 * g;                      // this lane's first pair
  const bool turns = mine && p0 < pairs;
  int c0, c1;                                // its two 8-element chunks
  if (p.adjacent || !turns) {
    c0 = 2 * g;
    c1 = c0 + 1;                             // behind the rotated part, chunks as they come
  } else {
    c0 = g;
    c1 = g + pairs / 8;
  }

  if (slot < 0) return;                      // padding token: nothing is read or written
  int bad = slot >= p.num_slots ? kErrSlot : 0;
  int64_t pos[kMaxRotaryAxes];
#pragma unroll
  for (int a = 0; a < kMaxRotaryAxes; ++a) {
    pos[a] = 0;
    if (a < p.num_axes) {
      const int64_t at = a * p.pos_sa + t;
      pos[a] = p.pos_are_i64 ? static_cast<const int64_t*>(p.positions)[at]
                             : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[at]);
      if (pos[a] < 0 || pos[a] >= p.num_positions) bad |= kErrPosition;
    }
  }
  if (bad) {
    if (lane == 0 && part == 0) atomicOr(p.err, bad);
    return;
  }

  float cs[8], sn[8];
  if (turns) {
    int axis = 0;
    while (axis < p.num_axes - 1 && p0 >= p.section_end[axis]) ++axis;
    if (p.table_vec && p0 + 8 <= p.section_end[axis]) {
      const int64_t row = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
      const float* tab = p.cos_sin + row * p.table_stride + p0;
      Chunk<float, true> c;
      c.load(tab);
      c.get(cs);
      c.load(tab + pairs);
      c.get(sn);
    } else {  // a section ends inside this lane's pairs, or rows without vector alignment
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        while (axis < p.num_axes - 1 && p0 + i >= p.section_end[axis]) ++axis;
        const int64_t row = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
        const float* tab = p.cos_sin + row * p.table_stride + p0 + i;
        cs[i] = __ldg(tab);
        sn[i] = __ldg(tab + pairs);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  }

  const int64_t blk = slot >> p.log2_bs;
  const int64_t off = slot & ((int64_t(1) << p.log2_bs) - 1);
  const T* q = static_cast<const T*>(p.q) + t * p.q_st;
  const T* k = static_cast<const T*>(p.key) + t * p.key_st;
  const T* v = static_cast<const T*>(p.value) + t * p.val_st;
  T* qo = static_cast<T*>(p.q_out) + t * p.qo_st;

  for (int s0 = part; s0 < steps; s0 += kRotateBatch * p.warps_per_token) {
    Chunk<T, VEC> x0[kRotateBatch], x1[kRotateBatch];
#pragma unroll
    for (int u = 0; u < kRotateBatch; ++u) {
      const int r = (s0 + u * p.warps_per_token) * rows_per_step + sub;
      if (mine && r < num_rows) {
        const T* src = r < p.num_q_heads                   ? q + r * p.q_sh
                       : r < p.num_q_heads + p.num_kv_heads ? k + (r - p.num_q_heads) * p.key_sh
                                                            : v + (r - p.num_q_heads - p.num_kv_heads) * p.val_sh;
        x0[u].load(src + 8 * c0);
        x1[u].load(src + 8 * c1);
      } else {
#pragma unroll
        for (int i = 0; i < Chunk<T, VEC>::kWords; ++i) x0[u].w[i] = x1[u].w[i] = 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kRotateBatch; ++u) {
      if (s0 + u * p.warps_per_token >= steps) break;
      const int r = (s0 + u * p.warps_per_token) * rows_per_step + sub;
      const bool is_q = r < p.num_q_heads;
      const bool is_v = r >= p.num_q_heads + p.num_kv_heads;
      float a[8], b[8];
      x0[u].get(a);
      x1[u].get(b);
      if (p.q_weight != nullptr || p.k_weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
        for (int m = p.row_lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(kFullMask, ss, m);
        const void* w = is_v ? nullptr : is_q ? p.q_weight : p.k_weight;
        if (w != nullptr && mine && r < num_rows) {
          const float inv = rsqrtf(ss * p.inv_dim + p.eps);
          float wa[8], wb[8];
          load_weight(p, w, 8 * c0, wa);
          load_weight(p, w, 8 * c1, wb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = a[i] * inv * wa[i];
            b[i] = b[i] * inv * wb[i];
          }
        }
      }
      if (!mine || r >= num_rows) continue;
      if (!is_v && turns) {
        if (p.adjacent) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float ea = a[2 * i], oa = a[2 * i + 1], eb = b[2 * i], ob = b[2 * i + 1];
            a[2 * i] = ea * cs[i] - oa * sn[i];
            a[2 * i + 1] = oa * cs[i] + ea * sn[i];
            b[2 * i] = eb * cs[4 + i] - ob * sn[4 + i];
            b[2 * i + 1] = ob * cs[4 + i] + eb * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = y * cs[i] + x * sn[i];
          }
        }
      }
      if (is_q) {
        T* dst = qo + r * p.qo_sh;
        x0[u].set(a);
        x1[u].set(b);
        x0[u].store(dst + 8 * c0);
        x1[u].store(dst + 8 * c1);
        continue;
      }
      const int h = r - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
      const int64_t row = ((blk * p.num_kv_heads + h) << p.log2_bs) + off;
      if constexpr (F8) {
        uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + row * p.head_dim;
        store_codes(dst + 8 * c0, a, is_v ? p.v_inv : p.k_inv);
        store_codes(dst + 8 * c1, b, is_v ? p.v_inv : p.k_inv);
      } else {
        if (!is_v) {
          x0[u].set(a);
          x1[u].set(b);
        }
        T* dst = reinterpret_cast<T*>(is_v ? p.v_cache : p.k_cache) + row * p.head_dim;
        x0[u].store(dst + 8 * c0);
        x1[u].store(dst + 8 * c1);
      }
    }
  }
}

template <typename T>
int launch_typed(const RotateParams& p, unsigned blocks, cudaStream_t stream) {
  const dim3 threads(kRotateWarps * 32);
  if (p.kv_fp8) {
    if (p.vec)
      rotate_kernel<T, true, true><<<blocks, threads, 0, stream>>>(p);
    else
      rotate_kernel<T, false, true><<<blocks, threads, 0, stream>>>(p);
  } else {
    if (p.vec)
      rotate_kernel<T, true, false><<<blocks, threads, 0, stream>>>(p);
    else
      rotate_kernel<T, false, false><<<blocks, threads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

int launch_rotate(RotateParams p, int num_sms, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 16 < p.head_dim) lanes *= 2;
  p.row_lanes = lanes;
  const int rows_per_step = 32 / lanes;
  const int steps = (p.num_q_heads + 2 * p.num_kv_heads + rows_per_step - 1) / rows_per_step;
  // one warp walks over a token's heads once the tokens alone give every SM 32
  // warps; below that the heads are spread, down to one step a warp
  int64_t w = (int64_t(num_sms) * 32 + p.num_tokens - 1) / p.num_tokens;
  if (w > steps) w = steps;
  p.warps_per_token = static_cast<int>(w < 1 ? 1 : w);
  const int64_t warps = int64_t(p.num_tokens) * p.warps_per_token;
  const unsigned blocks = static_cast<unsigned>((warps + kRotateWarps - 1) / kRotateWarps);
  int e;
  switch (p.src_dtype) {
    case 0: e = launch_typed<float>(p, blocks, stream); break;
    case 1: e = launch_typed<__half>(p, blocks, stream); break;
    case 2: e = launch_typed<__nv_bfloat16>(p, blocks, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
