// prefill_block_scaled.cu -- chunked-prefill (multi-query) attention over a paged
// cache of E4M3 codes with a scale for each block and kv head, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Mathematics: chunk token i of sequence b sits at position P = L_b - n_b + i and
// attends to tokens 0 .. P, whose K and V are ks_t k_t and vs_t v_t (codes' values,
// their block's scales).  Per query row, with the base 2,
//   x_t = scale log2(e) ks_t (q . k_t) + log2(vs_t),  w_t = 2^(x_t - m),
//   O = sum_t w_t v_t,  l = sum_t w_t / vs_t,  out = O / l,
// as in the decode (decode_block_scaled.cu): the value's scale is part of the
// weight.  m moves only when a row's largest x exceeds it by more than 8, so O is
// seldom rescaled and weights stay below 2^8; they are taken times 2^7 to be normal
// numbers of f16 down to 2^-21.  l sums the weights before they are rounded: behind
// a small vs a weight may round to nothing and still count in l.
//
// One CTA (one per SM) owns 256 query rows of one sequence and one kv head, as two
// 128-row tiles, row r being (token r / G, query head r % G of the group), and
// walks the rows' context in tiles of 128 tokens.  Tensor memory holds, per Q tile,
// the scores S (128 columns), over which the softmax writes the weights P (f16, two
// a column), and the output O.  Fourteen warps:
//
//   warp 0 (producer): the block table, the codes of each tile's K and then V by
//     TMA (16-row boxes, 128-byte swizzle) into a ring of raw slots, and their
//     scales by 4-byte asynchronous copies on the same mbarrier;
//   warps 10-13 (widening): thread r takes row r of a raw slot to f16, which is
//     exact, in a slot laid out for the products ([head_dim / 64][128 tokens][128
//     bytes], swizzled); V rows past the context become zeros, and so do NaN codes
//     (their first tokens are kept, and rows that see them get NaN at the end); and
//     once a tile the factors that each run of 8 tokens gives the softmax;
//   warp 1 (MMA): one thread issues S_x = Q_x K^T and O_x += P_x V (M = 128, f16)
//     for Q tile x as soon as either is ready;
//   warps 2-5 and 6-9 (softmax of Q tile 0 and 1): thread r owns row r.  Its scores
//     are read twice, once for the maximum and once for the weights, 32 at a time.
// The query rows go to f16 after a power of two was divided out of each.
//
// Every wait is bounded; on a timeout the CTA records the error, waits (bounded)
// for its copies and MMAs in flight, frees its tensor memory and returns.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "decode_kernel.cuh"
#include "launch.h"
#include "mma_e4m3.cuh"
#include "prefill_rows.cuh"
#include "tcgen05.cuh"

namespace wllm {
namespace {

constexpr int kTileRows = 128;               // rows of a Q tile (M = 128)
constexpr int kTiles = 2;                    // Q tiles of a CTA
constexpr int kRows = kTileRows * kTiles;
constexpr int kKv = 128;                     // tokens of a kv tile
constexpr int kOctets = kKv / 8;
constexpr int kThreads = (2 + 4 * kTiles + 4) * 32;
constexpr float kRescale = 8.f;              // the running maximum moves by more than this (log2) only
constexpr float kWeightShift = 7.f;
constexpr int kFactorTiles = 4;              // kv tiles whose factors are kept
constexpr int kScaleTiles = 2;               // and whose scales are, until the factors are made

template <int D>
struct Shape {
  using G = Geom<uint8_t, D>;
  static constexpr int kQBytes = kTileRows * D * 2;        // [chunk][128 rows][128 B]
  static constexpr int kSlotBytes = kKv * D * 2;           // [chunk][128 tokens][128 B]
  static constexpr int kChunkStride = kKv * 128;
  static constexpr int kRawBytes = kKv * D;
  static constexpr int kSlots = D == 64 ? 6 : 4;           // widened K or V tiles
  static constexpr int kRaws = D == 64 ? 4 : 2;            // tiles of codes
  static constexpr int kFactorBytes = kFactorTiles * kOctets * 16;
  static constexpr int kScaleBytes = kScaleTiles * 2 * kOctets * 4;
  static constexpr int kNanBytes = D * 4;
  static constexpr int kBarBytes = D == 64 ? 384 : 256;
  static constexpr int kSmem = 1024 + kTiles * kQBytes + kSlots * kSlotBytes + kRaws * kRawBytes + kFactorBytes + kScaleBytes +
                               kNanBytes + kBarBytes;
  static constexpr uint32_t kTmemCols = 512;
  // tensor-memory columns of Q tile x start at x * kTileCols: S (P over its first 64), O
  static constexpr int kTileCols = 256;
  static constexpr int kS = 0, kO = 128;
  static_assert(kSmem <= 232448, "227 KB");
  // a tile's factors are written once K's slot is free, that is once the scores of tile j - kSlots / 2 are computed, and with them the weights of the tile before
  static_assert(kFactorTiles >= kSlots / 2 + 1, "factors are not overwritten while they are needed");
  // a tile's scales are asked for once K's raw slot is free, that is once those of tile j - kRaws / 2 are used
  static_assert(kScaleTiles >= kRaws / 2, "nor scales");
};
static_assert(2 * (Shape<64>::kSmem + 1024) > 233472, "a second resident CTA would contend for tensor memory");

__device__ __forceinline__ void copy4_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void arrive_behind_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float scale_in_range(float s) {
  constexpr float kLeast = 1.f / (1ull << -kLeastScaleExp), kMost = static_cast<float>(1ull << kMostScaleExp);
  return fminf(fmaxf(s, kLeast), kMost);  // a NaN counts as the least
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2(float lo, float hi) { return Mma<__half>::pack(lo, hi); }

// Eight elements of a row, 16-bit.
template <typename T>
__device__ __forceinline__ uint4 load8(const T* src, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(src);
  const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e[2 * i] | static_cast<uint32_t>(e[2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float* v, float by, bool vec) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = Mma<T>::pack(v[2 * i] * by, v[2 * i + 1] * by);
  if (vec) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t* e = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[2 * i] = static_cast<uint16_t>(w[i]), e[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
  }
}

// RUN: tokens of a run with one scale that the softmax tells apart, 8 for blocks
// of 8 tokens, else 16.
template <typename T, int D, int RUN>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_block_scaled_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                const ScaledPrefillParams sp) {
  using S = Shape<D>;
  using G8 = typename S::G;
  const PrefillParams& p = sp.base;
  constexpr int R = S::kSlots, RR = S::kRaws;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                                  // [2][Q tile]
  uint8_t* ring = q_s + kTiles * S::kQBytes;            // widened tiles: K, V, K, V, ...
  uint8_t* raw = ring + R * S::kSlotBytes;              // tiles of codes, in the same order
  float4* factors = reinterpret_cast<float4*>(raw + RR * S::kRawBytes);              // [tile][octet] ks, log2 vs, 1 / vs
  float* scales = reinterpret_cast<float*>(factors + kFactorTiles * kOctets);        // [tile][K, V][octet]
  int* nan_from = reinterpret_cast<int*>(scales + kScaleTiles * 2 * kOctets);        // [D] first token whose value is NaN
  uint64_t* full = reinterpret_cast<uint64_t*>(nan_from + D);  // [R] widened (widening -> MMA)
  uint64_t* empty = full + R;      // [R] read by every product (MMA -> widening)
  uint64_t* rfull = empty + R;     // [RR] codes and scales landed (producer -> widening)
  uint64_t* rempty = rfull + RR;   // [RR] codes read (widening -> producer)
  uint64_t* ffull = rempty + RR;   // [kFactorTiles] a tile's factors written (widening -> softmax)
  uint64_t* sfull = ffull + kFactorTiles;  // [tile] S written (MMA -> softmax)
  uint64_t* pfull = sfull + 2;     // [tile] P written, O rescaled (softmax -> MMA)
  uint64_t* pvdone = pfull + 2;    // [tile] the PV product done (MMA -> MMA, softmax)
  uint64_t* qfull = pvdone + 2;    // Q written (softmax -> MMA)
  uint64_t* fin = qfull + 1;       // every MMA of the CTA done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(fin + 1);
  int* info = reinterpret_cast<int*>(tslot + 1);  // [0] sequence (-1: none), [1] its row block, [2] whether a value is NaN
  static_assert((2 * R + 2 * RR + kFactorTiles + 8) * 8 + 16 <= S::kBarBytes, "room for the barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  const int kvh = static_cast<int>(blockIdx.x % p.num_kv_heads);
  const int tgt_block = static_cast<int>(blockIdx.x / p.num_kv_heads);
  if (warp == 0) {
    if (lane == 0) tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
    if (lane == 0) {
      for (int s = 0; s < R; ++s) {
        mbar_init(smem_u32(full + s), 4);
        mbar_init(smem_u32(empty + s), 1);
      }
      for (int s = 0; s < RR; ++s) {
        mbar_init(smem_u32(rfull + s), 1 + 32);
        mbar_init(smem_u32(rempty + s), 4);
      }
      for (int s = 0; s < kFactorTiles; ++s) mbar_init(smem_u32(ffull + s), 1);
      for (int x = 0; x < kTiles; ++x) {
        mbar_init(smem_u32(sfull + x), 1);
        mbar_init(smem_u32(pfull + x), 4);
        mbar_init(smem_u32(pvdone + x), 1);
      }
      mbar_init(smem_u32(qfull), 4 * kTiles);
      mbar_init(smem_u32(fin), 1);
      fence_mbar_init();
    }
    __syncwarp();
    grid_wait();
    int seq, tile;
    row_block_of(p, kRows, tgt_block, lane, &seq, &tile);
    if (lane == 0) info[0] = seq, info[1] = tile, info[2] = 0;
    for (int d = lane; d < D; d += 32) nan_from[d] = INT_MAX;
  } else {
    grid_wait();
  }
  grid_launch_dependents();
  if (warp == 1) tc::alloc(smem_u32(tslot), S::kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;

  // starts that decrease are recorded whether or not a row block meets them, by the CTA that is launched last
  if (blockIdx.x == gridDim.x - 1) {
    for (int i = threadIdx.x; i < p.num_seqs; i += kThreads)
      if (p.query_start_loc[i + 1] < p.query_start_loc[i]) atomicOr(p.err, kErrLen);
  }

  // ---- the block's rows and the context they see (uniform over the CTA)
  const int b = info[0];
  int n_rows = 0, row0 = 0, pos0 = 0, s0 = 0;
  int nt[kTiles] = {0, 0};  // kv tiles each Q tile needs
  int kv_end = 0;           // tokens any row of the block sees
  if (b >= 0) {
    const int l_max = p.max_blocks * p.block_size;
    s0 = p.query_start_loc[b];
    int n = p.query_start_loc[b + 1] - s0;
    if (s0 < 0 || n < 0 || static_cast<int64_t>(s0) + n > p.num_tokens) {  // inconsistent query starts
      if (threadIdx.x == 0) atomicOr(p.err, kErrLen);
    } else {
      int L = p.context_lens[b];
      if (L < 0 || L > l_max || n > L) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrLen);
        L = L < 0 ? 0 : (L > l_max ? l_max : L);
        n = n > L ? L : n;
      }
      n_rows = n * G;
      row0 = info[1] * kRows;
      pos0 = L - n;
#pragma unroll
      for (int x = 0; x < kTiles; ++x) {  // (no rows only when n was clamped, error already flagged)
        const int rx = row0 + x * kTileRows;
        if (rx < n_rows) {
          const int end_x = pos0 + (min(n_rows, rx + kTileRows) - 1) / G + 1;
          nt[x] = (end_x + kKv - 1) / kKv;
          kv_end = max(kv_end, end_x);
        }
      }
    }
  }
  const int n_tiles = max(nt[0], nt[1]);

  // one lane waits, the warp learns the outcome
  auto wait_warp = [&](uint64_t* bar, int parity) -> bool {
    bool got = true;
    if (lane == 0) got = mbar_wait_bounded(smem_u32(bar), static_cast<uint32_t>(parity), p.wait_limit_ns);
    return __shfl_sync(kFullMask, got ? 1 : 0, 0) != 0;
  };
  bool ok = true;

  if (warp == 0 && n_tiles > 0) {
    // ------------------------------- producer -------------------------------
    constexpr int kBoxes = kKv / 16;  // 16-token boxes of a kv tile (times the row's column boxes, one for D <= 128)
    const int32_t* bt_row = p.block_tables + static_cast<int64_t>(b) * p.bt_stride;
    int issued = 0;                   // raw slots whose copies were issued
    for (int j = 0; ok && j < n_tiles; ++j) {
      // lanes 0..15: the table entry of each run of 8 tokens
      int entry = 0;
      const int t8 = j * kKv + 8 * (lane & 15);
      if (t8 < kv_end) {
        entry = bt_row[t8 >> p.log2_bs];
        if (entry < 0 || entry >= p.num_blocks) {
          atomicOr(p.err, kErrBlock);
          entry = 0;
        }
      }
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // K, then V
        const int c = 2 * j + half, s = c % RR;
        if (!wait_warp(rempty + s, ((c / RR) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t slot = smem_u32(raw + s * S::kRawBytes), bar = smem_u32(rfull + s);
        // a box a lane: 16 tokens, or 8 where blocks have no more
        const int octet = RUN == 8 ? lane & 15 : (2 * lane) & 15;
        const int phys = __shfl_sync(kFullMask, entry, octet);
        const int t = j * kKv + 8 * octet;
        const bool live = lane < (RUN == 8 ? kOctets : kBoxes) && t < kv_end;
        constexpr uint32_t kBoxBytes = RUN == 8 ? 1024u : static_cast<uint32_t>(G8::kTileBytes);
        const uint32_t bytes = kBoxBytes * __popc(__ballot_sync(kFullMask, live));
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (live) {
          const int at = kvh * p.block_size + (t & (p.block_size - 1));
          tma_load_3d(slot + lane * kBoxBytes, half ? &vmap : &kmap, bar, 0, G8::kPairRows ? at >> 1 : at, phys);
        }
        if (half == 0 && t8 < kv_end)  // both scales of a run come with its K: lanes 0-15 K's, 16-31 V's
          copy4_async(smem_u32(scales + (j % kScaleTiles) * 2 * kOctets + lane),
                      (lane < 16 ? sp.k_scales : sp.v_scales) + static_cast<int64_t>(entry) * p.num_kv_heads + kvh);
        arrive_behind_copies(bar);
        ++issued;
      }
    }
    // every copy still in flight lands before the CTA may leave
    for (int c = issued - RR > 0 ? issued - RR : 0; c < issued; ++c)
      if (!wait_warp(rfull + c % RR, (c / RR) & 1)) ok = false;
  } else if (warp == 1 && n_tiles > 0) {
    // --------------------------------- MMA ----------------------------------
    if (lane == 0) {
      constexpr uint32_t kIdS = tc::f16_idesc(false, false, false, kTileRows, kKv);
      constexpr uint32_t kIdO = tc::f16_idesc(false, false, true, kTileRows, D);
      const uint32_t q_a = smem_u32(q_s), ring_a = smem_u32(ring);
      // the operations of one kind in order: kv tile by kv tile, Q tile 0 then
      // 1, skipping Q tiles that need fewer kv tiles
      const int m2 = min(nt[0], nt[1]);
      const int total = nt[0] + nt[1];
      auto op_at = [&](int k, int& j, int& x) {
        if (k < 2 * m2) {
          j = k >> 1;
          x = k & 1;
        } else {
          j = m2 + (k - 2 * m2);
          x = nt[0] > nt[1] ? 0 : 1;
        }
      };
      // the last operation of its kind on kv tile j (then the slot can go back)
      auto last_on_tile = [&](int j, int x) { return x == 1 || j >= nt[1]; };
      ok = mbar_wait_bounded(smem_u32(qfull), 0, p.wait_limit_ns);
      int ks = 0, kp = 0;  // next S product, next PV product
      uint64_t t_idle = 0;
      int idle = 0;        // polls since the last issue (the timer is read every 64)
      while (ok && kp < total) {
        bool did = false;
        if (ks < total) {
          int j, x;
          op_at(ks, j, x);
          const int c = 2 * j, s = c % R;
          // S_x(j) overwrites P_x(j-1): O_x += P_x(j-1) V must be done
          if (mbar_test_wait(smem_u32(full + s), (c / R) & 1) &&
              (j == 0 || mbar_test_wait(smem_u32(pvdone + x), (j - 1) & 1))) {
            tc::fence_after_sync();
            const uint64_t qd = tc::sw128_desc(q_a + x * S::kQBytes, 16, 1024);
            const uint64_t kd = tc::sw128_desc(ring_a + s * S::kSlotBytes, 16, 1024);
            const uint32_t d = tmem + x * S::kTileCols + S::kS;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              // descriptor start addresses advance in 16-byte units
              const uint32_t qo = ((kk >> 2) * kTileRows * 128 + (kk & 3) * 32) >> 4;
              const uint32_t ko = ((kk >> 2) * S::kChunkStride + (kk & 3) * 32) >> 4;
              tc::mma_f16(d, qd + qo, kd + ko, kIdS, kk > 0 ? 1u : 0u);
            }
            tc::commit(smem_u32(sfull + x));
            if (last_on_tile(j, x)) tc::commit(smem_u32(empty + s));
            ++ks;
            did = true;
          }
        }
        if (kp < ks) {
          int j, x;
          op_at(kp, j, x);
          const int c = 2 * j + 1, s = c % R;
          if (mbar_test_wait(smem_u32(pfull + x), j & 1) && mbar_test_wait(smem_u32(full + s), (c / R) & 1)) {
            tc::fence_after_sync();
            const uint64_t vd = tc::sw128_desc(ring_a + s * S::kSlotBytes, S::kChunkStride, 1024);
            const uint32_t d = tmem + x * S::kTileCols + S::kO;
            const uint32_t pa = tmem + x * S::kTileCols + S::kS;  // P: 8 columns per 16 tokens
#pragma unroll
            for (int kk = 0; kk < kKv / 16; ++kk)
              tc::mma_f16_ts(d, pa + kk * 8, vd + ((kk * 2048) >> 4), kIdO, (j > 0 || kk > 0) ? 1u : 0u);
            tc::commit(smem_u32(pvdone + x));
            if (last_on_tile(j, x)) tc::commit(smem_u32(empty + s));
            ++kp;
            did = true;
          }
        }
        if (did) {
          idle = 0;
        } else if ((++idle & 63) == 0) {  // a bounded wait: no issue for wait_limit_ns gives up
          const uint64_t now = global_timer_ns();
          if (idle == 64) t_idle = now;
          else if (now - t_idle > p.wait_limit_ns) ok = false;
        }
      }
      tc::commit(smem_u32(fin));  // every MMA issued above, on every path
    }
    __syncwarp();
    ok = __shfl_sync(kFullMask, ok ? 1 : 0, 0) != 0;
  } else if (warp >= 2 + 4 * kTiles && n_tiles > 0) {
    // ------------------------------- widening -------------------------------
    const int r = threadIdx.x - (2 + 4 * kTiles) * 32;  // row of the kv tile
    constexpr int kRawChunks = D / 16;                  // 16-byte chunks of a row of codes
    for (int c = 0; c < 2 * n_tiles; ++c) {
      const int j = c >> 1, rs = c % RR, s = c % R;
      if (!wait_warp(rfull + rs, (c / RR) & 1)) {
        ok = false;
        break;
      }
      if (!wait_warp(empty + s, ((c / R) & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (!(c & 1) && warp == 2 + 4 * kTiles) {
        if (lane < kOctets) {
          const float* of = scales + (j % kScaleTiles) * 2 * kOctets + lane;
          const float ks = scale_in_range(of[0]), vs = scale_in_range(of[kOctets]);
          factors[(j % kFactorTiles) * kOctets + lane] = make_float4(ks, lg2(vs) + kWeightShift, __frcp_rn(vs), 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(ffull + j % kFactorTiles));
      }
      const uint8_t* src = raw + rs * S::kRawBytes + (r >> 4) * G8::kTileBytes;
      uint8_t* dst = ring + s * S::kSlotBytes + r * 128;
      const bool zero = (c & 1) && j * kKv + r >= kv_end;  // V rows past the context may hold anything
      uint32_t full_code = 0u;  // 0x80 in a byte: a NaN code, 0x7f or 0xff, was there
#pragma unroll
      for (int ch = 0; ch < kRawChunks; ++ch) {
        const uint4 x = zero ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(src + code_offset<D>(r & 15, ch));
        if (c & 1) {
          full_code |= ((x.x & 0x7f7f7f7fu) + 0x01010101u) | ((x.y & 0x7f7f7f7fu) + 0x01010101u) |
                       ((x.z & 0x7f7f7f7fu) + 0x01010101u) | ((x.w & 0x7f7f7f7fu) + 0x01010101u);
        }
        uint4 lo, hi;
        e4m3x4_to_f16x2x2(x.x, lo.x, lo.y);
        e4m3x4_to_f16x2x2(x.y, lo.z, lo.w);
        e4m3x4_to_f16x2x2(x.z, hi.x, hi.y);
        e4m3x4_to_f16x2x2(x.w, hi.z, hi.w);
        uint8_t* to = dst + (ch >> 2) * S::kChunkStride;
        const int c16 = (2 * ch) & 7;
        *reinterpret_cast<uint4*>(to + ((c16 ^ (r & 7)) << 4)) = lo;
        *reinterpret_cast<uint4*>(to + (((c16 + 1) ^ (r & 7)) << 4)) = hi;
      }
      if (full_code & 0x80808080u) {
        // NaN would reach rows that do not see this token (zero times NaN): it goes into the products as zero, and rows
        // from this token on get it at their end
        for (int d = 0; d < D; ++d) {
          if ((src[code_offset<D>(r & 15, d >> 4) + (d & 15)] & 0x7f) != 0x7f) continue;
          atomicMin(nan_from + d, j * kKv + r);
          info[2] = 1;
          *reinterpret_cast<uint16_t*>(dst + (d >> 6) * S::kChunkStride + ((((d >> 3) & 7) ^ (r & 7)) << 4) + (d & 7) * 2) = 0;
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(full + s));
        mbar_arrive(smem_u32(rempty + rs));
      }
    }
  } else if (warp >= 2 && n_tiles > 0) {
    // ------------------------------- softmax --------------------------------
    const int x = (warp - 2) >> 2;           // this warp's Q tile
    const int quarter = warp & 3;            // the TMEM lanes this warp reaches
    const int r = quarter * 32 + lane;       // this thread's row of the tile
    const int rowg = row0 + x * kTileRows + r;
    const bool valid = rowg < n_rows;
    const int tok = valid ? rowg / G : 0;
    const int gh = valid ? rowg - tok * G : 0;
    const int pos = valid ? pos0 + tok : 0;  // padding rows see token 0 only (output dropped)
    const uint32_t trow = tmem + x * S::kTileCols + (static_cast<uint32_t>(quarter * 32) << 16);
    float sl2;  // of a raw score, without the block's scale; positive
    {
      uint8_t* qx = q_s + x * S::kQBytes;
      const T* qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(s0 + tok) * p.q_st + static_cast<int64_t>(kvh * G + gh) * p.q_sh;
      uint4 v[D / 8];
      uint32_t most = 0u;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        v[i] = valid ? load8(qrow + 8 * i, sp.q_vec) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) most = max(most, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      // largest magnitude to 2^14 .. 2^15 (exponent fields of binary32); a negative scale's sign goes to the query, a
      // scale of zero makes the scores zero
      const uint16_t top_bits = static_cast<uint16_t>(most);
      const float top = to_f32(*reinterpret_cast<const T*>(&top_bits));
      const int field = min(max(127 + 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
      float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
      sl2 = p.scale_log2 == 0.f ? 1.f : __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * fabsf(p.scale_log2);
      up = p.scale_log2 < 0.f ? -up : p.scale_log2 == 0.f ? 0.f : up;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const T* q2 = reinterpret_cast<const T*>(&w[e]);
          f[e] = h2(to_f32(q2[0]) * up, to_f32(q2[1]) * up);
        }
        *reinterpret_cast<uint4*>(qx + (i >> 3) * (kTileRows * 128) + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
            make_uint4(f[0], f[1], f[2], f[3]);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(qfull));
    }
    float m = -INFINITY, l = 0.f;
    const int ntx = x ? nt[1] : nt[0];
    constexpr int kRuns = 32 / RUN;  // of 32 columns
    for (int j = 0; j < ntx; ++j) {
      const float4* of = factors + (j % kFactorTiles) * kOctets;
      if (!wait_warp(ffull + j % kFactorTiles, (j / kFactorTiles) & 1) || !wait_warp(sfull + x, j & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const int t0 = j * kKv;
      // tokens past pos are the causal edge, or were never staged
      const bool edge = t0 + kKv - 1 > pos;
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[32];
        tc::ld32(trow + S::kS + 32 * q, v);
        tc::wait_ld();
        if (edge) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = t0 + 32 * q + i <= pos ? v[i] : -INFINITY;
        }
#pragma unroll
        for (int g = 0; g < kRuns; ++g) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < RUN; i += 2) top = max3f(top, v[RUN * g + i], v[RUN * g + i + 1]);
          const float4 f = of[(32 * q + RUN * g) / 8];
          mx = fmaxf(mx, fmaf(top, fmaxf(sl2 * f.x, 1e-37f), f.y));  // positive: minus infinity stays
        }
      }
      float alpha = 1.f;
      if (mx - kWeightShift > m + kRescale) {  // also the first kv tile (m = -inf): token 0 is always seen
        alpha = ex2_approx(m - (mx - kWeightShift));
        m = mx - kWeightShift;
      }
      l *= alpha;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[32];
        tc::ld32(trow + S::kS + 32 * q, v);
        tc::wait_ld();
        if (edge) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = t0 + 32 * q + i <= pos ? v[i] : -INFINITY;
        }
        uint32_t w[16];
#pragma unroll
        for (int g = 0; g < kRuns; ++g) {
          const float4 f = of[(32 * q + RUN * g) / 8];
          const float by = fmaxf(sl2 * f.x, 1e-37f), add = f.y - m;
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < RUN; i += 2) {
            const float a = ex2_approx(fmaf(v[RUN * g + i], by, add)), c = ex2_approx(fmaf(v[RUN * g + i + 1], by, add));
            sum[0] += a, sum[1] += c;
            w[(RUN * g + i) / 2] = h2(a, c);
          }
          l = fmaf(sum[0] + sum[1], f.z, l);
        }
        // P takes columns 16q .. 16q + 15, whose scores have been read
        tc::st16(trow + S::kS + 16 * q, w);
      }
      if (j > 0 && __any_sync(kFullMask, alpha != 1.f)) {
        // O is at rest: its last product completed before S_j was issued
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::ld32(trow + S::kO + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tc::st32(trow + S::kO + 32 * c, o);
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(pfull + x));
    }
    if (ok && ntx > 0) ok = wait_warp(pvdone + x, (ntx - 1) & 1);  // this tile's last PV product
    if (ok && ntx > 0) {
      tc::fence_after_sync();
      const float inv = 1.f / l;
      T* orow = static_cast<T*>(p.out) + static_cast<int64_t>(s0 + tok) * p.o_st + static_cast<int64_t>(kvh * G + gh) * p.o_sh;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tc::ld32(trow + S::kO + 32 * c, o);
        tc::wait_ld();
        if (valid) {
          if (info[2]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = nan_from[32 * c + i] <= pos ? NAN : o[i];
          }
#pragma unroll
          for (int q8 = 0; q8 < 4; ++q8) store8(orow + 32 * c + 8 * q8, o + 8 * q8, inv, sp.o_vec);
        }
      }
    }
  }
  if (!ok && lane == 0) atomicOr(p.err, kErrWaitTimeout);

  // ---- teardown: every MMA has completed before the columns are freed
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    if (n_tiles > 0) wait_warp(fin, 0);
    tc::fence_after_sync();
    tc::dealloc(tmem, S::kTmemCols);
  }
}

template <typename T, int D, int RUN>
int launch_inst(const CUtensorMap& kmap, const CUtensorMap& vmap, const ScaledPrefillParams& p, int64_t blocks, cudaStream_t stream) {
  using S = Shape<D>;
  static std::atomic<int> configured[64];
  const int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&prefill_block_scaled_kernel<T, D, RUN>), S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(&prefill_block_scaled_kernel<T, D, RUN>, dim3(static_cast<unsigned>(blocks * p.base.num_kv_heads)),
                          dim3(kThreads), S::kSmem, 0, stream, kmap, vmap, p);
}

template <typename T>
int launch_type(int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap, const ScaledPrefillParams& p, int64_t blocks,
                cudaStream_t stream) {
  if (head_dim == 64) return launch_inst<T, 64, 16>(kmap, vmap, p, blocks, stream);
  if (head_dim == 128 && p.base.log2_bs < 4) return launch_inst<T, 128, 8>(kmap, vmap, p, blocks, stream);
  if (head_dim == 128) return launch_inst<T, 128, 16>(kmap, vmap, p, blocks, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

int launch_prefill_block_scaled(int dtype, int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                const ScaledPrefillParams& p, int64_t num_tokens, int64_t num_seqs, cudaStream_t stream) {
  // an upper bound on the row blocks: sum_b ceil(n_b G / 256) <= ceil(T G / 256) + B
  const int64_t blocks = (num_tokens * p.base.group + kRows - 1) / kRows + num_seqs;
  if (blocks <= 0) return cudaSuccess;
  const int e = dtype == 2 ? launch_type<__nv_bfloat16>(head_dim, kmap, vmap, p, blocks, stream)
                           : launch_type<__half>(head_dim, kmap, vmap, p, blocks, stream);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
