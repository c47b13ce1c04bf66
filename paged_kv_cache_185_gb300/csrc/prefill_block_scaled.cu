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
// numbers of f16 down to 2^-21.  They go to the products as two words of f16 (what the
// first leaves off is the second): 22 bits, or 2^-32 of the largest.  One word put up to
// 2^-12 of each weight into the output, as much as the rounding of an f16 output; the
// second costs 24 us of the 410 of 8 chunks of 1024 (below) to make and 57 to multiply,
// and 8 of the 85 of 64 drafts.  (Cut off by a mask instead of rounded 433, with the sums of
// two at once 419 and 8 registers spilled.)  l sums the weights before they are rounded:
// behind a small vs a weight may round to nothing and still count in l.
//
// One CTA (one per SM) works on up to 256 query rows of one sequence and one kv
// head, row r being (token r / G, query head r % G of the group), over a range of
// the context in steps of 64 tokens, as two streams: with more than 128 rows stream
// x has Q tile x and every step, otherwise both have the same rows and every other
// step, and their results meet at the end.  Tensor memory holds for each stream two
// score tiles S (64 columns; the softmax writes both words of the weights P, f16, two a
// column, over them) and the output O: the scores of the step after next are computed
// while a step's weights are.  Sixteen warps:
//
//   warps 14 and 15 (producers, of every other item): the block table, each step's K
//     and V codes by TMA (16-row boxes, 128-byte swizzle) into a ring of eight raw
//     slots, in the order in which the products need them; with K both scales, by
//     4-byte asynchronous copies on the same mbarrier;
//   warps 0-3 (widening), a pair of warps a raw slot: thread r takes row r to f16,
//     which is exact, in a slot laid out for the products ([head_dim / 64][64
//     tokens][128 bytes], swizzled).  V rows past the context become zeros, and so do
//     NaN codes (their first tokens are kept, and rows that see them get NaN at the
//     end).  With K: the factors that each run of 8 tokens gives the softmax.
//     (With weights of one word: codes through registers instead of raw slots, what an SM has in flight is then
//     bound by the little L1 that is left, 490 us instead of 372 for 8 chunks of 1024.
//     A warp an item instead of a pair: 369 instead of 346, more of the few slots are
//     then being written);
//   warps 4-7 and 8-11 (softmax of stream 0 and 1): thread r owns row r;
//   warps 12 and 13 (MMA of stream 0 and 1): for each step O += P V and, once that
//     is done, the S of the step after next, which takes P's place.
// The query rows go to f16 after a power of two was divided out of each.
//
// Where the row blocks do not fill the SMs, several CTAs share a block's context
// (launch_prefill_block_scaled); their results go to the workspace, and a second
// kernel, a programmatic dependent, merges them in their order.
//
// Bound: 8 chunks of 1024 tokens behind up to 5000 earlier ones, 28/4 heads of 128,
// block_size 16 (337 GFLOP): 410 us, 822 TFLOP/s, 0.43 of the measured cuBLAS rate.
// A step of 64 tokens takes 1.19 us and moves 224 KB through shared memory (the Q tile
// for the scores, codes in and out, the products' operands, V twice), which alone takes
// 0.93; the tensor pipe is busy 51 % of the time and 63 % of the issue slots are used.
// Chunks of 5 tokens of 64 sequences (300 to 6000 tokens, same heads; 211 MB): 85 us,
// 0.37 of the copy rate: 35 of 128 rows are used, and each step waits for its codes
// to be widened.  One chunk of 100 tokens, 32/8 heads, 2100 tokens: 28 us, latency
// (look-ups, 3 us of query rows, 4 or 5 steps, 3 us of outputs, the second kernel).
//
// Every wait is bounded; on a timeout the CTA records the error, waits (bounded)
// for its MMAs in flight, frees its tensor memory and returns.
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
constexpr int kStreams = 2;
constexpr int kRows = kTileRows * kStreams;  // of a CTA
constexpr int kStep = 64;                    // tokens of a step
constexpr int kOctets = kStep / 8;
constexpr int kWideners = 4;                 // warps, in pairs
constexpr int kSoftmax = kWideners;          // first warp of the softmax
constexpr int kMma = kSoftmax + 4 * kStreams;  // first of the MMA warps, one a stream
constexpr int kProducer = kMma + kStreams;   // first of two producers
constexpr int kThreads = (kProducer + 2) * 32;
constexpr float kRescale = 8.f;              // the running maximum moves by more than this (log2) only
constexpr float kWeightShift = 7.f;
constexpr float kNone = -3.402823466e38f;    // the maximum of nothing
constexpr int kFactorSteps = 8;              // steps whose factors are kept

// The rows of one block and the context that they see.
struct Rows {
  int b, n_rows, row0, pos0, s0;
  int end[kStreams];  // tokens that a row of Q tile x sees at most (0: the tile has no row)
};
__device__ __forceinline__ Rows rows_of(const PrefillParams& p, int b, int block, bool tell) {
  Rows r{b, 0, 0, 0, 0, {0, 0}};
  if (b < 0) return r;
  const int l_max = p.max_blocks * p.block_size;
  r.s0 = p.query_start_loc[b];
  int n = p.query_start_loc[b + 1] - r.s0;
  if (r.s0 < 0 || n < 0 || static_cast<int64_t>(r.s0) + n > p.num_tokens) {  // inconsistent query starts
    if (tell) atomicOr(p.err, kErrLen);
    return r;
  }
  int L = p.context_lens[b];
  if (L < 0 || L > l_max || n > L) {
    if (tell) atomicOr(p.err, kErrLen);
    L = L < 0 ? 0 : (L > l_max ? l_max : L);
    n = n > L ? L : n;
  }
  r.n_rows = n * p.group;
  r.row0 = block * kRows;
  r.pos0 = L - n;
#pragma unroll
  for (int x = 0; x < kStreams; ++x) {  // (no rows only when n was clamped, error already flagged)
    const int rx = r.row0 + x * kTileRows;
    if (rx < r.n_rows) r.end[x] = r.pos0 + (min(r.n_rows, rx + kTileRows) - 1) / p.group + 1;
  }
  return r;
}

template <int D>
struct Shape {
  using G = Geom<uint8_t, D>;
  static constexpr int kQBytes = kTileRows * D * 2;        // [chunk][128 rows][128 B]
  static constexpr int kSlotBytes = kStep * D * 2;         // [chunk][64 tokens][128 B]
  static constexpr int kChunkStride = kStep * 128;
  static constexpr int kRawBytes = kStep * D;
  // widened K or V steps; two more, in place of the second Q tile, where there is only one
  static constexpr int kSlots = 6, kMoreSlots = 8;
  static constexpr int kRaws = 8;                          // K or V steps as codes
  static constexpr uint32_t kTmemCols = 512;
  // tensor-memory columns of stream x start at x * 256: two score tiles, O
  static constexpr int kStreamCols = 256, kO = 128;
  static_assert(kQBytes == (kMoreSlots - kSlots) * kSlotBytes, "slots in a Q tile's place");
  // K of step s + 8 is widened into the slot that K of step s + 5 (both streams have it) or s + 4 (the stream of step s has
  // it) gives back, whose product comes behind the weights of the stream's step two before: behind those of step s
  static_assert(kFactorSteps == 8 && kSlots == 6 && kMoreSlots == 8, "factors are not overwritten while they are needed");
};

template <int D>
struct Shared {
  using S = Shape<D>;
  uint8_t q[kStreams][S::kQBytes];
  uint8_t ring[S::kSlots][S::kSlotBytes];  // items; at the end stream 1's maxima, sums and output, [D][128 rows] of f32
  uint8_t raw[S::kRaws][S::kRawBytes];     // items as codes
  float4 factors[kFactorSteps][kOctets];   // ks, log2 vs, 1 / vs of each run of 8 tokens
  float scales[S::kRaws][2 * kOctets];     // K's and V's of a K item's step
  uint8_t row_field[kStreams][kTileRows];  // the exponent field of the power of two that a query row was scaled by
  int nan_from[D];                         // first token whose value is NaN
  uint64_t full[S::kMoreSlots];            // widened (widening -> MMA)
  uint64_t empty[S::kMoreSlots];           // given up by both streams (MMA -> widening)
  uint64_t raw_full[S::kRaws];             // codes and scales landed (producer -> widening)
  uint64_t raw_empty[S::kRaws];            // read (widening -> producer)
  uint64_t factors_full[kFactorSteps];     // (widening -> softmax)
  uint64_t scored[kStreams][2];            // S written (MMA -> softmax)
  uint64_t weighed[kStreams][2];           // P written, O rescaled (softmax -> MMA)
  uint64_t added[kStreams];                // a step's PV product done (MMA -> softmax, MMA); never more than one step ahead
  uint64_t finished[kStreams];             // the last one done (MMA -> softmax)
  uint64_t q_full;                         // Q written (softmax -> MMA)
  uint64_t fin;                            // every MMA of the CTA done
  uint32_t tmem;
  int any_nan;
  Rows rows;
  int step0, n_steps;                      // this CTA's range of the context
};
static_assert(sizeof(Shared<128>) <= 232448, "227 KB");
// one CTA an SM: a second one would contend for tensor memory
constexpr int shared_bytes(int d) { return d == 64 ? 119808 : static_cast<int>(sizeof(Shared<128>)); }
static_assert(sizeof(Shared<64>) <= 119808 && 2 * (119808 + 1024) > 233472, "");

// The items of a CTA's n steps, in the order of their use: K of the first `lead`
// steps, then V of a step and K of the step `lead` behind it in turn.
struct Items {
  int n, lead;
  __device__ __forceinline__ int k(int s) const { return s < lead ? s : 2 * s - lead + 1; }
  __device__ __forceinline__ int v(int s) const { return s <= n - lead ? lead + 2 * s : n + s; }
  // whether item i is V, and its step
  __device__ __forceinline__ bool is_v(int i, int* s) const {
    if (i < min(lead, n)) {
      *s = i;
      return false;
    }
    if (i < 2 * n - lead) {
      const int m = i - lead;
      *s = (m >> 1) + (m & 1 ? lead : 0);
      return !(m & 1);
    }
    *s = i - n;
    return true;
  }
};

__device__ __forceinline__ uint32_t h2(float lo, float hi) { return Mma<__half>::pack(lo, hi); }
// Two elements at once.
__device__ __forceinline__ void fma2(float& x, float& y, float by, float add) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(by), "f"(add));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// Two numbers as two words of f16 each: what rounding to the first leaves off is the second.
__device__ __forceinline__ void two_words(float x, float y, uint32_t& first, uint32_t& rest) {
  first = h2(x, y);
  const float2 taken = __half22float2(*reinterpret_cast<const __half2*>(&first));
  rest = h2(x - taken.x, y - taken.y);
}

// Token and head (of the group) of a row, and of the rows behind it: one division for all.
struct RowAt {
  int token, head;
  __device__ __forceinline__ RowAt(int row, int group) : token(row / group) { head = row - token * group; }
  __device__ __forceinline__ void advance(int rows, int group) {
    head += rows;
    while (head >= group) head -= group, ++token;
  }
};

// How many of the CTAs launched for a row block share its context: each has a step for both streams at least.
__device__ __forceinline__ int parts_of(int splits, int steps) { return min(splits, max(1, (steps + 1) / 2)); }

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
__device__ __forceinline__ void store8(T* dst, const uint4& v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(dst) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
  const PrefillParams& p = sp.base;
  extern __shared__ __align__(1024) uint8_t raw[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  // CTA i: part i % splits of kv head (i / splits) % Hkv of a row block, so that what shares a block is launched together
  const int part = static_cast<int>(blockIdx.x % sp.splits);
  const int kvh = static_cast<int>(blockIdx.x / sp.splits % p.num_kv_heads);
  const int tgt_block = static_cast<int>(blockIdx.x / sp.splits / p.num_kv_heads);
  if (warp == kProducer && lane == 0) tma_prefetch_desc(&kmap);
  if (warp == kProducer + 1 && lane == 0) tma_prefetch_desc(&vmap);
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < S::kMoreSlots; ++s) {
        mbar_init(smem_u32(sh.full + s), kWideners / 2);
        mbar_init(smem_u32(sh.empty + s), kStreams);
      }
      for (int s = 0; s < S::kRaws; ++s) {
        mbar_init(smem_u32(sh.raw_full + s), 1 + 32);
        mbar_init(smem_u32(sh.raw_empty + s), kWideners / 2);
      }
      for (int s = 0; s < kFactorSteps; ++s) mbar_init(smem_u32(sh.factors_full + s), 1);
      for (int x = 0; x < kStreams; ++x) {
        for (int h = 0; h < 2; ++h) {
          mbar_init(smem_u32(&sh.scored[x][h]), 1);
          mbar_init(smem_u32(&sh.weighed[x][h]), 4);
        }
        mbar_init(smem_u32(sh.added + x), 1);
        mbar_init(smem_u32(sh.finished + x), 1);
      }
      mbar_init(smem_u32(&sh.q_full), 4 * kStreams);
      mbar_init(smem_u32(&sh.fin), kStreams);
      fence_mbar_init();
    }
    for (int d = lane; d < D; d += 32) sh.nan_from[d] = INT_MAX;
    __syncwarp();
    grid_wait();
    int seq, block;
    row_block_of(p, kRows, tgt_block, lane, &seq, &block);
    if (lane == 0) {
      Rows r = rows_of(p, seq, block, true);
      const int steps = (max(r.end[0], r.end[1]) + kStep - 1) / kStep, parts = parts_of(sp.splits, steps);
      if (part >= parts) r.end[0] = r.end[1] = 0;  // nothing for this CTA
      sh.step0 = part < parts ? steps * part / parts : 0;
      sh.n_steps = part < parts ? steps * (part + 1) / parts - sh.step0 : 0;
      sh.rows = r, sh.any_nan = 0;
    }
  } else {
    grid_wait();
  }
  grid_launch_dependents();
  if (warp == kMma) tc::alloc(smem_u32(&sh.tmem), S::kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // starts that decrease are recorded whether or not a row block meets them, by the CTA that is launched last
  if (blockIdx.x == gridDim.x - 1) {
    for (int i = threadIdx.x; i < p.num_seqs; i += kThreads)
      if (p.query_start_loc[i + 1] < p.query_start_loc[i]) atomicOr(p.err, kErrLen);
  }

  const Rows rows = sh.rows;
  const int b = rows.b, kv_end = max(rows.end[0], rows.end[1]);
  // this CTA's steps, step0 on, and each stream's (of all of them, or every other one)
  const int step0 = sh.step0, n_steps = sh.n_steps;
  const bool same_rows = rows.end[1] == 0;
  int steps[kStreams];
#pragma unroll
  for (int x = 0; x < kStreams; ++x)
    steps[x] = same_rows ? (n_steps + 1 - x) / 2 : max(0, min(n_steps, (rows.end[x] + kStep - 1) / kStep - step0));
  const bool work = n_steps > 0;
  const Items items{n_steps, same_rows ? 4 : 2};
  uint8_t* const ring = same_rows ? sh.q[1] : sh.ring[0];
  const int slots = same_rows ? S::kMoreSlots : S::kSlots;

  // one lane waits, the warp learns the outcome
  auto wait_warp = [&](uint64_t* bar, int parity) -> bool {
    bool got = true;
    if (lane == 0) got = mbar_wait_bounded(smem_u32(bar), static_cast<uint32_t>(parity), p.wait_limit_ns);
    return __shfl_sync(kFullMask, got ? 1 : 0, 0) != 0;
  };
  // two waits, asked together by every lane: mostly both are over already, and asking takes longer than waiting
  auto wait_both = [&](uint64_t* a, int parity_a, uint64_t* b, int parity_b) -> bool {
    if (__all_sync(kFullMask, mbar_try_both(smem_u32(a), static_cast<uint32_t>(parity_a), smem_u32(b), static_cast<uint32_t>(parity_b))))
      return true;
    const bool got_a = wait_warp(a, parity_a), got_b = wait_warp(b, parity_b);
    return got_a && got_b;
  };
  bool ok = true;

  if (warp >= kProducer && work) {
    // ------------------------------- producers ------------------------------
    // Items by turns: an item's raw slot then has had the same producer (and the same pair of widening warps) before,
    // which is what makes a wait for the slot's phase before one for that phase and not the one before it.
    const int32_t* bt_row = p.block_tables + static_cast<int64_t>(b) * p.bt_stride;
    // Table entries of four steps, a lane a run of 8 tokens: those of the furthest step so far, the four before and the four
    // behind them.  The loads are unconditional (behind the end: of the last token), so nothing waits for them here.
    auto entries = [&](int group) { return bt_row[min((step0 + 4 * group) * kStep + 8 * lane, kv_end - 1) >> p.log2_bs]; };
    auto checked = [&](int entry) {
      if (entry >= 0 && entry < p.num_blocks) return entry;
      atomicOr(p.err, kErrBlock);
      return 0;
    };
    // a box a lane: 16 tokens, or 8 where blocks have no more
    constexpr int kBoxes = RUN == 8 ? kOctets : kOctets / 2;
    constexpr uint32_t kBoxBytes = RUN == 8 ? 1024u : static_cast<uint32_t>(S::G::kTileBytes);
    const int octet = RUN == 8 ? lane & 7 : (2 * lane) & 7, row_base = kvh * p.block_size;
    const float* scales_of = (lane < kOctets ? sp.k_scales : sp.v_scales) + kvh;
    int before = 0, here = checked(entries(0)), behind = entries(1), group = 0;
    int i = warp - kProducer;
    for (; i < 2 * n_steps; i += 2) {
      int s;
      const bool is_v = items.is_v(i, &s);
      if (s >> 2 > group) before = here, here = checked(behind), ++group, behind = entries(group + 1);
      const int entry = s >> 2 == group ? here : before, rs = i % S::kRaws;
      const int phys = __shfl_sync(kFullMask, entry, (s & 3) * kOctets + octet);
      const int of = __shfl_sync(kFullMask, entry, (s & 3) * kOctets + (lane & 7));
      const int t = (step0 + s) * kStep + 8 * octet, at = row_base + (t & (p.block_size - 1));
      const bool live = lane < kBoxes && t < kv_end;
      const uint32_t bytes = kBoxBytes * __popc(__ballot_sync(kFullMask, live));
      const uint32_t bar = smem_u32(sh.raw_full + rs);
      if (!wait_warp(sh.raw_empty + rs, ((i / S::kRaws) & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (live)
        tma_load_3d(smem_u32(sh.raw[rs]) + lane * kBoxBytes, is_v ? &vmap : &kmap, bar, 0, S::G::kPairRows ? at >> 1 : at, phys);
      if (!is_v && lane < 2 * kOctets)  // both scales of a run come with its K: lanes 0-7 K's, 8-15 V's
        copy4_async(smem_u32(&sh.scales[rs][lane]), scales_of + static_cast<int64_t>(of) * p.num_kv_heads);
      arrive_behind_copies(bar);
    }
    // every copy still in flight lands before the CTA may leave
    for (int u = max(i - S::kRaws, warp - kProducer); u < i; u += 2)
      if (!wait_warp(sh.raw_full + u % S::kRaws, (u / S::kRaws) & 1)) ok = false;
  } else if (warp < kWideners && work) {
    // ------------------------------- widening -------------------------------
    const int r = threadIdx.x & 63;     // row of the step
    constexpr int kRawChunks = D / 16;  // 16-byte chunks of a row of codes
    int at = warp >> 1, turn = 1;       // slot; parity of its being free
    for (int i = warp >> 1; i < 2 * n_steps; i += kWideners / 2) {
      const int rs = i % S::kRaws;
      int s;
      const bool is_v = items.is_v(i, &s);
      if (!wait_both(sh.raw_full + rs, (i / S::kRaws) & 1, sh.empty + at, turn)) {
        ok = false;
        break;
      }
      const uint8_t* src = sh.raw[rs] + (r >> 4) * S::G::kTileBytes;
      uint8_t* dst = ring + at * S::kSlotBytes + r * 128;
      const int token = (step0 + s) * kStep + r;
      uint32_t nan_bits = 0u;                     // 0x80 in a byte: a NaN code, 0x7f or 0xff, was there
      uint4 codes[kRawChunks];  // read before anything is stored, which would have to be waited for one by one
#pragma unroll
      for (int ch = 0; ch < kRawChunks; ++ch) codes[ch] = *reinterpret_cast<const uint4*>(src + code_offset<D>(r & 15, ch));
      if (is_v && token >= kv_end) {  // V rows past the context may hold anything
#pragma unroll
        for (int ch = 0; ch < kRawChunks; ++ch) codes[ch] = make_uint4(0u, 0u, 0u, 0u);
      }
      const bool factors = !is_v && !(warp & 1);
      if (factors && lane < kOctets) {
        const float ks = scale_in_range(sh.scales[rs][lane]), vs = scale_in_range(sh.scales[rs][kOctets + lane]);
        sh.factors[s % kFactorSteps][lane] = make_float4(ks, lg2(vs) + kWeightShift, __frcp_rn(vs), 0.f);
      }
#pragma unroll
      for (int ch = 0; ch < kRawChunks; ++ch) {
        uint4 x = codes[ch];
        nan_bits |= ((x.x & 0x7f7f7f7fu) + 0x01010101u) | ((x.y & 0x7f7f7f7fu) + 0x01010101u) |
                    ((x.z & 0x7f7f7f7fu) + 0x01010101u) | ((x.w & 0x7f7f7f7fu) + 0x01010101u);
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
      if (is_v && (nan_bits & 0x80808080u)) {
        // NaN would reach rows that do not see its token (zero times NaN): it goes into the products as zero, and rows
        // from this token on get it at their end
        for (int d = 0; d < D; ++d) {
          if ((src[code_offset<D>(r & 15, d >> 4) + (d & 15)] & 0x7f) != 0x7f) continue;
          atomicMin(sh.nan_from + d, token);
          sh.any_nan = 1;
          *reinterpret_cast<uint16_t*>(dst + (d >> 6) * S::kChunkStride + ((((d >> 3) & 7) ^ (r & 7)) << 4) + (d & 7) * 2) = 0;
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(sh.full + at));
        if (factors) mbar_arrive(smem_u32(sh.factors_full + s % kFactorSteps));
        mbar_arrive(smem_u32(sh.raw_empty + rs));
      }
      at += kWideners / 2;
      if (at >= slots) at -= slots, turn ^= 1;
    }
  } else if (warp >= kMma && warp < kProducer && work) {
    // --------------------------------- MMA ----------------------------------
    // The whole warp goes through the loop and one lane issues: what the products are told (descriptors, columns) is
    // then uniform over the warp, as the instruction takes it.  (One lane by itself needed 0.3 to 0.5 us for 8 products.)
    constexpr uint32_t kIdS = tc::f16_idesc(false, false, false, kTileRows, kStep);
    constexpr uint32_t kIdO = tc::f16_idesc(false, false, true, kTileRows, D);
    const int x = warp - kMma;  // this warp's stream
    const bool same = __shfl_sync(kFullMask, same_rows ? 1 : 0, 0) != 0;
    const int n = __shfl_sync(kFullMask, steps[x], 0), all = __shfl_sync(kFullMask, n_steps, 0);
    const uint32_t base = __shfl_sync(kFullMask, tmem, 0) + x * S::kStreamCols;
    const Items order{all, same ? 4 : 2};
    const uint32_t ring_a = same ? smem_u32(sh.q[1]) : smem_u32(sh.ring);
    const uint64_t qd = tc::sw128_desc(smem_u32(sh.q) + (same ? 0 : x) * S::kQBytes, 16, 1024);
    auto wait = [&](uint64_t* bar, int parity) { ok = ok && mbar_wait_warp(smem_u32(bar), static_cast<uint32_t>(parity), p.wait_limit_ns); };
    struct Slot {
      int at, turn;
    };
    auto slot_of = [&](int item) {
      return same ? Slot{item % S::kMoreSlots, item / S::kMoreSlots & 1} : Slot{item % S::kSlots, item / S::kSlots & 1};
    };
    auto step_of = [&](int i) { return same ? 2 * i + x : i; };
    // a slot goes back once both streams have given it up; where only one has it, it does so twice
    auto give_up = [&](Slot s) {
      tc::commit(smem_u32(sh.empty + s.at));
      if (same) tc::commit(smem_u32(sh.empty + s.at));
    };
    auto scores = [&](int i, int h) {
      const Slot s = slot_of(order.k(step_of(i)));
      // (behind step 1: the weights whose place it takes have been read)
      ok = i < 2 ? wait_warp(sh.full + s.at, s.turn) : wait_both(sh.full + s.at, s.turn, sh.added + x, h);
      if (!ok) return;
      tc::fence_after_sync();
      const uint64_t kd = tc::sw128_desc(ring_a + s.at * S::kSlotBytes, 16, 1024);
      if (tc::elect()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          // descriptor start addresses advance in 16-byte units
          const uint32_t qo = ((kk >> 2) * kTileRows * 128 + (kk & 3) * 32) >> 4;
          const uint32_t ko = ((kk >> 2) * S::kChunkStride + (kk & 3) * 32) >> 4;
          tc::mma_f16(base + h * kStep, qd + qo, kd + ko, kIdS, kk > 0 ? 1u : 0u);
        }
        tc::commit(smem_u32(&sh.scored[x][h]));
        give_up(s);
      }
      __syncwarp();
    };
    auto values = [&](int i, int h) {
      const Slot s = slot_of(order.v(step_of(i)));
      ok = wait_both(sh.full + s.at, s.turn, &sh.weighed[x][h], (i >> 1) & 1);
      if (!ok) return;
      tc::fence_after_sync();
      const uint64_t vd = tc::sw128_desc(ring_a + s.at * S::kSlotBytes, S::kChunkStride, 1024);
      const uint32_t go_on = i > 0 ? 1u : 0u;
      if (tc::elect()) {
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk) {  // P: 16 columns per 16 tokens, the second words behind the first
          tc::mma_f16_ts(base + S::kO, base + h * kStep + kk * 16, vd + ((kk * 2048) >> 4), kIdO, kk > 0 ? 1u : go_on);
          tc::mma_f16_ts(base + S::kO, base + h * kStep + kk * 16 + 8, vd + ((kk * 2048) >> 4), kIdO, 1u);
        }
        tc::commit(smem_u32(sh.added + x));
        if (i + 1 == n) tc::commit(smem_u32(sh.finished + x));
        give_up(s);
      }
      __syncwarp();
    };
    wait(&sh.q_full, 0);
    if (ok && n > 0) scores(0, 0);
    if (ok && n > 1) scores(1, 1);
    for (int i = 0; ok && i < n; i += 2) {
      values(i, 0);
      if (ok && i + 2 < n) scores(i + 2, 0);
      if (ok && i + 1 < n) values(i + 1, 1);
      if (ok && i + 3 < n) scores(i + 3, 1);
    }
    // steps that only the other stream has: given up once they are there
    if (!same)
      for (int i = n; ok && i < all; ++i)
        for (int v = 0; v < 2; ++v) {
          const Slot s = slot_of(v ? order.v(i) : order.k(i));
          wait(sh.full + s.at, s.turn);
          if (ok && lane == 0) mbar_arrive(smem_u32(sh.empty + s.at));
        }
    if (tc::elect()) tc::commit(smem_u32(&sh.fin));  // every MMA issued above, on every path
    __syncwarp();
  } else if (warp >= kSoftmax && warp < kMma && rows.end[0] > 0) {
    // ------------------------------- softmax --------------------------------
    const int x = (warp - kSoftmax) >> 2;    // this warp's stream
    const int quarter = warp & 3;            // the TMEM lanes this warp reaches
    const int r = quarter * 32 + lane;       // this thread's row of the Q tile
    const int rowg = rows.row0 + (same_rows ? 0 : x * kTileRows) + r;
    const bool valid = rowg < rows.n_rows;
    const int tok = min(rowg, rows.n_rows - 1) / G;  // (a row behind the last sees what the last does; its output is dropped)
    const int gh = rowg - tok * G;
    const int pos = rows.pos0 + tok;
    const uint32_t trow = tmem + x * S::kStreamCols + (static_cast<uint32_t>(quarter * 32) << 16);
    // The warp's 32 rows are read together, kLanes lanes a row (each two pieces of 16 bytes), so that a load touches few lines.
    constexpr int kLanes = D / 16, kRowsAtOnce = 32 / kLanes;
    const int first_row = rows.row0 + (same_rows ? 0 : x * kTileRows) + quarter * 32, sub = lane / kLanes, piece = lane % kLanes;
    {
      // The rows go to shared memory as they are and every lane rewrites its own pieces: rolled loops, because
      // straight-line code runs once and is fetched more slowly than it runs.  Rows that both streams have are halved
      // between them.
      uint8_t* const qx = sh.q[same_rows ? 0 : x];
      const int rows_here = same_rows ? 16 : 32, in_tile = quarter * 32 + (same_rows ? 16 * x + sub : sub);
      const auto place = [&](int rr, int k) {
        const int c = piece + k * kLanes;
        return reinterpret_cast<uint4*>(qx + (c >> 3) * (kTileRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
      };
      const int first = rows.row0 + (same_rows ? 0 : x * kTileRows) + in_tile;
      const float sign = p.scale_log2 < 0.f ? -1.f : p.scale_log2 == 0.f ? 0.f : 1.f;
      {
        const int token = first / G;
        int head = first - token * G;
        const T* from = static_cast<const T*>(p.q) + static_cast<int64_t>(rows.s0 + token) * p.q_st +
                        static_cast<int64_t>(kvh * G + head) * p.q_sh + 8 * piece;
        // kRowsAtOnce rows on: so many heads, or a token more and as many less than the group
        const int heads_on = kRowsAtOnce % G;
        const int64_t on = kRowsAtOnce / G * p.q_st + heads_on * p.q_sh, over = p.q_st - G * p.q_sh;
        if (sp.q_vec) {
#pragma unroll 2
          for (int j = 0; j < rows_here; j += kRowsAtOnce) {  // (zeros behind the last row)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(in_tile + j, k))),
                           "l"(from + k * 8 * kLanes), "r"(first + j < rows.n_rows ? 16 : 0) : "memory");
            head += heads_on, from += on;
            if (head >= G) head -= G, from += over;
          }
        } else {
          for (int j = 0; j < rows_here; j += kRowsAtOnce) {
            for (int k = 0; k < 2; ++k)
              *place(in_tile + j, k) = first + j < rows.n_rows ? load8(from + k * 8 * kLanes, false) : make_uint4(0u, 0u, 0u, 0u);
            head += heads_on, from += on;
            if (head >= G) head -= G, from += over;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      constexpr int kTogether = 2;  // rows of a lane whose steps overlap
#pragma unroll 1
      for (int j = 0; j < rows_here; j += kTogether * kRowsAtOnce) {
        uint4 v[kTogether][2];
        uint32_t most[kTogether];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
          most[u] = 0u;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 c = v[u][k] = *place(in_tile + j + u * kRowsAtOnce, k);
            most[u] = __vmaxu2(most[u], __vmaxu2(__vmaxu2(c.x & 0x7fff7fffu, c.y & 0x7fff7fffu), __vmaxu2(c.z & 0x7fff7fffu, c.w & 0x7fff7fffu)));
          }
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
          for (int u = 0; u < kTogether; ++u) most[u] = __vmaxu2(most[u], __shfl_xor_sync(kFullMask, most[u], d));
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
          // largest magnitude to 2^14 .. 2^15 (exponent fields of binary32); a negative scale's sign goes to the query, a
          // scale of zero makes the scores zero
          const uint16_t top_bits = static_cast<uint16_t>(max(most[u] & 0xffffu, most[u] >> 16));
          const float top = to_f32(*reinterpret_cast<const T*>(&top_bits));
          const int field = min(max(127 + 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
          const float up = __uint_as_float(static_cast<uint32_t>(field) << 23) * sign;
          const int rr = in_tile + j + u * kRowsAtOnce;
          if (piece == 0) sh.row_field[same_rows ? 0 : x][rr] = static_cast<uint8_t>(field);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {v[u][k].x, v[u][k].y, v[u][k].z, v[u][k].w};
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const T* q2 = reinterpret_cast<const T*>(&w[e]);
              f[e] = h2(to_f32(q2[0]) * up, to_f32(q2[1]) * up);
            }
            *place(rr, k) = make_uint4(f[0], f[1], f[2], f[3]);
          }
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.q_full));
      if (same_rows) asm volatile("bar.sync 1, %0;" ::"r"(4 * kStreams * 32) : "memory");
    }
    // of a raw score, without the block's scale: what undoes the row's, times the scale's magnitude; positive
    const float sl2 = p.scale_log2 == 0.f ? 1.f
                                          : fminf(__uint_as_float((254u - sh.row_field[same_rows ? 0 : x][r]) << 23) * fabsf(p.scale_log2),
                                                  kMostRowFactor);
    float m = kNone, l = 0.f;
    const int n = steps[x];
    // rows behind the last get no weights: what the products make of the places they leave stays in such rows
    const bool idle = first_row >= rows.n_rows;
    constexpr int kRuns = kStep / RUN;
    for (int i = 0; i < n; ++i) {
      const int h = i & 1, s = same_rows ? 2 * i + x : i;  // step, counted from step0
      const float4* of = sh.factors[s % kFactorSteps];
      if (!wait_both(sh.factors_full + s % kFactorSteps, (s / kFactorSteps) & 1, &sh.scored[x][h], (i >> 1) & 1)) {
        ok = false;
        break;
      }
      if (idle) {
        if (lane == 0) mbar_arrive(smem_u32(&sh.weighed[x][h]));
        continue;
      }
      tc::fence_after_sync();
      float v[2][32];
      tc::ld32(trow + h * kStep, v[0]);
      tc::ld32(trow + h * kStep + 32, v[1]);
      tc::wait_ld();
      const int t0 = (step0 + s) * kStep;
      if (t0 + kStep - 1 > pos) {  // the causal edge (and tokens that were never staged)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[q][e] = t0 + 32 * q + e <= pos ? v[q][e] : -INFINITY;
      }
      float by[kRuns], add[kRuns], mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < kRuns; ++g) {
        const float4 f = of[g * (RUN / 8)];
        by[g] = fmaxf(sl2 * f.x, 1e-37f);  // positive: minus infinity stays
        add[g] = f.y;
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < RUN; e += 2) top = max3f(top, v[(RUN * g + e) >> 5][(RUN * g + e) & 31], v[(RUN * g + e) >> 5][(RUN * g + e + 1) & 31]);
        mx = fmaxf(mx, fmaf(top, by[g], add[g]));
      }
      float alpha = 1.f;
      if (mx - kWeightShift > m + kRescale) {  // also a row's first token
        alpha = ex2_approx(m - (mx - kWeightShift));
        m = mx - kWeightShift;
      }
      l *= alpha;
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // 32 tokens: for 16 of them 8 columns of first words, then 8 of second ones
        uint32_t w[32];
#pragma unroll
        for (int g = q * kRuns / 2; g < (q + 1) * kRuns / 2; ++g) {
          const float a = add[g] - m;
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int e = 0; e < RUN; e += 2) {
            const int t = (RUN * g + e) & 31, at = t >> 4 << 4 | (t & 15) >> 1;
            float y0 = v[q][t], y1 = v[q][t + 1];
            fma2(y0, y1, by[g], a);
            y0 = ex2_approx(y0), y1 = ex2_approx(y1);
            add2(s0, s1, y0, y1);
            two_words(y0, y1, w[at], w[at + 8]);
          }
          l = fmaf(s0 + s1, of[g * (RUN / 8)].z, l);
        }
        tc::st32(trow + h * kStep + 32 * q, *reinterpret_cast<const float(*)[32]>(&w));  // over the scores
      }
      if (__any_sync(kFullMask, alpha != 1.f) && i > 0) {
        // O is rescaled at rest: behind the product of the step before
        if (!wait_warp(sh.added + x, (i - 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::ld32(trow + S::kO + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tc::st32(trow + S::kO + 32 * c, o);
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.weighed[x][h]));
    }
    if (ok && n > 0) ok = wait_warp(sh.finished + x, 0);
    tc::fence_after_sync();
    // rows that both streams have: stream 1 leaves its results in the ring, which nothing reads any more
    float mine = 1.f, other = 0.f;
    float* left = reinterpret_cast<float*>(sh.ring);  // [D][128 rows], then maxima and sums
    static_assert((D + 2) * kTileRows * 4 <= S::kSlots * S::kSlotBytes, "the ring has room");
    const bool both = same_rows && steps[1] > 0;
    if (same_rows) {
      asm volatile("bar.sync 1, %0;" ::"r"(4 * kStreams * 32) : "memory");
      if (x == 1) {
        left[D * kTileRows + r] = m, left[(D + 1) * kTileRows + r] = l;
#pragma unroll 1
        for (int c = 0; both && c < D / 32; ++c) {
          float o[32];
          tc::ld32(trow + S::kO + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) left[(32 * c + e) * kTileRows + r] = o[e];
        }
      }
      asm volatile("bar.sync 1, %0;" ::"r"(4 * kStreams * 32) : "memory");
      if (x == 0 && both) {
        const float m2 = left[D * kTileRows + r], top = fmaxf(m, m2);
        mine = ex2_approx(m - top), other = ex2_approx(m2 - top);
        l = fmaf(l, mine, other * left[(D + 1) * kTileRows + r]);
        m = top;
      }
    }
    if (ok && !idle && (x == 0 || !same_rows)) {
      const float inv = sp.splits > 1 ? 1.f : 1.f / l;
      const bool any_nan = sh.any_nan != 0;
      // where this lane's pieces go, of rows lane / 8 + 4 i
      int64_t to[8];
      {
        RowAt at(first_row + (lane >> 3), G);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          to[i] = sp.splits > 1 ? ((static_cast<int64_t>(rows.s0 + at.token) * p.num_q_heads + kvh * G + at.head) * sp.splits + part) * (D + 4)
                                : static_cast<int64_t>(rows.s0 + at.token) * p.o_st + static_cast<int64_t>(kvh * G + at.head) * p.o_sh;
          at.advance(4, G);
        }
      }
      // 64 columns of the warp's rows at a time (of partial results 32), through shared memory (Q's place, which nothing
      // reads any more): [32 rows][8 pieces], piece c at c ^ (row % 8)
      uint4* turn = reinterpret_cast<uint4*>(sh.q[x] + quarter * 4096);
      const auto columns = [&](int c, float (&o)[32]) {
        if (n > 0) {
          tc::ld32(trow + S::kO + 32 * c, o);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (both) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(o[e], mine, other * left[(32 * c + e) * kTileRows + r]);
        }
        if (any_nan) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = sh.nan_from[32 * c + e] <= pos ? NAN : o[e];
        }
      };
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        columns(c, o);
        const int half = sp.splits > 1 ? 0 : 4 * (c & 1);
        if (half == 0) __syncwarp();
        if (sp.splits > 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            turn[lane * 8 + (e ^ (lane & 7))] = make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                                                           __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            turn[lane * 8 + ((half + e) ^ (lane & 7))] =
                make_uint4(Mma<T>::pack(o[8 * e] * inv, o[8 * e + 1] * inv), Mma<T>::pack(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                           Mma<T>::pack(o[8 * e + 4] * inv, o[8 * e + 5] * inv), Mma<T>::pack(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
          if (half == 0) continue;
        }
        __syncwarp();
        uint4 row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = turn[(4 * i + (lane >> 3)) * 8 + ((lane & 7) ^ ((4 * i + (lane >> 3)) & 7))];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (first_row + 4 * i + (lane >> 3) >= rows.n_rows) break;
          if (sp.splits > 1)
            *reinterpret_cast<uint4*>(sp.parts + to[i] + 32 * c + 4 * (lane & 7)) = row[i];
          else
            store8(static_cast<T*>(p.out) + to[i] + 32 * (c - 1) + 8 * (lane & 7), row[i], sp.o_vec);
        }
      }
      if (sp.splits > 1 && valid) {
        float* prow = sp.parts + ((static_cast<int64_t>(rows.s0 + tok) * p.num_q_heads + kvh * G + gh) * sp.splits + part) * (D + 4);
        prow[D] = m, prow[D + 1] = l;
      }
    }
  }
  if (!ok && lane == 0) atomicOr(p.err, kErrWaitTimeout);

  // ---- teardown: every MMA has completed before the columns are freed
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    if (work) wait_warp(&sh.fin, 0);
    tc::fence_after_sync();
    tc::dealloc(tmem, S::kTmemCols);
  }
}

// Rows whose context several CTAs shared: a warp a row, the partial results in
// their order.
constexpr int kMergeWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_prefill_kernel(const ScaledPrefillParams sp) {
  const PrefillParams& p = sp.base;
  __shared__ int found[2];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA i: rows i % kParts ... of kv head and row block as the kernel before numbers them
  constexpr int kParts = 8;
  const int part = static_cast<int>(blockIdx.x % kParts), kvh = static_cast<int>(blockIdx.x / kParts % p.num_kv_heads);
  if (warp == 0) {
    int seq, block;
    row_block_of(p, kRows, static_cast<int>(blockIdx.x / kParts / p.num_kv_heads), lane, &seq, &block);
    if (lane == 0) found[0] = seq, found[1] = block;
  }
  __syncthreads();
  const Rows rows = rows_of(p, found[0], found[1], false);
  const int parts = parts_of(sp.splits, (max(rows.end[0], rows.end[1]) + kStep - 1) / kStep);
  const int end = min(rows.row0 + kRows, rows.n_rows);
  for (int i = rows.row0 + part * (kRows / kParts) + warp; i < min(end, rows.row0 + (part + 1) * (kRows / kParts)); i += kMergeWarps) {
    const int tok = i / p.group, head = kvh * p.group + (i - tok * p.group);
    const float* from = sp.parts + (static_cast<int64_t>(rows.s0 + tok) * p.num_q_heads + head) * sp.splits * (D + 4);
    // lane s has part s's maximum and sum
    const float m = lane < parts ? from[lane * (D + 4) + D] : kNone;
    const float l = lane < parts ? from[lane * (D + 4) + D + 1] : 0.f;
    float v[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
    const float f = exp2f(m - top);
    float sum = f * l;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
    for (int s0 = 0; s0 < parts; s0 += 8) {
      float x[8][D / 32];
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[s][e] = s0 + s < parts ? from[(s0 + s) * (D + 4) + lane + 32 * e] : 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float g = __shfl_sync(kFullMask, f, (s0 + s) & 31);
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          if (s0 + s < parts) v[e] = fmaf(g, x[s][e], v[e]);
      }
    }
    T* out = static_cast<T*>(p.out) + static_cast<int64_t>(rows.s0 + tok) * p.o_st + head * p.o_sh;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[lane + 32 * e] = from_f32<T>(v[e] / sum);
  }
}

template <typename T, int D, int RUN>
int launch_inst(const CUtensorMap& kmap, const CUtensorMap& vmap, const ScaledPrefillParams& p, int64_t blocks, cudaStream_t stream) {
  constexpr int kSmem = shared_bytes(D);
  static std::atomic<int> configured[64];
  int e = raise_smem_limit(configured, reinterpret_cast<const void*>(&prefill_block_scaled_kernel<T, D, RUN>), kSmem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(&prefill_block_scaled_kernel<T, D, RUN>, dim3(static_cast<unsigned>(blocks * p.base.num_kv_heads * p.splits)),
                       dim3(kThreads), kSmem, 0, stream, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  note_launch();
  if (p.splits == 1) return e;
  e = launch_dependent(&merge_prefill_kernel<T, D>, dim3(static_cast<unsigned>(blocks * p.base.num_kv_heads * 8)),
                       dim3(kMergeWarps * 32), 0, 0, stream, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename T>
int launch_type(int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap, const ScaledPrefillParams& p, int64_t blocks,
                cudaStream_t stream) {
  if (head_dim == 64) return launch_inst<T, 64, 16>(kmap, vmap, p, blocks, stream);
  if (head_dim == 128 && p.base.log2_bs < 4) return launch_inst<T, 128, 8>(kmap, vmap, p, blocks, stream);
  if (head_dim == 128) return launch_inst<T, 128, 16>(kmap, vmap, p, blocks, stream);
  return cudaErrorInvalidValue;
}

constexpr int kMostSplits = 32;  // a lane of the merge each

}  // namespace

size_t prefill_block_scaled_workspace(int num_sms) { return size_t(num_sms) * kRows * (128 + 4) * sizeof(float); }

int launch_prefill_block_scaled(int dtype, int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap, ScaledPrefillParams p,
                                int64_t num_tokens, int64_t num_seqs, int num_sms, cudaStream_t stream) {
  // The most row blocks that there can be: k chunks that are not empty have sum_b ceil(n_b G / 256) <= k + sum_b floor((n_b G
  // - 1) / 256) <= k + floor((T G - k) / 256), which grows with k.
  const int64_t most = num_tokens < num_seqs ? num_tokens : num_seqs;
  const int64_t blocks = most + (num_tokens * p.base.group - most) / kRows;
  if (blocks <= 0) return cudaSuccess;
  // CTAs for a row block's context: as many as the SMs allow, or as three quarters of them do if that makes a CTA's run
  // longer by 4 steps at most: the merge's CTAs then start beside them instead of behind them (they find no registers on an
  // SM that has one).  One chunk of 100 tokens, 32/8 heads: 7 instead of 9 CTAs a block 27.9 us instead of 32.9 (2100 tokens),
  // 9 instead of 7 103 instead of 111 (30000), one 50 (2100).  How long the contexts are only the device knows, and how many
  // of the batch's places are in use: in a batch padded to 64 places one live sequence has one CTA a block.
  const int64_t tiles = (int64_t(p.base.max_blocks) * p.base.block_size + 2 * kStep - 1) / (2 * kStep);
  const auto splits_on = [&](int64_t sms) {
    const int64_t most_splits = tiles < kMostSplits ? tiles : kMostSplits, s = sms / (blocks * p.base.num_kv_heads);
    return s > most_splits ? most_splits : s;
  };
  int64_t splits = splits_on(num_sms);
  const int64_t fewer = splits_on(num_sms * 3 / 4);
  if (fewer > 0 && 2 * tiles * (splits - fewer) <= 4 * splits * fewer) splits = fewer;
  p.splits = splits < 1 ? 1 : static_cast<int>(splits);
  return dtype == 2 ? launch_type<__nv_bfloat16>(head_dim, kmap, vmap, p, blocks, stream)
                    : launch_type<__half>(head_dim, kmap, vmap, p, blocks, stream);
}

}  // namespace wllm
