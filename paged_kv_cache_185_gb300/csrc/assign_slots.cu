// assign_slots.cu -- block tables, slots, positions and packed starts of the
// tokens that each sequence is to get next, from lengths and a stack of free
// blocks on the device.
//
// Mathematics: with held_b = ceil(L_b / bs) and need_b = ceil((L_b + n_b) / bs)
// - held_b, everything follows from prefix sums over the sequences: of the blocks
// that ended sequences give back (their places on the stack), of the tokens
// wanted and of the blocks needed (who is served, and which places of the stack
// are whose), and of the tokens granted (the packed starts).  A row finds its
// sequence by a binary search in the starts.
//
// Work split: one cluster of 16 CTAs.  Every CTA makes all the sums for
// itself (a thousand sequences are one load a thread and two scans), keeps starts,
// lengths and places of the stack in shared memory, and then takes its share of
// the rows and table entries; so nothing is exchanged but one cluster barrier,
// which parts what is read from what is written in place (lengths, the count, the
// stack).  Only where a row that is given back turns out to hold entries that name no
// block does the stack get shorter behind the sums: it is then closed up and they are
// made again.  A lane takes two rows at once (their searches and look-ups overlap), a
// warp four rounds of table entries.  Bound: latency, a chain of dependent reads
// (length, stack entry, table) between barriers, and with many rows the stores of 16
// SMs: 32 sequences with a token each 3.9 us, 512 with 7900 new tokens and 24 that
// end 6.2, 40 prompts in 65536 rows 5.9.  With 8 CTAs 3.8, 8.8 and 8.1; with one
// 4.1, 18.6 and 38 (before rows that are given back were looked through: 3.8, 5.9 and
// 5.7 with 16).
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace wllm {
namespace {

constexpr int kSlotThreads = 1024;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr int kSlotCtas = 16;
constexpr int kRowsTogether = 2;

__device__ __forceinline__ long long up(long long x, int d) { return __shfl_up_sync(kFullMask, x, d); }

// Exclusive sums over the block's threads; *total: of all of them.  `room` is
// shared memory for one element a warp and one more; a warp that is not `used`
// has zeros only.
template <int N>
__device__ __forceinline__ void block_scan(long long (&x)[N], long long (&total)[N], long long* room, bool used) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) in[i] = x[i];
#pragma unroll
  for (int d = 1; d < 32 && used; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long y = up(x[i], d);
      if (lane >= d) x[i] += y;
    }
  __syncthreads();  // the room's last use
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) room[i * (kSlotWarps + 1) + warp] = x[i];
  __syncthreads();
  if (warp < N) {
    const long long mine = room[warp * (kSlotWarps + 1) + lane];
    long long y = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long z = up(y, d);
      if (lane >= d) y += z;
    }
    __syncwarp();
    room[warp * (kSlotWarps + 1) + lane] = y - mine;
    if (lane == 31) room[warp * (kSlotWarps + 1) + 32] = y;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = room[i * (kSlotWarps + 1) + 32];
    x[i] += room[i * (kSlotWarps + 1) + warp] - in[i];
  }
}

// What sequence b asks for; `valid`: L + n tokens fit its row of the table.
struct Ask {
  int len, held, need, want;
  bool ended, valid, bad;
};

__device__ __forceinline__ Ask ask_of(const SlotsParams& p, int b) {
  const int len = p.context_lens[b], n = p.new_tokens[b];
  Ask a{len, 0, 0, 0, n < 0, false, false};
  const bool known = len >= 0 && len <= p.max_tokens;
  const int round = (1 << p.log2_bs) - 1;
  if (known) a.held = static_cast<int>((static_cast<long long>(len) + round) >> p.log2_bs);
  a.valid = known && !a.ended && static_cast<long long>(len) + n <= p.max_tokens;
  a.bad = !known || (!a.ended && !a.valid);
  if (a.valid) {
    a.want = n;
    a.need = static_cast<int>((static_cast<long long>(len) + n + round) >> p.log2_bs) - a.held;
  }
  return a;
}

// A warp copies n entries, the loads of several rounds together; whether one of this
// lane's is negative.
__device__ __forceinline__ bool copy_entries(int32_t* to, const int32_t* from, int from_step, int n, int lane) {
  constexpr int kRounds = 4;
  bool negative = false;
  for (int k0 = lane; k0 < n; k0 += 32 * kRounds) {
    int32_t v[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (k0 + 32 * i < n) v[i] = from[(k0 + 32 * i) * from_step];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (k0 + 32 * i < n) to[k0 + 32 * i] = v[i], negative |= v[i] < 0;
  }
  return negative;
}

__global__ void __launch_bounds__(kSlotThreads) assign_slots_kernel(const SlotsParams p) {
  extern __shared__ __align__(16) int32_t table_of_seqs[];  // [B+1] starts, [B] lengths, [B] places of the stack
  __shared__ long long room[3 * (kSlotWarps + 1)];
  __shared__ int kept;  // entries of the stack once it has been closed up; -1: it need not be, -2: it has to be
  int32_t* starts = table_of_seqs;
  int32_t* lens = starts + p.num_seqs + 1;
  int32_t* tops = lens + p.num_seqs;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) kept = -1;
  cluster.barrier_arrive();  // behind it every CTA of the cluster has begun, and its `kept` is set
  grid_wait();
  grid_launch_dependents();

  // this thread's sequences, one after another
  const int per = (p.num_seqs + kSlotThreads - 1) / kSlotThreads;
  const int b0 = min(tid * per, p.num_seqs), b1 = min(b0 + per, p.num_seqs);
  const int stored = *p.num_free;
  long long sum[3] = {0, 0, 0}, total[3];  // blocks given back, tokens wanted, blocks needed
  bool bad = false;
  Ask first{};  // of b0, which is all of them up to 1024 sequences
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, b);
    if (b == b0) first = a;
    bad |= a.bad;
    sum[0] += a.ended ? a.held : 0;
    sum[1] += a.want;
    sum[2] += a.need;
  }
  const bool used = (tid & ~31) * per < p.num_seqs;
  block_scan<3>(sum, total, room, used);
  const int had = min(max(stored, 0), p.free_room);
  int count = static_cast<int>(min(static_cast<long long>(had) + total[0], static_cast<long long>(p.free_room)));
  if (rank == 0 && (bad || (tid == 0 && (stored != had || had + total[0] > p.free_room)))) atomicOr(p.err, kErrLen);

  const int warps = ctas * kSlotWarps, warp = (tid >> 5) * ctas + rank;
  const int round = (1 << p.log2_bs) - 1;
  long long all[2];  // tokens and blocks granted
  // who is served of `count` free blocks
  const auto serve = [&](int count) {
    long long got[2] = {0, 0}, back = sum[0], want = sum[1], need = sum[2];
    for (int b = b0; b < b1; ++b) {
      const Ask a = b == b0 ? first : ask_of(p, b);
      want += a.want, need += a.need;
      const bool served = a.valid && want <= p.num_rows && (a.need == 0 || need <= count);
      lens[b] = a.len;
      // the place of its first block; of an ended sequence: where its blocks go, as -1 - place
      tops[b] = a.ended ? -1 - static_cast<int>(min(had + back, static_cast<long long>(p.free_room))) : static_cast<int>(count - 1 - (need - a.need));
      if (a.ended) back += a.held;
      got[0] += served ? a.want : 0;
      got[1] += served ? a.need : 0;
    }
    block_scan<2>(got, all, room, used);
    long long w = sum[1], r = sum[2];
    int at = static_cast<int>(got[0]);
    for (int b = b0; b < b1; ++b) {
      const Ask a = b == b0 ? first : ask_of(p, b);
      w += a.want, r += a.need;
      const bool served = a.valid && w <= p.num_rows && (a.need == 0 || r <= count);
      starts[b] = at;
      at += served ? a.want : 0;
    }
    if (b1 == p.num_seqs && (b1 > b0 || tid == 0)) starts[p.num_seqs] = at;
    __syncthreads();
  };
  serve(count);

  // blocks of ended sequences go on the stack; a warp a sequence
  cluster.barrier_wait();
  if (total[0] > 0) {
    bool negative = false;
    for (int b = warp; b < p.num_seqs; b += warps) {
      const int len = lens[b];
      if (tops[b] >= 0 || len < 0 || len > p.max_tokens || p.new_tokens[b] >= 0) continue;
      const int32_t* row = p.block_tables + b * p.bt_stride;
      const int held = static_cast<int>((static_cast<long long>(len) + round) >> p.log2_bs), to = -1 - tops[b];
      negative |= copy_entries(p.free_blocks + to, row, 1, min(held, p.free_room - to), lane);
    }
    if (__builtin_expect(negative, 0))
      for (int r = 0; r < ctas; ++r) *cluster.map_shared_rank(&kept, r) = -2;
  }
  // everything that is written in place below has been read by every CTA, and the stack is written
  cluster.sync();
  if (__builtin_expect(total[0] > 0 && kept != -1, 0)) {
    // what names no block leaves the stack, and what is there now is granted anew
    if (rank == 0 && tid < 32) {
      int to = had;
      for (int k0 = had; k0 < count; k0 += 32) {
        const int v = k0 + lane < count ? p.free_blocks[k0 + lane] : -1;
        const unsigned good = __ballot_sync(kFullMask, v >= 0);
        if (v >= 0) p.free_blocks[to + __popc(good & ((1u << lane) - 1u))] = v;
        to += __popc(good);
      }
      if (lane < ctas) *cluster.map_shared_rank(&kept, lane) = to;
      if (lane == 0) atomicOr(p.err, kErrBlock);
    }
    cluster.sync();
    count = kept;
    serve(count);
  }

  const int rows = starts[p.num_seqs];
  const int top_step = p.num_seqs > 1 ? 1 << (31 - __clz(p.num_seqs - 1)) : 0;
  for (int b = rank * kSlotThreads + tid; b < p.num_seqs; b += ctas * kSlotThreads) {
    const int n = starts[b + 1] - starts[b], len = lens[b];
    p.starts[b] = starts[b];
    p.lens_out[b] = p.new_tokens[b] < 0 ? 0 : len + n;
  }
  if (rank == 0 && tid == 0) {
    p.starts[p.num_seqs] = rows;
    *p.free_out = count - static_cast<int>(all[1]);
  }
  // table entries of new blocks; a warp a sequence
  for (int b = warp; b < p.num_seqs; b += warps) {
    const int n = starts[b + 1] - starts[b], len = lens[b];
    if (n == 0) continue;
    const int held = static_cast<int>((static_cast<long long>(len) + round) >> p.log2_bs);
    const int end = static_cast<int>((static_cast<long long>(len) + n + round) >> p.log2_bs), top = tops[b];
    int32_t* row = p.block_tables + b * p.bt_stride;
    copy_entries(row + held, p.free_blocks + top, -1, end - held, lane);
  }
  // rows: kRowsTogether a lane, so that their searches and look-ups overlap
  const unsigned num_rows = static_cast<unsigned>(p.num_rows);
  for (unsigned t0 = warp * 32 * kRowsTogether + lane; t0 < num_rows; t0 += warps * 32 * kRowsTogether) {
    int b[kRowsTogether], at[kRowsTogether], block[kRowsTogether];
#pragma unroll
    for (int k = 0; k < kRowsTogether; ++k) b[k] = 0;
    for (int step = top_step; step > 0; step >>= 1)  // the last sequence that begins at or before the row
#pragma unroll
      for (int k = 0; k < kRowsTogether; ++k)
        if (b[k] + step < p.num_seqs && static_cast<unsigned>(starts[b[k] + step]) <= t0 + 32 * k) b[k] += step;
#pragma unroll
    for (int k = 0; k < kRowsTogether; ++k) {
      const unsigned t = t0 + 32 * k;
      at[k] = block[k] = 0;
      if (t < static_cast<unsigned>(rows)) {
        const int len = lens[b[k]];
        at[k] = len + static_cast<int>(t) - starts[b[k]];
        const int held = static_cast<int>((static_cast<long long>(len) + round) >> p.log2_bs), j = at[k] >> p.log2_bs;
        const int32_t* from = j < held ? p.block_tables + b[k] * p.bt_stride + j : p.free_blocks + (tops[b[k]] - (j - held));
        block[k] = *from;
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsTogether; ++k) {
      const unsigned t = t0 + 32 * k;
      if (t >= num_rows) break;
      const bool good = t < static_cast<unsigned>(rows) && block[k] >= 0;
      if (t < static_cast<unsigned>(rows) && !good) atomicOr(p.err, kErrBlock);
      p.slots[t] = good ? (static_cast<long long>(block[k]) << p.log2_bs) + (at[k] & round) : -1;
      if (p.positions != nullptr) p.positions[t] = at[k];
    }
  }
}

}  // namespace

int launch_assign_slots(const SlotsParams& p, cudaStream_t stream) {
  static std::atomic<int> configured[64];
  static std::atomic<bool> wide[64];  // clusters of more than 8 CTAs are allowed, per device
  int dev = 0;
  cudaError_t c = cudaGetDevice(&dev);
  if (c == cudaSuccess && !(dev < 64 && wide[dev].load(std::memory_order_acquire))) {
    c = cudaFuncSetAttribute(reinterpret_cast<const void*>(&assign_slots_kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (c == cudaSuccess && dev < 64) wide[dev].store(true, std::memory_order_release);
  }
  if (c != cudaSuccess) return c;
  const int smem = (3 * p.num_seqs + 1) * static_cast<int>(sizeof(int32_t));
  const int e0 = raise_smem_limit(configured, reinterpret_cast<const void*>(&assign_slots_kernel), smem);
  if (e0 != cudaSuccess) return e0;
  const int e = launch_dependent(&assign_slots_kernel, dim3(kSlotCtas), dim3(kSlotThreads), smem, kSlotCtas, stream, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace wllm
