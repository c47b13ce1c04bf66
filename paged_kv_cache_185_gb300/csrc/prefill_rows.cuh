// prefill_rows.cuh -- which rows a prefill CTA works on, and small helpers that the
// tcgen05 prefill kernels share.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace wllm {

constexpr int kTcSortSeqs = 64;  // batches of up to this many sequences: longest first

// The sequence (-1: none) and its row block that launch position `tgt_block` works
// on, for row blocks of `rows` query rows: sequence b owns ceil(n_b * G / rows)
// consecutive ones.  With up to kTcSortSeqs sequences they are taken longest
// context first (the block scheduler starts CTAs in launch order, so the longest
// CTAs start first and the short ones fill the end); within a sequence its last
// rows (the longest context) come first.  Called by a whole warp.
__device__ __forceinline__ void row_block_of(const PrefillParams& p, int rows, int tgt_block, int lane, int* seq_out,
                                             int* tile_out) {
  const int G = p.group;
  int seq = -1, tile = 0, base = 0;
  if (p.num_seqs <= kTcSortSeqs) {
    // lane l holds sequences l and l + 32: length (the sort key) and row blocks
    int key[2], nb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = lane + 32 * h;
      key[h] = -1;
      nb[h] = 0;
      if (b < p.num_seqs) {
        int n = p.query_start_loc[b + 1] - p.query_start_loc[b];
        n = n < 0 ? 0 : n;
        nb[h] = static_cast<int>((static_cast<int64_t>(n) * G + rows - 1) / rows);
        key[h] = p.context_lens[b];
      }
    }
    // start of each of this lane's sequences in the sorted order (ties in sequence order)
    int start[2] = {0, 0};
    for (int bb = 0; bb < p.num_seqs; ++bb) {
      const int kb = __shfl_sync(kFullMask, bb < 32 ? key[0] : key[1], bb & 31);
      const int nbb = __shfl_sync(kFullMask, bb < 32 ? nb[0] : nb[1], bb & 31);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = lane + 32 * h;
        if (kb > key[h] || (kb == key[h] && bb < b)) start[h] += nbb;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = lane + 32 * h;
      const bool hit = b < p.num_seqs && tgt_block >= start[h] && tgt_block < start[h] + nb[h];
      const unsigned m = __ballot_sync(kFullMask, hit);
      if (m != 0u) {
        const int src = __ffs(m) - 1;
        seq = src + 32 * h;
        tile = __shfl_sync(kFullMask, nb[h] - 1 - (tgt_block - start[h]), src);
      }
    }
  }
  for (int b0 = 0; b0 < p.num_seqs && seq < 0 && p.num_seqs > kTcSortSeqs; b0 += 32) {
    const int b = b0 + lane;
    int n = 0;
    if (b < p.num_seqs) n = p.query_start_loc[b + 1] - p.query_start_loc[b];
    n = n < 0 ? 0 : n;
    const int tiles = static_cast<int>((static_cast<int64_t>(n) * G + rows - 1) / rows);
    int incl = tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFullMask, incl, off);
      if (lane >= off) incl += v;
    }
    const int excl = incl - tiles;
    const int tgt = tgt_block - base;
    const unsigned hit = __ballot_sync(kFullMask, b < p.num_seqs && tgt >= excl && tgt < incl);
    if (hit != 0u) {
      const int src = __ffs(hit) - 1;
      seq = b0 + src;
      const int t_in = tgt - __shfl_sync(kFullMask, excl, src);
      const int t_all = __shfl_sync(kFullMask, tiles, src);
      tile = t_all - 1 - t_in;  // the sequence's last rows (longest context) first
    }
    base += __shfl_sync(kFullMask, incl, 31);
  }
  *seq_out = seq;
  *tile_out = tile;
}

// max(a, b, c) in one three-input max.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

}  // namespace wllm
