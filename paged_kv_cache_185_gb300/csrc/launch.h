// launch.h -- internal interface between the C ABI (api.cu) and the kernel
// translation units.  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <utility>

namespace wllm {

// The 256-byte per-device control block, offsets in ints: the error word;
// two spare words used only by the bounded-wait self-test (a counter that
// stays zero, and its result); the persistent scheduler's claim and finish
// counters; the fused step's 64-bit count of CTAs whose KV append is written.
constexpr int kCtrlBytes = 256;
constexpr int kSelftestNeverOffset = 8;
constexpr int kSelftestResultOffset = 9;
constexpr int kSchedNextOffset = 16;
constexpr int kSchedDoneOffset = 32;
constexpr int kGridCountOffset = 48;  // 8-byte aligned: two ints

// Kernel launches the library has issued (successful launch calls), for
// wllm_launch_count().  Every launch site calls note_launch() once per kernel.
void note_launch();

// Raise a kernel's dynamic shared-memory limit to `bytes` on the current
// device: `configured` is the kernel's own per-device record of the limit (64
// entries).  Thread-safe: the limit is raised under a lock and never lowered, so a
// thread that needs less cannot take away what another has just asked for.
inline int raise_smem_limit(std::atomic<int>* configured, const void* func, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < 64;
  if (tracked && configured[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  static std::mutex one_at_a_time;  // the limit only grows, whichever thread comes last
  std::lock_guard<std::mutex> lock(one_at_a_time);
  if (tracked && configured[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if (tracked) configured[dev].store(bytes, std::memory_order_release);
  return cudaSuccess;
}

// Launch as a programmatic dependent of the kernel before it in the stream: its
// CTAs may start early, so the kernel calls grid_wait() before it touches global
// memory.  `cluster` > 0: thread-block clusters of that many CTAs along x.
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Everything one paged-decode launch needs besides the two tensor maps.
struct DecodeParams {
  void* out;                 // [B][Hq][D]
  const void* q;             // [B][Hq][D]
  int64_t q_sb, q_sh;        // q strides (elements) of the seq and head dims
  int64_t o_sb, o_sh;        // out strides
  const int32_t* block_tables;
  int64_t bt_stride;         // elements between two sequences' tables
  const int32_t* context_lens;
  int num_seqs, num_q_heads, num_kv_heads, group;
  int head_tile, num_head_tiles;  // query heads per CTA, tiles per kv head
  int max_blocks, block_size, log2_bs, num_blocks;
  int part_tokens, max_parts;     // split-KV partition size / count
  float scale_log2;               // scale * log2(e) (times k_scale for an fp8 cache)
  float v_scale;                  // fp8 cache: factor of every output (1 otherwise)
  float* ws_o;                    // [B*Hq][max_parts][D] unnormalised partial sums
  float* ws_ml;                   // [B*Hq][max_parts][2] running max (log2 units), sum
  int* ws_count;                  // counters, zero between calls: grid kernel [B*Hkv*tiles] arrivals;
                                  // persistent kernel [2][B*Hkv*tiles] units finished, rows merged
  int* err;                       // device error word
  unsigned long long wait_limit_ns;
  int prefix_groups;              // process shared-prefix partitions once per group of sequences
};

struct AppendParams {
  const uint8_t* key;
  const uint8_t* value;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const void* slots;
  int slots_are_i64;
  int num_tokens, num_kv_heads;
  int row_bytes;                  // bytes of one cache row: head_dim * cache element size
  int64_t key_st, key_sh;         // strides in bytes
  int64_t val_st, val_sh;
  int log2_bs;
  int64_t num_slots;              // num_blocks * block_size
  int vec16;                      // rows and strides allow 16-byte copies
  int kv_fp8;                     // caches hold E4M3 codes of key * k_inv and value * v_inv
  int src_dtype;                  // fp8: key/value element type, a wllm_dtype code (0 f32, 1 f16, 2 bf16)
  float k_inv, v_inv;             // fp8: binary32 reciprocals of the scales
  int* err;
};

// Kernel variants of the decode: tensor-core (16-bit only) or fp32 FMA.
enum class DecodeVariant { kMma, kFma };

// Head tile (query heads of one KV head handled by one CTA) for a variant.
int decode_head_tile(int dtype, int head_dim, int group, DecodeVariant v, bool kv_fp8);

// Launch the decode kernel; returns a cudaError_t value.
int launch_decode(int dtype, int head_dim, DecodeVariant v, const CUtensorMap& kmap,
                  const CUtensorMap& vmap, const DecodeParams& p, cudaStream_t stream);

// Persistent warp-specialised decode (f16/bf16 only).  `separate_combine`
// appends the split-KV combine kernel (needed when a sequence can span
// several partitions and `fuse_combine` is not set).  `ap` (may be null)
// fuses the KV append in front; `fuse_combine` merges the partitions inside
// the launch, as they complete (p.ws_count must then hold the zeroed
// counters).  Either makes it a cooperative launch.
// `kv_fp8`: the caches hold E4M3 codes (head_dim 128 or 256, head tile 8);
// dtype is then the query / output type.
int launch_decode_persistent(int dtype, int head_dim, int head_tile, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const DecodeParams& p, int grid, bool separate_combine,
                             const AppendParams* ap, bool fuse_combine, bool kv_fp8, cudaStream_t stream);
int decode_persistent_occupancy(int dtype, int head_dim, int head_tile, int num_seqs, bool kv_fp8);
constexpr int kPersistentConsumers = 4;
constexpr int kPersistentMaxSeqs = 1024;      // sequences per launch (the host splits larger batches)
constexpr int kPersistentMaxParts = 256;      // partitions per sequence (the host widens partitions to fit)

int launch_append(const AppendParams& p, cudaStream_t stream);

// One-thread kernel whose two bounded waits (an mbarrier and the counter at
// ctrl[never_offset], which must stay below 1) time out after limit_ns: sets
// kErrWaitTimeout in ctrl[0], adds 1 to ctrl[sched_offset] and writes which
// waits gave up (bit 0 mbarrier, bit 1 counter) to *result (device memory).
int launch_wait_selftest(int* ctrl, int never_offset, int sched_offset, unsigned long long limit_ns, int* result,
                         cudaStream_t stream);

// Chunked-prefill (multi-query) paged attention: q/out [T][Hq][D] packed by
// sequence (query_start_loc [B+1]); each chunk is the last n_b of the
// sequence's context_lens[b] tokens and attends causally.
struct PrefillParams {
  void* out;
  const void* q;
  int64_t q_st, q_sh;             // q strides (elements) of the token and head dims
  int64_t o_st, o_sh;             // out strides
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
  int max_blocks, block_size, log2_bs, num_blocks;
  float scale_log2;               // scale * log2(e) (times k_scale for an fp8 cache)
  float v_scale;                  // fp8 cache: factor of every output (1 otherwise)
  int* err;
  unsigned long long wait_limit_ns;
};
// CTAs along x for T packed tokens of B sequences (grid y = kv heads).
int prefill_grid_x(int64_t num_tokens, int64_t num_seqs, int group);
// f16/bf16 queries (dtype code 1/2), head_dim 64 or 128; `kv_fp8`: E4M3 caches
// (head_dim 64 needs blocks of >= 16 tokens).  Returns a cudaError_t value.
int launch_prefill(int dtype, int head_dim, bool kv_fp8, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   const PrefillParams& p, int grid_x, cudaStream_t stream);

// The same operation on the fifth-generation tensor cores (tcgen05 MMAs with
// TMEM accumulators): 16-bit caches, head_dim 64 or 128, q/out rows 16-byte
// aligned (base and strides), a positive scale.  256 query rows per CTA.
int prefill_tc_grid_x(int64_t num_tokens, int64_t num_seqs, int group);
int launch_prefill_tc(int dtype, int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap,
                      const PrefillParams& p, int grid_x, cudaStream_t stream);

// The rotary append (rotate.cu): norms, rotary positions, query out, key and
// value to their slots.  Strides in elements.
constexpr int kMaxRotaryAxes = 4;
constexpr int kRotateWarps = 4;  // warps of a CTA of the form for few tokens
struct RotateParams {
  void* q_out;
  const void* q;
  const void* key;
  const void* value;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const void* slots;
  const void* positions;          // [axes][T]
  const float* cos_sin;           // [num_positions][rot_dim]: cosines, then sines
  const void* q_weight;           // [D] or null
  const void* k_weight;
  int64_t q_st, q_sh, key_st, key_sh, val_st, val_sh, qo_st, qo_sh;
  int64_t pos_sa;                 // elements between two axes' positions
  int64_t table_stride, num_positions, num_slots;
  int slots_are_i64, pos_are_i64;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, log2_bs;
  int num_axes, section_end[kMaxRotaryAxes];  // pairs below section_end[a] and not below section_end[a-1] turn by axis a
  int adjacent;                   // pairs (2p, 2p+1) instead of (p, p + R/2)
  int src_dtype, weight_dtype;    // wllm_dtype codes
  int kv_fp8;
  int vec, weight_vec, table_vec; // 16-byte accesses are aligned
  int row_lanes, warps_per_token; // set by launch_rotate
  float eps, inv_dim, k_inv, v_inv;
  unsigned long long wait_limit_ns;
  int* err;
};
int launch_rotate(RotateParams p, int num_sms, cudaStream_t stream);

// Minimum and maximum of the keys of every block that new tokens filled
// (key_bounds.cu).  A null query_start_loc means one new token a sequence.
struct BoundsParams {
  uint8_t* bounds;                // [N_b][Hkv][2][D] of the cache's type
  const uint8_t* k_cache;
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int num_seqs, num_kv_heads, num_blocks, log2_bs;
  int max_tokens;                 // the most a block table row can name
  unsigned check_ctas;            // set by launch_key_bounds: leading CTAs that check query_start_loc
  int* err;
};
int launch_key_bounds(int dtype, int head_dim, BoundsParams p, int num_sms, cudaStream_t stream);

// The blocks that a decode has to read (select.cu), by their key bounds.
struct SelectParams {
  int32_t* selected;              // [B][Hkv][top]
  int64_t sel_sb, sel_sh;
  const void* q;                  // [B][Hq][D]
  int64_t q_sb, q_sh;
  const uint8_t* bounds;          // [N_b][Hkv][2][D]
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  int num_seqs, num_kv_heads, group, num_blocks, log2_bs, max_tokens;
  int top, sink, recent;
  int room, longest_first;        // set by launch_select: scores a row has room for; launch order
  int* err;
};
int select_max_blocks();
int launch_select(int dtype, int bounds_dtype, int head_dim, const SelectParams& p, int max_blocks, int num_sms,
                  cudaStream_t stream);

// Decode attention over the listed blocks (sparse_decode.cu).
struct SparseParams {
  void* out;                      // [B][Hq][D]
  const void* q;
  int64_t q_sb, q_sh, o_sb, o_sh; // strides (elements)
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  const int32_t* selected;        // [B][Hkv][top]
  int64_t sel_sb, sel_sh;
  int num_seqs, num_kv_heads, group, num_head_tiles, num_blocks, log2_bs, max_tokens, top;
  int q_pairs;                    // query rows allow 4-byte loads
  float scale_log2, v_scale;
  unsigned long long wait_limit_ns;
  int* err;
};
int launch_sparse_decode(int dtype, bool kv_fp8, int head_dim, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         SparseParams p, int num_sms, cudaStream_t stream);

// Check-mode kernels: record index errors in the device error word.
int launch_check_decode(const int32_t* block_tables, int64_t bt_stride,
                        const int32_t* context_lens, int num_seqs, int max_blocks,
                        int block_size, int num_blocks, int* err, cudaStream_t stream);
int launch_check_append(const void* slots, int slots_are_i64, int num_tokens,
                        int64_t num_slots, int* err, cudaStream_t stream);

// Bytes of shared memory one decode CTA uses, and its thread count.
int decode_smem_bytes(int dtype, int head_dim, DecodeVariant v, int head_tile);
int decode_threads(int dtype, int head_dim);

}  // namespace wllm
