// api_block_scaled.cu -- C ABI of the cache with a scale for each block and head
// (wllm_assign_slots, wllm_reshape_and_cache_block_scaled,
// wllm_paged_attention_decode_block_scaled, wllm_paged_attention_prefill_block_scaled):
// argument checks and launches.
#include <algorithm>
#include <initializer_list>

#include "api_internal.h"
#include "launch.h"

using namespace wllm;

namespace {

int check_vector(const wllm_tensor* t, const char* name, int dtype, int64_t n) {
  int rc;
  if ((rc = check_desc(t, name, 1))) return rc;
  if (t->dtype != dtype) return fail(WLLM_ERR_INVALID_ARG, "%s: dtype must be %s", name, dtype == WLLM_I64 ? "I64" : "I32");
  if (t->shape[0] != n) return fail(WLLM_ERR_INVALID_ARG, "%s must have %lld entries", name, (long long)n);
  if (n > 1 && t->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "%s must be contiguous", name);
  return WLLM_OK;
}

// Caches of codes and their scales.
int check_cache(const wllm_tensor* k_cache, const wllm_tensor* v_cache, const wllm_tensor* k_scales, const wllm_tensor* v_scales) {
  int rc;
  if ((rc = check_desc(k_cache, "k_cache", 4)) || (rc = check_desc(v_cache, "v_cache", 4)) ||
      (rc = check_desc(k_scales, "k_scales", 2)) || (rc = check_desc(v_scales, "v_scales", 2)))
    return rc;
  if (k_cache->dtype != WLLM_FP8_E4M3 || v_cache->dtype != WLLM_FP8_E4M3)
    return fail(WLLM_ERR_INVALID_ARG, "caches must be FP8_E4M3");
  if (!same_shape(k_cache, v_cache)) return fail(WLLM_ERR_INVALID_ARG, "k_cache and v_cache shapes differ");
  if (!contiguous(k_cache) || !contiguous(v_cache)) return fail(WLLM_ERR_INVALID_ARG, "caches must be dense");
  for (const wllm_tensor* s : {k_scales, v_scales}) {
    if (s->dtype != WLLM_F32) return fail(WLLM_ERR_INVALID_ARG, "k_scales and v_scales: dtype must be F32");
    if (s->shape[0] != k_cache->shape[0] || s->shape[1] != k_cache->shape[1])
      return fail(WLLM_ERR_INVALID_ARG, "k_scales and v_scales must be [N_b, Hkv] of the caches");
    if (!contiguous(s)) return fail(WLLM_ERR_INVALID_ARG, "k_scales and v_scales must be dense");
  }
  return WLLM_OK;
}

int check_starts(const wllm_tensor* query_start_loc, int64_t B) {
  int rc;
  if ((rc = check_desc(query_start_loc, "query_start_loc", 1))) return rc;
  if (query_start_loc->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc: dtype must be I32");
  if (query_start_loc->shape[0] != B + 1) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc must have B+1 entries");
  if (B > 0 && query_start_loc->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc must be contiguous");
  return WLLM_OK;
}

// What the two attention calls share: out, q, the cache, tables and lengths of B sequences.
int check_attention(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache, const wllm_tensor* v_cache,
                    const wllm_tensor* k_scales, const wllm_tensor* v_scales, const wllm_tensor* block_tables,
                    const wllm_tensor* context_lens, int64_t B, int num_kv_heads, float scale, int block_size) {
  int rc;
  if ((rc = check_cache(k_cache, v_cache, k_scales, v_scales))) return rc;
  const int dt = q->dtype;
  if (dt != WLLM_F16 && dt != WLLM_BF16) return fail(WLLM_ERR_INVALID_ARG, "q: dtype must be F16 or BF16");
  if (out->dtype != dt) return fail(WLLM_ERR_INVALID_ARG, "out must have the dtype of q");
  if (!same_shape(out, q)) return fail(WLLM_ERR_INVALID_ARG, "out and q shapes differ");
  const int64_t hq = q->shape[1], d = q->shape[2];
  const int64_t nb = k_cache->shape[0], hkv = k_cache->shape[1], bs = k_cache->shape[2];
  if (k_cache->shape[3] != d) return fail(WLLM_ERR_INVALID_ARG, "cache head_dim differs from q");
  if ((rc = check_pool_args(hkv, bs, num_kv_heads, block_size))) return rc;
  if (hkv <= 0 || hq % hkv != 0) return fail(WLLM_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if ((rc = check_tables(block_tables, context_lens, B, nb, bs))) return rc;
  if (d > 1 && (q->stride[2] != 1 || out->stride[2] != 1))
    return fail(WLLM_ERR_INVALID_ARG, "q/out last dimension must be contiguous");
  if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
    return fail(WLLM_ERR_INVALID_ARG, "scale must be finite");
  if (d == 64 && bs < 16) return fail(WLLM_ERR_UNSUPPORTED, "head_dim 64 needs block_size >= 16");
  if (hq > 65535 || block_tables->shape[1] * bs > INT32_MAX / 32 || q->shape[0] * hq > INT32_MAX / 8)
    return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  return WLLM_OK;
}

// The pool that the attention reads, once there is something to do.
int check_attention_data(const wllm_tensor* k_cache, const wllm_tensor* v_cache) {
  if (k_cache->shape[0] < 1) return fail(WLLM_ERR_INVALID_ARG, "the pool has no blocks");
  if (!aligned(k_cache->data, 16) || !aligned(v_cache->data, 16))
    return fail(WLLM_ERR_INVALID_ARG, "cache base pointers must be 16-byte aligned");
  return WLLM_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

size_t workspace_bytes(int num_sms) {
  return std::max(decode_block_scaled_workspace(num_sms), prefill_block_scaled_workspace(num_sms));
}

int check_workspace(const wllm_tensor* workspace, int num_sms) {
  if (workspace->dtype != WLLM_FP8_E4M3) return fail(WLLM_ERR_INVALID_ARG, "workspace must be bytes");
  if (workspace->shape[0] > 1 && workspace->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "workspace must be contiguous");
  const size_t need = workspace_bytes(num_sms);
  if (static_cast<size_t>(workspace->shape[0]) < need)
    return fail(WLLM_ERR_INVALID_ARG, "workspace has %lld bytes, %zu are needed", (long long)workspace->shape[0], need);
  if (!aligned(workspace->data, 256)) return fail(WLLM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return WLLM_OK;
}

unsigned long long wait_limit() { return static_cast<unsigned long long>(env_int("WLLM_WAIT_LIMIT_NS", 200000000LL)); }

}  // namespace

extern "C" {

int wllm_assign_slots(const wllm_tensor* slot_mapping, const wllm_tensor* positions, const wllm_tensor* query_start_loc,
                      const wllm_tensor* context_lens_out, const wllm_tensor* num_free_out, const wllm_tensor* block_tables,
                      const wllm_tensor* context_lens, const wllm_tensor* new_tokens, const wllm_tensor* free_blocks,
                      const wllm_tensor* num_free, int block_size, wllm_stream stream) {
  int rc;
  if ((rc = check_desc(block_tables, "block_tables", 2)) || (rc = check_desc(slot_mapping, "slot_mapping", 1)) ||
      (rc = check_desc(free_blocks, "free_blocks", 1)))
    return rc;
  const int64_t B = block_tables->shape[0], T = slot_mapping->shape[0], F = free_blocks->shape[0];
  if ((rc = check_vector(slot_mapping, "slot_mapping", WLLM_I64, T)) ||
      (positions != nullptr && (rc = check_vector(positions, "positions", WLLM_I64, T))) ||
      (rc = check_vector(query_start_loc, "query_start_loc", WLLM_I32, B + 1)) ||
      (rc = check_vector(context_lens_out, "context_lens_out", WLLM_I32, B)) ||
      (rc = check_vector(num_free_out, "num_free_out", WLLM_I32, 1)) ||
      (rc = check_vector(context_lens, "context_lens", WLLM_I32, B)) || (rc = check_vector(new_tokens, "new_tokens", WLLM_I32, B)) ||
      (rc = check_vector(free_blocks, "free_blocks", WLLM_I32, F)) || (rc = check_vector(num_free, "num_free", WLLM_I32, 1)))
    return rc;
  if (block_tables->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "block_tables: dtype must be I32");
  if (block_tables->shape[1] > 1 && block_tables->stride[1] != 1)
    return fail(WLLM_ERR_INVALID_ARG, "block_tables rows must be contiguous");
  if (B > 1 && block_tables->shape[1] > 0 && block_tables->stride[0] < block_tables->shape[1])
    return fail(WLLM_ERR_INVALID_ARG, "block_tables rows must not overlap");
  if (!is_pow2(block_size)) return fail(WLLM_ERR_UNSUPPORTED, "block_size %d is not a power of two", block_size);
  if (B > kMaxSlotSeqs) return fail(WLLM_ERR_UNSUPPORTED, "%lld sequences not supported (%d at most)", (long long)B, kMaxSlotSeqs);
  if (T > INT32_MAX || F > INT32_MAX || block_tables->shape[1] * block_size > INT32_MAX)
    return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  // what is written must not be read elsewhere: only a length and the count may be updated in place
  const wllm_tensor* written[] = {slot_mapping, positions, query_start_loc, context_lens_out, num_free_out, block_tables, free_blocks};
  const wllm_tensor* all[] = {slot_mapping, positions, query_start_loc, context_lens_out, num_free_out, block_tables, free_blocks,
                              context_lens, new_tokens, num_free};
  for (int i = 0; i < 7; ++i)
    for (int j = 0; j < 10; ++j) {
      const wllm_tensor *a = written[i], *b = all[j];
      if (a == nullptr || b == nullptr || (j < 7 && j <= i) || numel(a) == 0 || numel(b) == 0 || !spans_meet(a, b)) continue;
      if (((a == context_lens_out && b == context_lens) || (a == num_free_out && b == num_free)) && a->data == b->data) continue;
      return fail(WLLM_ERR_INVALID_ARG, "tensors that are written overlap others");
    }
  SlotsParams p{};
  p.slots = static_cast<int64_t*>(slot_mapping->data);
  p.positions = positions != nullptr ? static_cast<int64_t*>(positions->data) : nullptr;
  p.starts = static_cast<int32_t*>(query_start_loc->data);
  p.lens_out = static_cast<int32_t*>(context_lens_out->data);
  p.free_out = static_cast<int32_t*>(num_free_out->data);
  p.block_tables = static_cast<int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.new_tokens = static_cast<const int32_t*>(new_tokens->data);
  p.free_blocks = static_cast<int32_t*>(free_blocks->data);
  p.num_free = static_cast<const int32_t*>(num_free->data);
  p.num_seqs = static_cast<int>(B);
  p.num_rows = static_cast<int>(T);
  p.free_room = static_cast<int>(F);
  p.log2_bs = ilog2(block_size);
  p.max_tokens = static_cast<int>(block_tables->shape[1] * block_size);
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(launch_assign_slots(p, st));
  if (e != cudaSuccess) return cuda_fail(e, "assign slots launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "assign_slots") : WLLM_OK;
}

int wllm_reshape_and_cache_block_scaled(const wllm_tensor* key, const wllm_tensor* value, const wllm_tensor* k_cache,
                                        const wllm_tensor* v_cache, const wllm_tensor* k_scales, const wllm_tensor* v_scales,
                                        const wllm_tensor* block_tables, const wllm_tensor* context_lens,
                                        const wllm_tensor* query_start_loc, int block_size, wllm_stream stream) {
  int rc;
  if ((rc = check_desc(key, "key", 3)) || (rc = check_desc(value, "value", 3)) ||
      (rc = check_cache(k_cache, v_cache, k_scales, v_scales)) || (rc = check_desc(block_tables, "block_tables", 2)) ||
      (rc = check_desc(context_lens, "context_lens", 1)))
    return rc;
  const int dt = key->dtype;
  if (!is_float(dt)) return fail(WLLM_ERR_INVALID_ARG, "key: dtype must be F32, F16 or BF16");
  if (value->dtype != dt) return fail(WLLM_ERR_INVALID_ARG, "key and value must share one dtype");
  if (!same_shape(key, value)) return fail(WLLM_ERR_INVALID_ARG, "key and value shapes differ");
  const int64_t T = key->shape[0], hkv = key->shape[1], d = key->shape[2], B = context_lens->shape[0];
  const int64_t nb = k_cache->shape[0], bs = k_cache->shape[2];
  if (k_cache->shape[1] != hkv || k_cache->shape[3] != d)
    return fail(WLLM_ERR_INVALID_ARG, "cache shape [%lld,%lld,%lld,%lld] does not match key [T,%lld,%lld]", (long long)nb,
                (long long)k_cache->shape[1], (long long)bs, (long long)k_cache->shape[3], (long long)hkv, (long long)d);
  if (bs != block_size)
    return fail(WLLM_ERR_INVALID_ARG, "block_size %d differs from cache dim %lld", block_size, (long long)bs);
  if ((rc = check_tables(block_tables, context_lens, B, nb, bs))) return rc;
  if (query_start_loc != nullptr) {
    if ((rc = check_starts(query_start_loc, B))) return rc;
  } else if (T != B) {
    return fail(WLLM_ERR_INVALID_ARG, "without query_start_loc key must have a row a sequence (%lld), has %lld", (long long)B, (long long)T);
  }
  if (d > 1 && (key->stride[2] != 1 || value->stride[2] != 1))
    return fail(WLLM_ERR_INVALID_ARG, "key/value last dimension must be contiguous");
  if (d != 64 && d != 128 && d != 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)d);
  if (hkv > 65535 || T > INT32_MAX / 8 || B > INT32_MAX / 8) return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  if (T == 0 || B == 0 || hkv == 0) return WLLM_OK;
  if (nb < 1) return fail(WLLM_ERR_INVALID_ARG, "the pool has no blocks");
  if (!aligned(k_cache->data, 16) || !aligned(v_cache->data, 16))
    return fail(WLLM_ERR_INVALID_ARG, "cache base pointers must be 16-byte aligned");
  ScaledAppendParams p{};
  const wllm_tensor* src[2] = {key, value};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = src[i]->data;
    p.src_st[i] = src[i]->stride[0], p.src_sh[i] = src[i]->stride[1];
  }
  p.cache[0] = static_cast<uint8_t*>(k_cache->data), p.cache[1] = static_cast<uint8_t*>(v_cache->data);
  p.scales[0] = static_cast<float*>(k_scales->data), p.scales[1] = static_cast<float*>(v_scales->data);
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.query_start_loc = query_start_loc != nullptr ? static_cast<const int32_t*>(query_start_loc->data) : nullptr;
  p.num_seqs = static_cast<int>(B);
  p.num_tokens = static_cast<int>(T);
  p.num_kv_heads = static_cast<int>(hkv);
  p.num_blocks = static_cast<int>(nb);
  p.log2_bs = ilog2(bs);
  p.max_tokens = static_cast<int>(block_tables->shape[1] * bs);
  p.vec = rows_aligned(key, 2, 16) && rows_aligned(value, 2, 16);
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(launch_append_block_scaled(dt, static_cast<int>(d), p, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "block-scaled append launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "reshape_and_cache_block_scaled") : WLLM_OK;
}

size_t wllm_block_scaled_workspace_bytes(void) {
  DeviceState* s = nullptr;
  return locked_state(&s) == WLLM_OK ? workspace_bytes(s->num_sms) : 0;
}

int wllm_paged_attention_decode_block_scaled(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache,
                                             const wllm_tensor* v_cache, const wllm_tensor* k_scales,
                                             const wllm_tensor* v_scales, const wllm_tensor* block_tables,
                                             const wllm_tensor* context_lens, const wllm_tensor* workspace, int num_kv_heads,
                                             float scale, int block_size, wllm_stream stream) {
  int rc;
  if ((rc = check_desc(out, "out", 3)) || (rc = check_desc(q, "q", 3)) || (rc = check_desc(block_tables, "block_tables", 2)) ||
      (rc = check_desc(context_lens, "context_lens", 1)) || (rc = check_desc(workspace, "workspace", 1)))
    return rc;
  const int64_t B = q->shape[0], hq = q->shape[1], d = q->shape[2];
  if ((rc = check_attention(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, B, num_kv_heads, scale, block_size)))
    return rc;
  if (d != 64 && d != 128 && d != 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)d);
  if (B == 0 || hq == 0) return WLLM_OK;
  if ((rc = check_attention_data(k_cache, v_cache))) return rc;
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  if ((rc = check_workspace(workspace, s->num_sms))) return rc;
  ScaledDecodeParams p{};
  p.out = out->data;
  p.q = q->data;
  p.q_sb = q->stride[0], p.q_sh = q->stride[1];
  p.o_sb = out->stride[0], p.o_sh = out->stride[1];
  p.k_scales = static_cast<const float*>(k_scales->data);
  p.v_scales = static_cast<const float*>(v_scales->data);
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  const int64_t nb = k_cache->shape[0], hkv = k_cache->shape[1], bs = k_cache->shape[2];
  p.num_seqs = static_cast<int>(B);
  p.num_q_heads = static_cast<int>(hq);
  p.num_kv_heads = static_cast<int>(hkv);
  p.group = static_cast<int>(hq / hkv);
  p.num_blocks = static_cast<int>(nb);
  p.log2_bs = ilog2(bs);
  p.max_tokens = static_cast<int>(block_tables->shape[1] * bs);
  p.bf16 = q->dtype == WLLM_BF16;
  p.q_pairs = rows_aligned(q, 2, 4);
  p.o_pairs = rows_aligned(out, 2, 4);
  p.scale_log2 = scale * kLog2e;
  p.parts = static_cast<float*>(workspace->data);
  p.wait_limit_ns = wait_limit();
  p.err = s->err;
  CUtensorMap kmap, vmap;
  if ((rc = make_pool_map(&kmap, k_cache->data, WLLM_FP8_E4M3, nb, hkv, bs, d, "k_cache"))) return rc;
  if ((rc = make_pool_map(&vmap, v_cache->data, WLLM_FP8_E4M3, nb, hkv, bs, d, "v_cache"))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(launch_decode_block_scaled(static_cast<int>(d), kmap, vmap, p, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "block-scaled decode launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "paged_attention_decode_block_scaled") : WLLM_OK;
}

int wllm_paged_attention_prefill_block_scaled(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache,
                                              const wllm_tensor* v_cache, const wllm_tensor* k_scales,
                                              const wllm_tensor* v_scales, const wllm_tensor* block_tables,
                                              const wllm_tensor* context_lens, const wllm_tensor* query_start_loc,
                                              const wllm_tensor* workspace, int num_kv_heads, float scale, int block_size,
                                              wllm_stream stream) {
  int rc;
  if ((rc = check_desc(out, "out", 3)) || (rc = check_desc(q, "q", 3)) || (rc = check_desc(block_tables, "block_tables", 2)) ||
      (rc = check_desc(context_lens, "context_lens", 1)) || (rc = check_desc(workspace, "workspace", 1)))
    return rc;
  const int64_t T = q->shape[0], hq = q->shape[1], d = q->shape[2], B = context_lens->shape[0];
  if ((rc = check_attention(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, B, num_kv_heads, scale, block_size)) ||
      (rc = check_starts(query_start_loc, B)))
    return rc;
  if (d != 64 && d != 128) return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128)", (long long)d);
  if (T == 0 || B == 0 || hq == 0) return WLLM_OK;
  if ((rc = check_attention_data(k_cache, v_cache))) return rc;
  const int64_t nb = k_cache->shape[0], hkv = k_cache->shape[1], bs = k_cache->shape[2];
  if ((T * (hq / hkv) / 256 + 1 + B) * hkv > INT32_MAX) return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  ScaledPrefillParams sp{};
  PrefillParams& p = sp.base;
  p.out = out->data;
  p.q = q->data;
  p.q_st = q->stride[0], p.q_sh = q->stride[1];
  p.o_st = out->stride[0], p.o_sh = out->stride[1];
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.query_start_loc = static_cast<const int32_t*>(query_start_loc->data);
  p.num_seqs = static_cast<int>(B);
  p.num_tokens = static_cast<int>(T);
  p.num_q_heads = static_cast<int>(hq);
  p.num_kv_heads = static_cast<int>(hkv);
  p.group = static_cast<int>(hq / hkv);
  p.max_blocks = static_cast<int>(block_tables->shape[1]);
  p.block_size = static_cast<int>(bs);
  p.log2_bs = ilog2(bs);
  p.num_blocks = static_cast<int>(nb);
  p.scale_log2 = scale * kLog2e;
  p.v_scale = 1.f;
  p.wait_limit_ns = wait_limit();
  sp.k_scales = static_cast<const float*>(k_scales->data);
  sp.v_scales = static_cast<const float*>(v_scales->data);
  sp.parts = static_cast<float*>(workspace->data);
  sp.q_vec = rows_aligned(q, 2, 16);
  sp.o_vec = rows_aligned(out, 2, 16);
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  if ((rc = check_workspace(workspace, s->num_sms))) return rc;
  p.err = s->err;
  CUtensorMap kmap, vmap;
  if ((rc = make_pool_map(&kmap, k_cache->data, WLLM_FP8_E4M3, nb, hkv, bs, d, "k_cache"))) return rc;
  if ((rc = make_pool_map(&vmap, v_cache->data, WLLM_FP8_E4M3, nb, hkv, bs, d, "v_cache"))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(
      launch_prefill_block_scaled(q->dtype, static_cast<int>(d), kmap, vmap, sp, T, B, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "block-scaled prefill launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "paged_attention_prefill_block_scaled") : WLLM_OK;
}

}  // extern "C"
