// api_sparse.cu -- C ABI of the rotary append and the block-sparse decode
// (wllm_rotate_and_cache, wllm_update_key_bounds, wllm_select_blocks,
// wllm_paged_attention_decode_sparse and their fp8 forms): argument checks and
// launches.  None of them uses the device workspace.
#include <algorithm>

#include "api_internal.h"
#include "launch.h"

using namespace wllm;

namespace wllm {

// Bytes that a tensor's elements span, and whether two tensors' spans meet.
bool spans_meet(const wllm_tensor* a, const wllm_tensor* b) {
  auto span = [](const wllm_tensor* t, const uint8_t** lo, const uint8_t** hi) {
    int64_t first = 0, last = 0;
    for (int i = 0; i < t->ndim; ++i) {
      const int64_t reach = (t->shape[i] - 1) * t->stride[i];
      (reach < 0 ? first : last) += reach;
    }
    const int64_t elt = elt_size(t->dtype);
    *lo = static_cast<const uint8_t*>(t->data) + first * elt;
    *hi = static_cast<const uint8_t*>(t->data) + (last + 1) * elt;
  };
  const uint8_t *a0, *a1, *b0, *b1;
  span(a, &a0, &a1);
  span(b, &b0, &b1);
  return a0 < b1 && b0 < a1;
}

bool rows_aligned(const wllm_tensor* t, int dims, int64_t bytes) {
  if (!aligned(t->data, static_cast<uintptr_t>(bytes))) return false;
  for (int i = 0; i < dims; ++i)
    if (t->shape[i] > 1 && (t->stride[i] * elt_size(t->dtype)) % bytes != 0) return false;
  return true;
}

// The current device's state; the lock covers its creation.
int locked_state(DeviceState** s) {
  std::lock_guard<std::mutex> lock(g_mutex);
  return device_state(s);
}

// A block pool [N_b][Hkv][bs][D], its table rows and lengths: what the block-sparse
// and the block-scaled calls share.
int check_tables(const wllm_tensor* block_tables, const wllm_tensor* context_lens, int64_t B, int64_t nb, int64_t bs) {
  if (block_tables->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "block_tables: dtype must be I32");
  if (context_lens->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "context_lens: dtype must be I32");
  if (block_tables->shape[0] != B) return fail(WLLM_ERR_INVALID_ARG, "block_tables must have B rows");
  if (context_lens->shape[0] != B) return fail(WLLM_ERR_INVALID_ARG, "context_lens must have B entries");
  if (B > 1 && context_lens->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "context_lens must be contiguous");
  if (block_tables->shape[1] > 1 && block_tables->stride[1] != 1)
    return fail(WLLM_ERR_INVALID_ARG, "block_tables rows must be contiguous");
  if (!is_pow2(bs) || bs < 8 || bs > 256)
    return fail(WLLM_ERR_UNSUPPORTED, "block_size %lld not supported (power of two in [8, 256])", (long long)bs);
  if (B > INT32_MAX || nb > INT32_MAX || block_tables->shape[1] * bs > INT32_MAX)
    return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  return WLLM_OK;
}

int check_pool_args(int64_t hkv, int64_t bs, int num_kv_heads, int block_size) {
  if (hkv != num_kv_heads)
    return fail(WLLM_ERR_INVALID_ARG, "num_kv_heads %d differs from cache dim %lld", num_kv_heads, (long long)hkv);
  if (bs != block_size)
    return fail(WLLM_ERR_INVALID_ARG, "block_size %d differs from cache dim %lld", block_size, (long long)bs);
  return WLLM_OK;
}

}  // namespace wllm

namespace {

int rotate_call(const wllm_tensor* q_out, const wllm_tensor* q, const wllm_tensor* key, const wllm_tensor* value,
                const wllm_tensor* k_cache, const wllm_tensor* v_cache, const wllm_tensor* slot_mapping,
                const wllm_tensor* positions, const wllm_tensor* cos_sin, const wllm_tensor* q_weight,
                const wllm_tensor* k_weight, const wllm_rotary* how, bool kv_fp8, float k_scale, float v_scale,
                wllm_stream stream) {
  int rc;
  if ((rc = check_desc(q_out, "q_out", 3)) || (rc = check_desc(q, "q", 3)) || (rc = check_desc(key, "key", 3)) ||
      (rc = check_desc(value, "value", 3)) || (rc = check_desc(k_cache, "k_cache", 4)) ||
      (rc = check_desc(v_cache, "v_cache", 4)) || (rc = check_desc(slot_mapping, "slot_mapping", 1)) ||
      (rc = check_desc(cos_sin, "cos_sin", 2)))
    return rc;
  if (positions == nullptr) return fail(WLLM_ERR_INVALID_ARG, "positions: null descriptor");
  if (how == nullptr) return fail(WLLM_ERR_INVALID_ARG, "how: null");
  if (how->num_axes < 1 || how->num_axes > kMaxRotaryAxes)
    return fail(WLLM_ERR_INVALID_ARG, "num_axes must be 1..%d, got %d", kMaxRotaryAxes, how->num_axes);
  if (how->style != WLLM_ROTARY_HALVES && how->style != WLLM_ROTARY_ADJACENT)
    return fail(WLLM_ERR_INVALID_ARG, "unknown rotary style %d", how->style);
  if (!(how->eps >= 0.f && how->eps < INFINITY)) return fail(WLLM_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((rc = check_desc(positions, "positions", positions->ndim == 1 && how->num_axes == 1 ? 1 : 2))) return rc;
  const int dt = q->dtype;
  if (!is_float(dt)) return fail(WLLM_ERR_INVALID_ARG, "q: dtype must be F32, F16 or BF16");
  if (q_out->dtype != dt || key->dtype != dt || value->dtype != dt)
    return fail(WLLM_ERR_INVALID_ARG, "q_out, q, key and value must share one dtype");
  if (kv_fp8) {
    if (k_cache->dtype != WLLM_FP8_E4M3 || v_cache->dtype != WLLM_FP8_E4M3)
      return fail(WLLM_ERR_INVALID_ARG, "caches must be FP8_E4M3");
    if (!positive_finite(k_scale) || !positive_finite(v_scale))
      return fail(WLLM_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  } else if (k_cache->dtype != dt || v_cache->dtype != dt) {
    return fail(WLLM_ERR_INVALID_ARG, "q, key, value and caches must share one dtype");
  }
  for (const wllm_tensor* x : {slot_mapping, positions})
    if (x->dtype != WLLM_I64 && x->dtype != WLLM_I32)
      return fail(WLLM_ERR_INVALID_ARG, "slot_mapping and positions: dtype must be I64 or I32");
  if (cos_sin->dtype != WLLM_F32) return fail(WLLM_ERR_INVALID_ARG, "cos_sin: dtype must be F32");
  if (!same_shape(q_out, q)) return fail(WLLM_ERR_INVALID_ARG, "q_out and q shapes differ");
  if (!same_shape(key, value)) return fail(WLLM_ERR_INVALID_ARG, "key and value shapes differ");
  if (!same_shape(k_cache, v_cache)) return fail(WLLM_ERR_INVALID_ARG, "k_cache and v_cache shapes differ");
  const int64_t T = q->shape[0], hq = q->shape[1], d = q->shape[2], hkv = key->shape[1];
  const int64_t nb = k_cache->shape[0], bs = k_cache->shape[2], rot = cos_sin->shape[1];
  if (key->shape[0] != T || key->shape[2] != d) return fail(WLLM_ERR_INVALID_ARG, "key must be [T, Hkv, D] with q's T and D");
  if (k_cache->shape[1] != hkv || k_cache->shape[3] != d)
    return fail(WLLM_ERR_INVALID_ARG, "cache shape [%lld,%lld,%lld,%lld] does not match key [T,%lld,%lld]", (long long)nb,
                (long long)k_cache->shape[1], (long long)bs, (long long)k_cache->shape[3], (long long)hkv, (long long)d);
  if (!contiguous(k_cache) || !contiguous(v_cache)) return fail(WLLM_ERR_INVALID_ARG, "caches must be dense");
  if (slot_mapping->shape[0] != T) return fail(WLLM_ERR_INVALID_ARG, "slot_mapping must have T entries");
  if (T > 1 && slot_mapping->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "slot_mapping must be contiguous");
  const int pd = positions->ndim;
  if (positions->shape[pd - 1] != T || (pd == 2 && positions->shape[0] != how->num_axes))
    return fail(WLLM_ERR_INVALID_ARG, "positions must be [T] or [num_axes, T]");
  if (T > 1 && positions->stride[pd - 1] != 1) return fail(WLLM_ERR_INVALID_ARG, "positions rows must be contiguous");
  if (d > 1 && (q->stride[2] != 1 || q_out->stride[2] != 1 || key->stride[2] != 1 || value->stride[2] != 1))
    return fail(WLLM_ERR_INVALID_ARG, "q_out/q/key/value last dimension must be contiguous");
  if (rot > 1 && cos_sin->stride[1] != 1) return fail(WLLM_ERR_INVALID_ARG, "cos_sin rows must be contiguous");
  for (const wllm_tensor* w : {q_weight, k_weight}) {
    if (w == nullptr) continue;
    if ((rc = check_desc(w, "norm weight", 1))) return rc;
    if (w->dtype != dt && w->dtype != WLLM_F32)
      return fail(WLLM_ERR_INVALID_ARG, "norm weights must be F32 or of q's dtype");
    if (w->shape[0] != d || (d > 1 && w->stride[0] != 1))
      return fail(WLLM_ERR_INVALID_ARG, "norm weights must be contiguous [D]");
    if (!aligned(w->data, static_cast<uintptr_t>(elt_size(w->dtype))))
      return fail(WLLM_ERR_INVALID_ARG, "norm weights must be aligned to their element size");
  }
  if (q_weight != nullptr && k_weight != nullptr && q_weight->dtype != k_weight->dtype)
    return fail(WLLM_ERR_INVALID_ARG, "the two norm weights must share one dtype");
  if (rot > d) return fail(WLLM_ERR_INVALID_ARG, "cos_sin has %lld columns, head_dim is %lld", (long long)rot, (long long)d);
  int64_t turned = rot / 2;
  if (how->num_axes > 1) {
    turned = 0;
    for (int a = 0; a < how->num_axes; ++a) {
      if (how->sections[a] < 0) return fail(WLLM_ERR_INVALID_ARG, "sections must not be negative");
      turned += how->sections[a];
    }
  }
  if (turned != rot / 2)
    return fail(WLLM_ERR_INVALID_ARG, "sections sum to %lld pairs, cos_sin has %lld", (long long)turned, (long long)(rot / 2));
  if (d % 16 != 0 || d < 16 || d > 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (multiples of 16 up to 256)", (long long)d);
  if (rot % 16 != 0 || rot < 16)
    return fail(WLLM_ERR_UNSUPPORTED, "%lld rotated dims not supported (multiples of 16)", (long long)rot);
  if (!is_pow2(bs)) return fail(WLLM_ERR_UNSUPPORTED, "block_size %lld is not a power of two", (long long)bs);
  if (hq > 65535 || hkv > 65535 || T > INT32_MAX / 8 || nb > INT32_MAX || bs > INT32_MAX)
    return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  if (T == 0 || hq + hkv == 0) return WLLM_OK;
  for (const wllm_tensor* x : {q_out, q, key, value, k_cache, v_cache})
    if (!aligned(x->data, static_cast<uintptr_t>(elt_size(x->dtype))))
      return fail(WLLM_ERR_INVALID_ARG, "q_out/q/key/value and caches must be aligned to their element size");
  if (kv_fp8 && !(aligned(k_cache->data, 8) && aligned(v_cache->data, 8)))
    return fail(WLLM_ERR_INVALID_ARG, "fp8 caches must be 8-byte aligned");
  // q_out may be q itself; any other overlap would read turned values
  if (hq > 0 && spans_meet(q_out, q) &&
      !(q_out->data == q->data && (T == 1 || q_out->stride[0] == q->stride[0]) && (hq == 1 || q_out->stride[1] == q->stride[1])))
    return fail(WLLM_ERR_INVALID_ARG, "q_out overlaps q without being q");

  RotateParams p{};
  p.q_out = q_out->data;
  p.q = q->data;
  p.key = key->data;
  p.value = value->data;
  p.k_cache = static_cast<uint8_t*>(k_cache->data);
  p.v_cache = static_cast<uint8_t*>(v_cache->data);
  p.slots = slot_mapping->data;
  p.slots_are_i64 = slot_mapping->dtype == WLLM_I64;
  p.positions = positions->data;
  p.pos_are_i64 = positions->dtype == WLLM_I64;
  p.pos_sa = pd == 2 ? positions->stride[0] : 0;
  p.cos_sin = static_cast<const float*>(cos_sin->data);
  p.table_stride = cos_sin->stride[0];
  p.num_positions = cos_sin->shape[0];
  p.num_slots = nb * bs;
  p.q_weight = q_weight != nullptr ? q_weight->data : nullptr;
  p.k_weight = k_weight != nullptr ? k_weight->data : nullptr;
  p.q_st = q->stride[0], p.q_sh = q->stride[1];
  p.key_st = key->stride[0], p.key_sh = key->stride[1];
  p.val_st = value->stride[0], p.val_sh = value->stride[1];
  p.qo_st = q_out->stride[0], p.qo_sh = q_out->stride[1];
  p.num_tokens = static_cast<int>(T);
  p.num_q_heads = static_cast<int>(hq);
  p.num_kv_heads = static_cast<int>(hkv);
  p.head_dim = static_cast<int>(d);
  p.rot_dim = static_cast<int>(rot);
  p.log2_bs = ilog2(bs);
  p.num_axes = how->num_axes;
  int end = 0;
  for (int a = 0; a < kMaxRotaryAxes; ++a) {
    if (a < how->num_axes) end += how->num_axes == 1 ? p.rot_dim / 2 : how->sections[a];
    p.section_end[a] = end;
  }
  p.adjacent = how->style == WLLM_ROTARY_ADJACENT;
  p.src_dtype = dt;
  const wllm_tensor* w = q_weight != nullptr ? q_weight : k_weight;
  p.weight_dtype = w != nullptr ? w->dtype : WLLM_F32;
  p.weight_vec = (q_weight == nullptr || aligned(q_weight->data, 16)) && (k_weight == nullptr || aligned(k_weight->data, 16));
  p.kv_fp8 = kv_fp8;
  p.vec = rows_aligned(q_out, 2, 16) && rows_aligned(q, 2, 16) && rows_aligned(key, 2, 16) && rows_aligned(value, 2, 16) &&
          (kv_fp8 || (aligned(k_cache->data, 16) && aligned(v_cache->data, 16)));
  p.table_vec = aligned(cos_sin->data, 16) && p.table_stride % 4 == 0;
  p.eps = how->eps;
  p.inv_dim = 1.f / static_cast<float>(d);
  p.wait_limit_ns = static_cast<unsigned long long>(env_int("WLLM_WAIT_LIMIT_NS", 200000000LL));
  p.k_inv = 1.f / k_scale;
  p.v_inv = 1.f / v_scale;

  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool check = env_flag("WLLM_CHECK");
  cudaError_t e;
  if (check) {
    e = static_cast<cudaError_t>(launch_check_append(p.slots, p.slots_are_i64, p.num_tokens, p.num_slots, s->err, st));
    if (e != cudaSuccess) return cuda_fail(e, "check_append launch");
    if ((rc = collect_device_errors(s, st, "rotate_and_cache"))) return rc;
  }
  e = static_cast<cudaError_t>(launch_rotate(p, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "rotate launch");
  return check ? collect_device_errors(s, st, "rotate_and_cache") : WLLM_OK;
}

int sparse_call(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache, const wllm_tensor* v_cache,
                const wllm_tensor* block_tables, const wllm_tensor* context_lens, const wllm_tensor* selected,
                int num_kv_heads, float scale, int block_size, bool kv_fp8, float k_scale, float v_scale,
                wllm_stream stream) {
  int rc;
  if ((rc = check_desc(out, "out", 3)) || (rc = check_desc(q, "q", 3)) || (rc = check_desc(k_cache, "k_cache", 4)) ||
      (rc = check_desc(v_cache, "v_cache", 4)) || (rc = check_desc(block_tables, "block_tables", 2)) ||
      (rc = check_desc(context_lens, "context_lens", 1)) || (rc = check_desc(selected, "selected", 3)))
    return rc;
  const int dt = q->dtype;
  if (kv_fp8) {
    if (dt != WLLM_F16 && dt != WLLM_BF16)
      return fail(WLLM_ERR_INVALID_ARG, "q: dtype must be F16 or BF16 with an fp8 cache");
    if (k_cache->dtype != WLLM_FP8_E4M3 || v_cache->dtype != WLLM_FP8_E4M3)
      return fail(WLLM_ERR_INVALID_ARG, "caches must be FP8_E4M3");
    if (!positive_finite(k_scale) || !positive_finite(v_scale))
      return fail(WLLM_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  } else {
    if (!is_float(dt)) return fail(WLLM_ERR_INVALID_ARG, "q: dtype must be F32, F16 or BF16");
    if (k_cache->dtype != dt || v_cache->dtype != dt)
      return fail(WLLM_ERR_INVALID_ARG, "q, out and caches must share one dtype");
  }
  if (out->dtype != dt) return fail(WLLM_ERR_INVALID_ARG, "out must have the dtype of q");
  if (selected->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "selected: dtype must be I32");
  if (!same_shape(out, q)) return fail(WLLM_ERR_INVALID_ARG, "out and q shapes differ");
  if (!same_shape(k_cache, v_cache)) return fail(WLLM_ERR_INVALID_ARG, "k_cache and v_cache shapes differ");
  const int64_t B = q->shape[0], hq = q->shape[1], d = q->shape[2];
  const int64_t nb = k_cache->shape[0], hkv = k_cache->shape[1], bs = k_cache->shape[2], top = selected->shape[2];
  if (k_cache->shape[3] != d) return fail(WLLM_ERR_INVALID_ARG, "cache head_dim differs from q");
  if ((rc = check_pool_args(hkv, bs, num_kv_heads, block_size))) return rc;
  if (hkv <= 0 || hq % hkv != 0) return fail(WLLM_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if ((rc = check_tables(block_tables, context_lens, B, nb, bs))) return rc;
  if (selected->shape[0] != B || selected->shape[1] != hkv)
    return fail(WLLM_ERR_INVALID_ARG, "selected must be [B, Hkv, top]");
  if (top > 1 && selected->stride[2] != 1) return fail(WLLM_ERR_INVALID_ARG, "selected rows must be contiguous");
  if (!contiguous(k_cache) || !contiguous(v_cache)) return fail(WLLM_ERR_INVALID_ARG, "caches must be dense");
  if (d > 1 && (q->stride[2] != 1 || out->stride[2] != 1))
    return fail(WLLM_ERR_INVALID_ARG, "q/out last dimension must be contiguous");
  if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
    return fail(WLLM_ERR_INVALID_ARG, "scale must be finite");
  if (d != 64 && d != 128 && d != 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)d);
  if (kv_fp8 && d == 64 && bs < 16)
    return fail(WLLM_ERR_UNSUPPORTED, "an fp8 cache with head_dim 64 needs block_size >= 16");
  if (hq > 65535 || top * bs > INT32_MAX || B * hq > INT32_MAX / 8) return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  if (B == 0 || hq == 0) return WLLM_OK;
  if (nb < 1) return fail(WLLM_ERR_INVALID_ARG, "the pool has no blocks");
  if (!aligned(k_cache->data, 16) || !aligned(v_cache->data, 16))
    return fail(WLLM_ERR_INVALID_ARG, "cache base pointers must be 16-byte aligned");
  const uintptr_t elt = static_cast<uintptr_t>(elt_size(dt));
  if (!aligned(q->data, elt) || !aligned(out->data, elt))
    return fail(WLLM_ERR_INVALID_ARG, "q/out must be aligned to their element size");

  SparseParams p{};
  p.out = out->data;
  p.q = q->data;
  p.q_sb = q->stride[0], p.q_sh = q->stride[1];
  p.o_sb = out->stride[0], p.o_sh = out->stride[1];
  p.k_cache = static_cast<const uint8_t*>(k_cache->data);
  p.v_cache = static_cast<const uint8_t*>(v_cache->data);
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.selected = static_cast<const int32_t*>(selected->data);
  p.sel_sb = selected->stride[0], p.sel_sh = selected->stride[1];
  p.num_seqs = static_cast<int>(B);
  p.num_kv_heads = static_cast<int>(hkv);
  p.group = static_cast<int>(hq / hkv);
  p.num_blocks = static_cast<int>(nb);
  p.log2_bs = ilog2(bs);
  p.max_tokens = static_cast<int>(block_tables->shape[1] * bs);
  p.top = static_cast<int>(top);
  // an fp8 cache holds K / k_scale and V / v_scale: the scales return here
  p.scale_log2 = (kv_fp8 ? scale * k_scale : scale) * 1.4426950408889634f;
  p.v_scale = kv_fp8 ? v_scale : 1.f;
  p.q_pairs = rows_aligned(q, 2, 4);
  p.wait_limit_ns = static_cast<unsigned long long>(env_int("WLLM_WAIT_LIMIT_NS", 200000000LL));
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap kmap, vmap;
  const int kv_dt = kv_fp8 ? WLLM_FP8_E4M3 : dt;
  if ((rc = make_pool_map(&kmap, k_cache->data, kv_dt, nb, hkv, bs, d, "k_cache"))) return rc;
  if ((rc = make_pool_map(&vmap, v_cache->data, kv_dt, nb, hkv, bs, d, "v_cache"))) return rc;
  const cudaError_t e = static_cast<cudaError_t>(
      launch_sparse_decode(dt, kv_fp8, static_cast<int>(d), kmap, vmap, p, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "sparse decode launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "paged_attention_decode_sparse") : WLLM_OK;
}

}  // namespace

extern "C" {

int wllm_rotate_and_cache(const wllm_tensor* q_out, const wllm_tensor* q, const wllm_tensor* key, const wllm_tensor* value,
                          const wllm_tensor* k_cache, const wllm_tensor* v_cache, const wllm_tensor* slot_mapping,
                          const wllm_tensor* positions, const wllm_tensor* cos_sin, const wllm_tensor* q_weight,
                          const wllm_tensor* k_weight, const wllm_rotary* how, wllm_stream stream) {
  return rotate_call(q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight, k_weight, how,
                     false, 1.f, 1.f, stream);
}

int wllm_rotate_and_cache_fp8(const wllm_tensor* q_out, const wllm_tensor* q, const wllm_tensor* key,
                              const wllm_tensor* value, const wllm_tensor* k_cache, const wllm_tensor* v_cache,
                              const wllm_tensor* slot_mapping, const wllm_tensor* positions, const wllm_tensor* cos_sin,
                              const wllm_tensor* q_weight, const wllm_tensor* k_weight, const wllm_rotary* how,
                              float k_scale, float v_scale, wllm_stream stream) {
  return rotate_call(q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight, k_weight, how,
                     true, k_scale, v_scale, stream);
}

int wllm_update_key_bounds(const wllm_tensor* key_bounds, const wllm_tensor* k_cache, const wllm_tensor* block_tables,
                           const wllm_tensor* context_lens, const wllm_tensor* query_start_loc, int block_size,
                           wllm_stream stream) {
  int rc;
  if ((rc = check_desc(key_bounds, "key_bounds", 4)) || (rc = check_desc(k_cache, "k_cache", 4)) ||
      (rc = check_desc(block_tables, "block_tables", 2)) || (rc = check_desc(context_lens, "context_lens", 1)) ||
      (query_start_loc != nullptr && (rc = check_desc(query_start_loc, "query_start_loc", 1))))
    return rc;
  const int dt = k_cache->dtype;
  if (!is_float(dt) && dt != WLLM_FP8_E4M3)
    return fail(WLLM_ERR_INVALID_ARG, "k_cache: dtype must be F32, F16, BF16 or FP8_E4M3");
  if (key_bounds->dtype != dt) return fail(WLLM_ERR_INVALID_ARG, "key_bounds must have the dtype of k_cache");
  const int64_t nb = k_cache->shape[0], hkv = k_cache->shape[1], bs = k_cache->shape[2], d = k_cache->shape[3];
  const int64_t B = context_lens->shape[0];
  if ((rc = check_pool_args(hkv, bs, static_cast<int>(std::min<int64_t>(hkv, INT32_MAX)), block_size))) return rc;
  if (key_bounds->shape[0] != nb || key_bounds->shape[1] != hkv || key_bounds->shape[2] != 2 || key_bounds->shape[3] != d)
    return fail(WLLM_ERR_INVALID_ARG, "key_bounds must be [N_b, Hkv, 2, D] of k_cache");
  if (!contiguous(k_cache) || !contiguous(key_bounds)) return fail(WLLM_ERR_INVALID_ARG, "k_cache and key_bounds must be dense");
  if ((rc = check_tables(block_tables, context_lens, B, nb, bs))) return rc;
  if (query_start_loc != nullptr) {
    if (query_start_loc->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc: dtype must be I32");
    if (query_start_loc->shape[0] != B + 1) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc must have B+1 entries");
    if (B > 0 && query_start_loc->stride[0] != 1) return fail(WLLM_ERR_INVALID_ARG, "query_start_loc must be contiguous");
  }
  if (d != 64 && d != 128 && d != 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)d);
  if (hkv > 65535 || B > INT32_MAX / 8) return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  if (B == 0 || hkv == 0) return WLLM_OK;
  if (nb < 1) return fail(WLLM_ERR_INVALID_ARG, "the pool has no blocks");
  if (!aligned(k_cache->data, 16) || !aligned(key_bounds->data, 16))
    return fail(WLLM_ERR_INVALID_ARG, "cache and bounds base pointers must be 16-byte aligned");
  BoundsParams p{};
  p.bounds = static_cast<uint8_t*>(key_bounds->data);
  p.k_cache = static_cast<const uint8_t*>(k_cache->data);
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.query_start_loc = query_start_loc != nullptr ? static_cast<const int32_t*>(query_start_loc->data) : nullptr;
  p.num_seqs = static_cast<int>(B);
  p.num_kv_heads = static_cast<int>(hkv);
  p.num_blocks = static_cast<int>(nb);
  p.log2_bs = ilog2(bs);
  p.max_tokens = static_cast<int>(block_tables->shape[1] * bs);
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(launch_key_bounds(dt, static_cast<int>(d), p, s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "key bounds launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "update_key_bounds") : WLLM_OK;
}

int wllm_select_blocks(const wllm_tensor* selected, const wllm_tensor* q, const wllm_tensor* key_bounds,
                       const wllm_tensor* block_tables, const wllm_tensor* context_lens, int num_kv_heads, int block_size,
                       int num_sink, int num_recent, wllm_stream stream) {
  int rc;
  if ((rc = check_desc(selected, "selected", 3)) || (rc = check_desc(q, "q", 3)) ||
      (rc = check_desc(key_bounds, "key_bounds", 4)) || (rc = check_desc(block_tables, "block_tables", 2)) ||
      (rc = check_desc(context_lens, "context_lens", 1)))
    return rc;
  const int dt = q->dtype;
  if (!is_float(dt)) return fail(WLLM_ERR_INVALID_ARG, "q: dtype must be F32, F16 or BF16");
  if (key_bounds->dtype != dt && !(key_bounds->dtype == WLLM_FP8_E4M3 && dt != WLLM_F32))
    return fail(WLLM_ERR_INVALID_ARG, "key_bounds must have the dtype of q, or FP8_E4M3 with F16 or BF16 queries");
  if (selected->dtype != WLLM_I32) return fail(WLLM_ERR_INVALID_ARG, "selected: dtype must be I32");
  const int64_t B = q->shape[0], hq = q->shape[1], d = q->shape[2];
  const int64_t nb = key_bounds->shape[0], hkv = key_bounds->shape[1], top = selected->shape[2];
  if (key_bounds->shape[2] != 2 || key_bounds->shape[3] != d)
    return fail(WLLM_ERR_INVALID_ARG, "key_bounds must be [N_b, Hkv, 2, D] with q's D");
  if (hkv != num_kv_heads)
    return fail(WLLM_ERR_INVALID_ARG, "num_kv_heads %d differs from key_bounds dim %lld", num_kv_heads, (long long)hkv);
  if (hkv <= 0 || hq % hkv != 0) return fail(WLLM_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if ((rc = check_tables(block_tables, context_lens, B, nb, block_size))) return rc;
  if (selected->shape[0] != B || selected->shape[1] != hkv)
    return fail(WLLM_ERR_INVALID_ARG, "selected must be [B, Hkv, top]");
  if (top > 1 && selected->stride[2] != 1) return fail(WLLM_ERR_INVALID_ARG, "selected rows must be contiguous");
  if (!contiguous(key_bounds)) return fail(WLLM_ERR_INVALID_ARG, "key_bounds must be dense");
  if (d > 1 && q->stride[2] != 1) return fail(WLLM_ERR_INVALID_ARG, "q last dimension must be contiguous");
  if (num_sink < 0 || num_recent < 1)
    return fail(WLLM_ERR_INVALID_ARG, "num_sink must not be negative and num_recent at least 1 (the last block has no bounds yet)");
  if (int64_t(num_sink) + num_recent > top)
    return fail(WLLM_ERR_INVALID_ARG, "num_sink + num_recent exceed the %lld selected blocks", (long long)top);
  if (d != 64 && d != 128 && d != 256)
    return fail(WLLM_ERR_UNSUPPORTED, "head_dim %lld not supported (64, 128, 256)", (long long)d);
  if (hq > 65535 || top > INT32_MAX || B * hkv > INT32_MAX / 8) return fail(WLLM_ERR_UNSUPPORTED, "sizes too large");
  if (B == 0) return WLLM_OK;
  const int64_t mb = block_tables->shape[1];
  if (mb > select_max_blocks())
    return fail(WLLM_ERR_UNSUPPORTED, "block tables of %lld blocks not supported (%d at most)", (long long)mb,
                select_max_blocks());
  if (nb < 1) return fail(WLLM_ERR_INVALID_ARG, "the pool has no blocks");
  if (!aligned(key_bounds->data, 16)) return fail(WLLM_ERR_INVALID_ARG, "key_bounds must be 16-byte aligned");
  if (!aligned(q->data, static_cast<uintptr_t>(elt_size(dt))))
    return fail(WLLM_ERR_INVALID_ARG, "q must be aligned to its element size");
  SelectParams p{};
  p.selected = static_cast<int32_t*>(selected->data);
  p.sel_sb = selected->stride[0], p.sel_sh = selected->stride[1];
  p.q = q->data;
  p.q_sb = q->stride[0], p.q_sh = q->stride[1];
  p.bounds = static_cast<const uint8_t*>(key_bounds->data);
  p.block_tables = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.num_seqs = static_cast<int>(B);
  p.num_kv_heads = static_cast<int>(hkv);
  p.group = static_cast<int>(hq / hkv);
  p.num_blocks = static_cast<int>(nb);
  p.log2_bs = ilog2(block_size);
  p.max_tokens = static_cast<int>(mb * block_size);
  p.top = static_cast<int>(top);
  p.sink = num_sink;
  p.recent = num_recent;
  DeviceState* s = nullptr;
  if ((rc = locked_state(&s))) return rc;
  p.err = s->err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = static_cast<cudaError_t>(
      launch_select(dt, key_bounds->dtype, static_cast<int>(d), p, static_cast<int>(mb), s->num_sms, st));
  if (e != cudaSuccess) return cuda_fail(e, "select launch");
  return env_flag("WLLM_CHECK") ? collect_device_errors(s, st, "select_blocks") : WLLM_OK;
}

int wllm_paged_attention_decode_sparse(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache,
                                       const wllm_tensor* v_cache, const wllm_tensor* block_tables,
                                       const wllm_tensor* context_lens, const wllm_tensor* selected, int num_kv_heads,
                                       float scale, int block_size, wllm_stream stream) {
  return sparse_call(out, q, k_cache, v_cache, block_tables, context_lens, selected, num_kv_heads, scale, block_size, false,
                     1.f, 1.f, stream);
}

int wllm_paged_attention_decode_sparse_fp8(const wllm_tensor* out, const wllm_tensor* q, const wllm_tensor* k_cache,
                                           const wllm_tensor* v_cache, const wllm_tensor* block_tables,
                                           const wllm_tensor* context_lens, const wllm_tensor* selected, int num_kv_heads,
                                           float scale, float k_scale, float v_scale, int block_size, wllm_stream stream) {
  return sparse_call(out, q, k_cache, v_cache, block_tables, context_lens, selected, num_kv_heads, scale, block_size, true,
                     k_scale, v_scale, stream);
}

}  // extern "C"
