// api_internal.h -- what the translation units behind the C ABI share: status
// and message of a failed call, per-device state, and descriptor checks.
// Defined in api.cu; not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "wllm.h"

namespace wllm {

// Record the message for wllm_last_error() and return `status`.
int fail(int status, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

struct DeviceState {
  bool ready = false;
  int num_sms = 0;
  int* err = nullptr;               // device error word
  uint8_t* ws = nullptr;            // split-KV workspace
  size_t ws_bytes = 0;
  bool ws_owned = true;
  size_t counter_bytes = 0;         // leading bytes reserved for arrival counters (kept zero)
};

extern std::mutex g_mutex;          // guards the per-device states and the shared workspace

// Current device's state, created on first use (error word allocated and zeroed).
int device_state(DeviceState** out);

// Read and clear the error word after synchronising `stream` (check mode).
int collect_device_errors(DeviceState* s, cudaStream_t stream, const char* op);

bool env_flag(const char* name);
bool env_is(const char* name, const char* value);
long long env_int(const char* name, long long dflt);

int elt_size(int dtype);
bool is_float(int dtype);
bool is_pow2(int64_t x);
int ilog2(int64_t x);
int64_t numel(const wllm_tensor* t);
int check_desc(const wllm_tensor* t, const char* name, int ndim);
bool contiguous(const wllm_tensor* t);
bool same_shape(const wllm_tensor* a, const wllm_tensor* b);
bool aligned(const void* p, uintptr_t a);
bool positive_finite(float x);

// TMA map of a [N_b][Hkv][bs][D] pool: 3-D view {D, Hkv*bs, N_b}; one box is
// 128 bytes of a row by min(bs, 16) rows, 128-byte swizzled.
int make_pool_map(CUtensorMap* map, const void* base, int dtype, int64_t num_blocks, int64_t hkv, int64_t bs, int64_t d,
                  const char* name);

}  // namespace wllm
