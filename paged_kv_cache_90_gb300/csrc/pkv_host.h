// pkv_host.h — host-side pieces of the C ABI shared by its translation units
// (pkv_api.cu, token_api.cu): error reporting, descriptor checks, per-device state and the
// decode workspace.  Not part of the public ABI.
#pragma once

#include <mutex>

#include "pkv_internal.h"

namespace pkv {

struct DeviceState {
  bool ready = false;
  unsigned int* err = nullptr;  // address of the device's error word
  int num_sms = 0;
  void* ws = nullptr;           // decode workspace
  size_t ws_bytes = 0;
  // Held from a workspace check to the end of the launch that uses the workspace, so
  // a growth on one host thread cannot free a buffer another thread is queueing work on.
  std::mutex ws_use;
};

// Records a message (printf format) as the thread's last error and returns `st`.
pkv_status fail(pkv_status st, const char* fmt, ...);
// The current device's state.
pkv_status device_state(DeviceState** out);
// Grows the current device's workspace to `bytes`; the caller holds s->ws_use.
pkv_status ensure_workspace(DeviceState* s, size_t bytes, cudaStream_t stream);
// Maps a launch result to a status (and, with debug sync on, checks the device).
pkv_status finish_call(DeviceState* s, cudaError_t launch_err, cudaStream_t stream, const char* what);
// Whether calls only validate their arguments (PKV_OPT_DRY_RUN).
bool dry_run();

int elt_bytes(int dtype);
const char* dtype_name(int dtype);
bool aligned16(const void* p);
bool supported_head_dim(int64_t d);
bool supported_block_size(int64_t bs);
pkv_status check_basic(const pkv_tensor* t, const char* name, int ndim);
pkv_status check_dtype(const pkv_tensor* t, const char* name, int a, int b = -1, int c = -1);
// A cache descriptor; `i8`: token-scaled PKV_I8 caches are taken too.
pkv_status check_cache(const pkv_tensor* c, const char* name, bool i8 = false);
// Scales of a token-scaled cache, [num_blocks, num_kv_heads, block_size] f32.
pkv_status check_scales(const pkv_tensor* t, const char* name);
bool same_layout(const pkv_tensor* a, const pkv_tensor* b);

}  // namespace pkv
