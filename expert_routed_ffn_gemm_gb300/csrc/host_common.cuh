// Host-side pieces shared by the C entry points: pointer checks, error
// tracing, the device of a call, and the driver's tensor-map encoder.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "../../include/moe.h"

namespace moe {

// cuTensorMapEncodeTiled, looked up once per process (NULL without a driver).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

inline bool load_encode() { return tensor_map_encode() != nullptr; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device (or managed) memory.
inline bool is_device_ptr(const void* p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

// The buffers of one call: memory of one device, the given one or that of the
// first buffer (a kernel that reads another device's memory faults unless peer
// access was enabled).  Managed memory goes with any.
class CallBuffers {
 public:
  explicit CallBuffers(int device = -1) : device_(device) {}
  // Not null, aligned, device memory of the call's device.
  bool need(const void* p, uintptr_t align = 16) {
    if (p == nullptr || !aligned(p, align)) return false;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    if (at.type == cudaMemoryTypeManaged) {
      managed_on_ = at.device;
      return true;
    }
    if (at.type != cudaMemoryTypeDevice) return false;
    if (device_ < 0) device_ = at.device;
    return at.device == device_;
  }
  // The same for a buffer that may be absent.
  bool maybe(const void* p, uintptr_t align = 16) { return p == nullptr || need(p, align); }
  int device() const { return device_ >= 0 ? device_ : managed_on_; }

 private:
  int device_, managed_on_ = 0;
};

// MOE_TRACE_ERRORS=1 in the environment: every failing CUDA call is reported
// on stderr with its source line and error name.
inline bool trace_errors() {
  static const bool on = [] {
    const char* v = std::getenv("MOE_TRACE_ERRORS");
    return v != nullptr && v[0] == '1';
  }();
  return on;
}

inline int cuda_failed(cudaError_t e, const char* what, int line) {
  if (trace_errors()) std::fprintf(stderr, "moe: line %d: %s -> %s\n", line, what, cudaGetErrorName(e));
  return MOE_ERR_CUDA;
}

#define MOE_CUDA(call)                                   \
  do {                                                   \
    const cudaError_t moe_e_ = (call);                   \
    if (moe_e_ != cudaSuccess) {                         \
      return ::moe::cuda_failed(moe_e_, #call, __LINE__); \
    }                                                    \
  } while (0)

// Every call on a handle runs with the handle's device current in the calling
// thread (and puts the previous device back): a thread that has not used CUDA
// yet gets the device's primary context before the first driver call (the
// tensor-map encoding), and a caller working on another device is unaffected.
struct DeviceGuard {
  int prev = -1, dev;
  explicit DeviceGuard(int d) : dev(d) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      cudaGetLastError();
      prev = -1;
    }
    if (cudaSetDevice(dev) != cudaSuccess) cudaGetLastError();
  }
  ~DeviceGuard() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
};

}  // namespace moe
