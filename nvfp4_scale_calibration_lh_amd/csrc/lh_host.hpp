// Host helpers shared by the C-ABI translation units: the calling thread's error message, pointer
// and alignment checks, and the guard that makes the pointers' device current for one call.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/lh.h"

namespace lh {
namespace host {

// Message of the last error on this thread; a fixed buffer, so that reporting cannot throw.
inline thread_local char g_last_error[512] = "";

inline lh_status fail(lh_status code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}

inline lh_status ok() {
  g_last_error[0] = 0;
  return LH_OK;
}

inline lh_status hip_fail(hipError_t e, const char* what) {
  (void)hipGetLastError();  // clear the sticky launch error so the caller's next call is clean
  return fail(LH_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool dtype_ok(int d) { return d == LH_DTYPE_F32 || d == LH_DTYPE_BF16; }

// Device that owns `p`, or -1 (with the error message set) if p is not device memory.
inline int device_of(const void* p, const char* name) {
  hipPointerAttribute_t attr;
  std::memset(&attr, 0, sizeof(attr));
  hipError_t e = hipPointerGetAttributes(&attr, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    fail(LH_ERR_INVALID_ARGUMENT, "%s is not a device pointer (%s)", name, hipGetErrorString(e));
    return -1;
  }
  if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) {
    fail(LH_ERR_INVALID_ARGUMENT, "%s is not device memory", name);
    return -1;
  }
  return attr.device;
}

struct PtrCheck {
  const void* p;
  const char* name;
};

// All non-null pointers must be device memory of one device, 16-byte aligned where required.
inline lh_status check_pointers(std::initializer_list<PtrCheck> ptrs, int* dev_out) {
  int dev = -1;
  for (const PtrCheck& c : ptrs) {
    if (!c.p) continue;
    int d = device_of(c.p, c.name);
    if (d < 0) return LH_ERR_INVALID_ARGUMENT;
    if (dev >= 0 && d != dev) return fail(LH_ERR_INVALID_ARGUMENT, "%s is on device %d, other pointers on device %d", c.name, d, dev);
    dev = d;
  }
  if (dev < 0) return fail(LH_ERR_INVALID_ARGUMENT, "no device pointer given");
  *dev_out = dev;
  return LH_OK;
}

inline lh_status check_aligned(const void* p, const char* name) {
  if (p && (reinterpret_cast<uintptr_t>(p) % 16) != 0)
    return fail(LH_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", name);
  return LH_OK;
}

// One of the 126 positive finite values: 3 bits below the leading one, or a multiple of 2^-9 (a search
// through them took 0.3 us a call).
inline bool e4m3_value(float x) {
  if (!(x >= 0x1p-9f && x <= 448.0f)) return false;
  if (x < 0x1p-6f) return x * 512.0f == std::floor(x * 512.0f);
  uint32_t bits;
  std::memcpy(&bits, &x, sizeof bits);
  return (bits & 0xFFFFF) == 0;
}

inline lh_status check_stride(int64_t stride, int64_t least, lh_dtype dtype, const char* name) {
  if (stride < least || stride % (dtype == LH_DTYPE_BF16 ? 8 : 4))
    return fail(LH_ERR_INVALID_ARGUMENT, "%s must be at least %lld elements and a multiple of 16 bytes (got %lld)", name,
                (long long)least, (long long)stride);
  return LH_OK;
}

// Status of a call whose launch returned e.
inline lh_status launched(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration) return fail(LH_ERR_INVALID_ARGUMENT, "%s: too large for one call (2^32 work-items or more)", what);
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

// Switches to `dev` for the lifetime of the guard and checks that it is a gfx950 device.
class DeviceGuard {
 public:
  lh_status enter(int dev) {
    hipError_t e = hipGetDevice(&prev_);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (prev_ != dev) {
      e = hipSetDevice(dev);
      if (e != hipSuccess) return hip_fail(e, "hipSetDevice");
      switched_ = true;
    }
    static std::atomic<signed char> arch_ok[64];        // 0 unknown, 1 gfx950, -1 another part
    if (dev < 0 || dev >= 64) return fail(LH_ERR_UNSUPPORTED, "device %d out of range", dev);
    if (arch_ok[dev] == 0) {
      hipDeviceProp_t prop;
      e = hipGetDeviceProperties(&prop, dev);
      if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
      arch_ok[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    }
    if (arch_ok[dev] < 0) return fail(LH_ERR_UNSUPPORTED, "device %d is not gfx950 (MI355X)", dev);
    return LH_OK;
  }
  ~DeviceGuard() {
    if (switched_) (void)hipSetDevice(prev_);
  }

 private:
  int prev_ = 0;
  bool switched_ = false;
};

}  // namespace host
}  // namespace lh
