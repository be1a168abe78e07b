// rowops_host.h -- host-side checks and launching shared by the row operators'
// C calls.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <stdint.h>
#include <string.h>

#include "exact_row_top.h"

namespace ert {

inline bool at(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dtype_ok(int32_t d) { return d >= TOPK_DT_F32 && d <= TOPK_DT_F16; }
inline uintptr_t elem(int32_t d) { return d == TOPK_DT_F32 ? 4 : 2; }

// Whether two arrays of `bytes` each (or one that is not given) lie apart.
inline bool apart(const void* a, const void* b, uint64_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !a || !b || (x < y ? y - x : x - y) >= bytes;
}

// Whether the current device is gfx950 (0 unknown, 1 yes, 2 no per device).
constexpr int kMaxDev = 64;
inline std::atomic<int> g_arch[kMaxDev];

inline int device_ok() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDev) return TOPK_EDEVICE;
  int a = g_arch[dev].load(std::memory_order_relaxed);
  if (a == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return TOPK_EDEVICE;
    a = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch[dev].store(a, std::memory_order_relaxed);
  }
  return a == 1 ? TOPK_OK : TOPK_EDEVICE;
}

inline int launch(const void* kernel, int64_t grid, int block, void* params, size_t lds, hipStream_t stream) {
  if (!kernel || grid < 1 || grid >= ((int64_t)1 << 31)) return TOPK_EINVAL;
  void* args[] = {params};
  if (hipLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)block), args, lds, stream) !=
      hipSuccess) {
    (void)hipGetLastError();  // reported here, not by the caller's next call
    return TOPK_ELAUNCH;
  }
  return TOPK_OK;
}

}  // namespace ert
