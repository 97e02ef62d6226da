// Host helpers shared by the C ABI's translation units: operand checks, the
// device's CU count, and launching.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dpg.h"
#include "planner.h"

namespace dpg {

// CU count of the current device (fast mode only), cached per device id.
inline int device_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return kDetCus;
  if (cached[dev] == 0) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
      cus = kDetCus;
    cached[dev] = cus;
  }
  return cached[dev];
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

struct Mat {
  const void* ptr;
  int64_t ld, rows, cols;
  int elt;  // bytes per element
};

inline dpg_status check_mat(const Mat& m) {
  if (m.rows < 0 || m.cols < 0) return DPG_ERR_INVALID_ARG;
  if (m.rows == 0 || m.cols == 0) return DPG_OK;  // empty: pointer and ld unused
  if (!m.ptr) return DPG_ERR_INVALID_ARG;
  if (m.ld < m.cols) return DPG_ERR_INVALID_ARG;
  if (!aligned16(m.ptr) || (m.ld * m.elt) % 16 != 0 || m.cols % 8 != 0) return DPG_ERR_ALIGNMENT;
  return DPG_OK;
}

// a launch takes fewer than 2^32 threads
inline dpg_status launch(const void* kernel, int64_t grid, int threads, size_t lds, void** args, hipStream_t stream) {
  if (grid * threads >= (1ll << 32)) return DPG_ERR_UNSUPPORTED;
  const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), args, lds, stream);
  return e == hipSuccess ? DPG_OK : DPG_ERR_HIP;
}

}  // namespace dpg
