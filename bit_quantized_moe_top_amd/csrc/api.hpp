// Helpers of the C-ABI layer: the device check and argument tests shared by the
// entry points (api.hip, api_mx.hip).
#pragma once

#include <string.h>

#include "kernels.hpp"

namespace moeq {

constexpr int kMaxDevices = 64;
// per-device result of the architecture check: 0 unknown, 1 gfx950, -1 other
inline int g_device_ok[kMaxDevices];

inline int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MOEQ_ERR_DEVICE;
  if (dev < kMaxDevices && g_device_ok[dev] != 0) return g_device_ok[dev] > 0 ? MOEQ_OK : MOEQ_ERR_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOEQ_ERR_DEVICE;
  const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_device_ok[dev] = ok ? 1 : -1;
  return ok ? MOEQ_OK : MOEQ_ERR_DEVICE;
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

inline int launch_status(hipError_t err) { return err == hipSuccess ? MOEQ_OK : MOEQ_ERR_LAUNCH; }

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// a plan read by a kernel: 4-byte aligned and at least moe_plan_size(E, R) bytes
inline int check_plan(const void* plan, size_t plan_bytes, int E, int R) {
  if (!aligned_to(plan, 4)) return MOEQ_ERR_INVALID_ARG;
  if (plan_bytes < plan_words(E, R) * sizeof(int32_t)) return MOEQ_ERR_WORKSPACE;
  return MOEQ_OK;
}

}  // namespace moeq
