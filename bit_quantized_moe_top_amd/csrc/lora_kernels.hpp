// Launchers of the shared projection with low-rank adapters (lora.hip) and of its
// plan (permute.hip).  Arguments are validated by the C-ABI layer first; each returns
// hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "lora_paths.hpp"

namespace moeq {

struct LoraArgs {
  const uint16_t *a, *w, *lora_a, *lora_b;
  const float* scale;
  void* plan;
  uint16_t* out;
  void* ws;
};

hipError_t launch_adapter_plan(const int32_t* ids, int M, int L, void* plan, hipStream_t stream);

hipError_t launch_shared_gemm_lora(const LoraArgs& args, const LoraShape& s, hipStream_t stream);

}  // namespace moeq
