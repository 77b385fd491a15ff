// Launchers of expert routing (route_experts.hip).
// Arguments are validated by the C-ABI layer first; each returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moeq_route.h"

namespace moeq {

struct RouteShape {
  int T, E, k;
  int64_t ld;               // row stride of the logits, elements
  int scoring;              // MOEQ_SCORE_*
  int n_group, topk_group, group_best;
  int renormalize;
  float scale;
};

hipError_t launch_route_experts(const void* logits, int logits_dtype, const float* bias,
                                const RouteShape& shape, int32_t* ids, float* w,
                                hipStream_t stream);

}  // namespace moeq
