// C ABI of moe_route_experts (declared in include/moeq_route.h): argument
// validation before any HIP call, the device check, and the launch on the caller's stream.
#include "api.hpp"
#include "serve_kernels.hpp"

#include <math.h>

using moeq::aligned_to;
using moeq::as_stream;
using moeq::check_device;
using moeq::launch_status;

extern "C" {

int moe_route_experts(const void* logits, int logits_dtype, int64_t ld_logits, const float* bias,
                      int T, int E, int k, int scoring, int n_group, int topk_group,
                      int group_best, int renormalize, float scale, int32_t* topk_ids,
                      float* topk_w, void* stream) {
  if (T < 0 || E <= 0 || k <= 0 || n_group <= 0 || topk_group <= 0 || ld_logits < E ||
      !isfinite(scale))
    return MOEQ_ERR_INVALID_ARG;
  if (logits_dtype != MOEQ_F32 && logits_dtype != MOEQ_BF16) return MOEQ_ERR_INVALID_ARG;
  if (scoring != MOEQ_SCORE_SOFTMAX && scoring != MOEQ_SCORE_SIGMOID) return MOEQ_ERR_INVALID_ARG;
  if (group_best != 1 && group_best != 2) return MOEQ_ERR_INVALID_ARG;
  if (E > MOEQ_MAX_EXPERTS || k > MOEQ_MAX_TOPK || n_group > MOEQ_MAX_GROUPS || T > 1 << 25 ||
      ld_logits > int64_t(1) << 40)
    return MOEQ_ERR_UNSUPPORTED;
  if (E % n_group != 0 || topk_group > n_group || k > topk_group * (E / n_group))
    return MOEQ_ERR_INVALID_ARG;
  if (T == 0) return MOEQ_OK;
  if (!logits || !topk_ids || !topk_w) return MOEQ_ERR_INVALID_ARG;
  if (!aligned_to(logits, logits_dtype == MOEQ_BF16 ? 2 : 4) || !aligned_to(bias, 4) ||
      !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4))
    return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_device()) return rc;
  const moeq::RouteShape shape = {T, E, k, ld_logits, scoring, n_group, topk_group, group_best,
                                  renormalize, scale};
  return launch_status(moeq::launch_route_experts(logits, logits_dtype, bias, shape, topk_ids,
                                                  topk_w, as_stream(stream)));
}

}  // extern "C"
