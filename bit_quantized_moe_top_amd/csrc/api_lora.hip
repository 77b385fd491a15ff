// C ABI of the shared projection with low-rank adapters (declared in
// include/moeq_lora.h): argument validation before any HIP call, the device check, and
// the launches on the caller's stream.
#include "api.hpp"
#include "lora_kernels.hpp"

using moeq::aligned16;
using moeq::aligned_to;
using moeq::as_stream;
using moeq::check_device;
using moeq::check_plan;
using moeq::launch_status;

namespace {

constexpr int64_t kMaxGrid = 0xFFFFFF;         // workgroups of 256 threads in one launch
constexpr int kMaxRows = 1 << 24, kMaxK = 1 << 20, kMaxN = 1 << 20;

int check_shape(const moeq::LoraShape& s) {
  if (s.M < 0 || s.N <= 0 || s.K <= 0 || s.L <= 0 || s.r <= 0) return MOEQ_ERR_INVALID_ARG;
  if (s.slices != 1 && s.slices != 2) return MOEQ_ERR_INVALID_ARG;
  if (s.epilogue != MOEQ_EPI_NONE && s.epilogue != MOEQ_EPI_SILU_MUL) return MOEQ_ERR_INVALID_ARG;
  const bool halves = s.slices == 2 || s.epilogue == MOEQ_EPI_SILU_MUL;
  if (s.M >= kMaxRows || s.K % 8 != 0 || s.K >= kMaxK || s.N % (halves ? 32 : 16) != 0 ||
      s.N > kMaxN || s.r % 8 != 0 || s.r > MOEQ_LORA_MAX_RANK || s.L > MOEQ_MAX_ADAPTERS)
    return MOEQ_ERR_UNSUPPORTED;
  if (int64_t((s.M + 63) / 64) * ((s.N + 63) / 64) > kMaxGrid) return MOEQ_ERR_UNSUPPORTED;
  return MOEQ_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

}  // namespace

extern "C" {

int moe_adapter_plan(const int32_t* ids, int M, int L, void* plan, size_t plan_bytes, void* stream) {
  if (M < 0 || L <= 0) return MOEQ_ERR_INVALID_ARG;
  if (M >= kMaxRows || L > MOEQ_MAX_ADAPTERS) return MOEQ_ERR_UNSUPPORTED;
  if (!plan || (M > 0 && !ids) || !aligned_to(ids, 4)) return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_plan(plan, plan_bytes, L + 1, M)) return rc;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_adapter_plan(ids, M, L, plan, as_stream(stream)));
}

size_t moe_shared_gemm_lora_ws_size(int M, int N, int K, int L, int slices, int r) {
  const moeq::LoraShape s = {M, N, K, L, slices, r, K, MOEQ_EPI_NONE};
  return check_shape(s) ? 0 : moeq::lora_path(s).ws_bytes();
}

int moe_shared_gemm_lora_bf16(const uint16_t* a, int64_t ld_a, const uint16_t* w, int M, int N,
                              int K, const uint16_t* lora_a, const uint16_t* lora_b,
                              const float* scale, int L, int slices, int r, const void* plan,
                              size_t plan_bytes, int epilogue, uint16_t* out, void* ws,
                              size_t ws_bytes, void* stream) {
  const moeq::LoraShape s = {M, N, K, L, slices, r, ld_a, epilogue};
  if (int rc = check_shape(s)) return rc;
  if (ld_a < K) return MOEQ_ERR_INVALID_ARG;
  if (ld_a % 8 != 0 || ld_a > int64_t(1) << 38) return MOEQ_ERR_UNSUPPORTED;
  if (M == 0) return MOEQ_OK;
  if (!a || !w || !lora_a || !lora_b || !scale || !plan || !out || !ws) return MOEQ_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(w) || !aligned16(lora_a) || !aligned16(lora_b) ||
      !aligned16(out) || !aligned_to(scale, 4) || !aligned_to(ws, 256))
    return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_plan(plan, plan_bytes, L + 1, M)) return rc;
  const size_t need = moeq::lora_path(s).ws_bytes();
  if (ws_bytes < need) return MOEQ_ERR_WORKSPACE;
  // what is written must not lie over what is read
  const int64_t cols = epilogue == MOEQ_EPI_SILU_MUL ? N / 2 : N;
  const struct { const void* p; int64_t n; } in[] = {
      {a, 2 * ((int64_t(M) - 1) * ld_a + K)}, {w, 2 * int64_t(N) * K},
      {lora_a, 2 * int64_t(L) * slices * r * K}, {lora_b, 2 * int64_t(L) * N * r},
      {scale, 4 * int64_t(L)}, {plan, int64_t(moeq::plan_words(L + 1, M)) * 4}};
  for (const auto& i : in)
    if (overlap(i.p, i.n, out, 2 * int64_t(M) * cols) || overlap(i.p, i.n, ws, int64_t(need)))
      return MOEQ_ERR_INVALID_ARG;
  if (overlap(out, 2 * int64_t(M) * cols, ws, int64_t(need))) return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_device()) return rc;
  const moeq::LoraArgs args = {a, w, lora_a, lora_b, scale, const_cast<void*>(plan), out, ws};
  return launch_status(moeq::launch_shared_gemm_lora(args, s, as_stream(stream)));
}

}  // extern "C"
