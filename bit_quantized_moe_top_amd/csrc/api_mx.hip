// C ABI of the MXFP4 calls (declared in include/moeq_mx.h): argument validation
// before any HIP call, the device check, and the launches on the caller's stream.
#include "../../include/moeq_mx.h"
#include "api.hpp"
#include "mx_kernels.hpp"

using moeq::aligned16;
using moeq::aligned_to;
using moeq::as_stream;
using moeq::check_device;
using moeq::check_plan;
using moeq::launch_status;

static_assert(MOEQ_FEW_TOKENS == moeq::kFewTokens, "header and library agree");

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 35;
constexpr int64_t kMaxGrid = 0xFFFFFF;         // workgroups of 256 threads in one launch

bool dtype_ok(int d) { return d == MOEQ_F32 || d == MOEQ_BF16; }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

// M rows of K elements in blocks of 32
int check_rows(int64_t M, int K) {
  if (M < 0 || K <= 0) return MOEQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > kMaxElements / K) return MOEQ_ERR_UNSUPPORTED;
  return MOEQ_OK;
}

int check_product(int E, int N, int K) {
  if (E <= 0 || N <= 0 || K <= 0) return MOEQ_ERR_INVALID_ARG;
  if (E > MOEQ_MAX_EXPERTS || N % 32 != 0 || K % 32 != 0 || K > MOEQ_MX_MAX_K)
    return MOEQ_ERR_UNSUPPORTED;
  return MOEQ_OK;
}

int check_few(int T, int k, int H, int I) {
  if (T < 0 || k <= 0 || H <= 0 || I <= 0) return MOEQ_ERR_INVALID_ARG;
  if (T > MOEQ_FEW_TOKENS || k > MOEQ_MAX_TOPK || H % 32 != 0 || I % 32 != 0 ||
      H > MOEQ_MX_MAX_K || I > MOEQ_MX_MAX_K)
    return MOEQ_ERR_UNSUPPORTED;
  return MOEQ_OK;
}

}  // namespace

extern "C" {

int quant_mxfp4(const void* x, int x_dtype, int64_t M, int K, int64_t ld_x, uint8_t* q,
                uint8_t* scale, void* stream) {
  if (int rc = check_rows(M, K)) return rc;
  if (!dtype_ok(x_dtype) || ld_x < K) return MOEQ_ERR_INVALID_ARG;
  if (ld_x % 8 != 0) return MOEQ_ERR_UNSUPPORTED;
  if (M == 0) return MOEQ_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q)) return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_quant_mxfp4(x, x_dtype, M, K, ld_x, q, scale, as_stream(stream)));
}

int dequant_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t M, int K, void* out,
                  int out_dtype, void* stream) {
  if (int rc = check_rows(M, K)) return rc;
  if (!dtype_ok(out_dtype)) return MOEQ_ERR_INVALID_ARG;
  if (M == 0) return MOEQ_OK;
  if (!q || !scale || !out || !aligned_to(q, 4) || !aligned16(out)) return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_dequant_mxfp4(q, scale, M, K, out, out_dtype, as_stream(stream)));
}

int moe_tile_mxfp4_weights(const uint8_t* q, const uint8_t* scale, int64_t rows, int K, uint8_t* w,
                           uint8_t* ws, void* stream) {
  if (int rc = check_rows(rows, K)) return rc;
  if (rows % 16 != 0 || K > MOEQ_MX_MAX_K) return MOEQ_ERR_UNSUPPORTED;
  if (rows == 0) return MOEQ_OK;
  const int64_t units = rows / 16 * ((K + 511) / 512);
  if (units > kMaxGrid) return MOEQ_ERR_UNSUPPORTED;
  if (!q || !scale || !w || !ws || !aligned16(q) || !aligned16(w) || !aligned16(ws))
    return MOEQ_ERR_INVALID_ARG;
  const int64_t nq = rows * (K / 2), ns = rows * (K / 32), nw = units * 4096, nws = units * 256;
  if (overlap(q, nq, w, nw) || overlap(q, nq, ws, nws) || overlap(scale, ns, w, nw) ||
      overlap(scale, ns, ws, nws) || overlap(w, nw, ws, nws))
    return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_tile_mxfp4(q, scale, rows, K, w, ws, as_stream(stream)));
}

int moe_grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, int a_topk, const void* plan,
                           size_t plan_bytes, int E, int R, const uint8_t* w, const uint8_t* ws,
                           int N, int K, int epilogue, void* out, int out_dtype, void* stream) {
  if (R < 0 || a_topk < 0) return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_product(E, N, K)) return rc;
  if (epilogue != MOEQ_EPI_NONE && epilogue != MOEQ_EPI_SILU_MUL) return MOEQ_ERR_INVALID_ARG;
  if (!dtype_ok(out_dtype) || (epilogue == MOEQ_EPI_SILU_MUL && out_dtype != MOEQ_BF16))
    return MOEQ_ERR_INVALID_ARG;
  if (a_topk > MOEQ_MAX_TOPK) return MOEQ_ERR_UNSUPPORTED;
  if (a_topk > 0 && R % a_topk != 0) return MOEQ_ERR_INVALID_ARG;
  if (R > 0x3FFFFFFF || moeq::mxfp4_gemm_grid(E, R, N) > kMaxGrid) return MOEQ_ERR_UNSUPPORTED;
  if (R == 0) return MOEQ_OK;
  if (!a_q || !a_s || !plan || !w || !ws || !out) return MOEQ_ERR_INVALID_ARG;
  if (!aligned16(a_q) || !aligned_to(a_s, 4) || !aligned16(w) || !aligned16(ws) || !aligned16(out))
    return MOEQ_ERR_INVALID_ARG;
  if (int rc = check_plan(plan, plan_bytes, E, R)) return rc;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_grouped_gemm_mxfp4(a_q, a_s, a_topk, plan, E, R, w, ws, N, K,
                                                       epilogue, out, out_dtype,
                                                       as_stream(stream)));
}

size_t moe_layer_mxfp4_few_ws_size(int T, int k, int H, int I) {
  if (check_few(T, k, H, I)) return 0;
  return moeq::few_ws_bytes(T, k, H, I);
}

int moe_layer_mxfp4_few(const float* logits, const float* bias, int T, int E, int k,
                        int renormalize, const uint16_t* x, int H, const uint8_t* w13,
                        const uint8_t* ws13, const uint8_t* w2, const uint8_t* ws2, int I,
                        const uint16_t* shared, int32_t* topk_ids, float* topk_w, uint16_t* y,
                        void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_few(T, k, H, I)) return rc;
  if (E <= 0 || k > E) return MOEQ_ERR_INVALID_ARG;
  if (E > MOEQ_MAX_EXPERTS) return MOEQ_ERR_UNSUPPORTED;
  if (T == 0) return MOEQ_OK;
  if (!logits || !x || !w13 || !ws13 || !w2 || !ws2 || !topk_ids || !topk_w || !y || !ws)
    return MOEQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w13) || !aligned16(ws13) || !aligned16(w2) || !aligned16(ws2) ||
      !aligned16(shared) || !aligned16(y) || !aligned_to(ws, 256) || !aligned_to(logits, 4) ||
      !aligned_to(bias, 4) || !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4))
    return MOEQ_ERR_INVALID_ARG;
  if (ws_bytes < moeq::few_ws_bytes(T, k, H, I)) return MOEQ_ERR_WORKSPACE;
  if (int rc = check_device()) return rc;
  return launch_status(moeq::launch_layer_mxfp4_few(logits, bias, T, E, k, renormalize, x, H, w13,
                                                    ws13, w2, ws2, I, shared, topk_ids, topk_w, y,
                                                    ws, as_stream(stream)));
}

}  // extern "C"
