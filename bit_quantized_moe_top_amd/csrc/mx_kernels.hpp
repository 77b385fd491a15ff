// Launchers of the MXFP4 kernels (arguments validated by api_mx.hip; each returns
// hipGetLastError()).
#pragma once

#include "kernels.hpp"

namespace moeq {

// E2M1 codes (two per byte) with an E8M0 scale byte per 32 K (mx.hpp)
hipError_t launch_quant_mxfp4(const void* x, int x_dtype, int64_t M, int K, int64_t ld_x,
                              uint8_t* q, uint8_t* scale, hipStream_t stream);
hipError_t launch_dequant_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t M, int K,
                                void* out, int out_dtype, hipStream_t stream);
// weight rows into the tiled order (rows % 16 == 0, K % 32 == 0, no overlap)
hipError_t launch_tile_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t rows, int K,
                             uint8_t* w, uint8_t* ws, hipStream_t stream);
// MXFP4 activations (a_topk = 0: rows in plan order; else row r reads row
// r / a_topk) against tiled MXFP4 weights
hipError_t launch_grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, int a_topk,
                                     const void* plan, int E, int R, const uint8_t* w,
                                     const uint8_t* ws, int N, int K, int epilogue, void* out,
                                     int out_dtype, hipStream_t stream);

// its workgroups
int64_t mxfp4_gemm_grid(int E, int R, int N);

// a whole layer for at most kFewTokens tokens (few.hip)
constexpr int kFewTokens = 16;
size_t few_ws_bytes(int T, int k, int H, int I);
hipError_t launch_layer_mxfp4_few(const float* logits, const float* bias, int T, int E, int k,
                                  int renormalize, const uint16_t* x, int H, const uint8_t* w13,
                                  const uint8_t* ws13, const uint8_t* w2, const uint8_t* ws2, int I,
                                  const uint16_t* shared, int32_t* ids, float* topk_w, uint16_t* y,
                                  void* ws, hipStream_t stream);

}  // namespace moeq
