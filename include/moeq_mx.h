/*
 * moeq_mx.h -- the MXFP4 part of libmoeq's C ABI: microscaled 4-bit floating
 * point experts for the layer of moeq.h (gfx950).
 *
 * Format (OCP Microscaling Formats specification 1.0, MXFP4): E2M1 codes, two
 * per byte, the low nibble first; one E8M0 scale byte per block of 32
 * consecutive elements of a row:
 *   value(k) = e2m1(code[k]) * 2^(scale[k / 32] - 127)
 *   e2m1: bit 3 the sign, bits 0..2 one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * A scale byte of 255 marks a block of NaNs.
 *
 * The conventions of moeq.h hold: device pointers, caller-owned buffers,
 * asynchronous work on `stream`, no allocation, no synchronization, the same
 * status codes, arguments checked before any HIP call, deterministic results.
 */
#ifndef MOEQ_MX_H
#define MOEQ_MX_H

#include "moeq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest K (H, I) of the MXFP4 products. */
#define MOEQ_MX_MAX_K (1 << 20)
/* Most tokens of moe_layer_mxfp4_few. */
#define MOEQ_FEW_TOKENS 16

/*
 * quant_mxfp4 -- rows to MXFP4.  For each block of 32 consecutive elements:
 *   a = max |x|;  s = max(floor(log2 a) - 2, -127)   (a = 0: -127)
 *   scale = s + 127;  code = E2M1_RNE_saturating(x * 2^-s), the sign kept
 * (floor(log2 a) - 2: the specification's rule, 2 being E2M1's largest
 * exponent; values in (6, 8) * 2^s saturate to 6).  Exact: every output byte is
 * determined by the formula.  A block that holds an infinity or a NaN gets
 * scale 255 and codes 0.
 *
 *   x [M, K] fp32 or bf16 (x_dtype), row stride ld_x elements
 *   q [M, K/2] (out)     scale [M, K/32] (out), both contiguous
 * Limits: M >= 0, K % 32 == 0, ld_x >= K, ld_x % 8 == 0, M * K <= 2^35;
 * x and q 16-byte aligned; outputs do not overlap x.
 */
int quant_mxfp4(const void* x, int x_dtype, int64_t M, int K, int64_t ld_x, uint8_t* q,
                uint8_t* scale, void* stream);

/*
 * dequant_mxfp4 -- the values that MXFP4 rows stand for, exact in fp32 and in
 * bf16 (2 significant bits) for scale bytes up to 252, which is all that
 * quant_mxfp4 writes; 253 and 254 may overflow to infinity, 255 gives NaN.
 *
 *   q [M, K/2], scale [M, K/32]   out [M, K] fp32 or bf16 (out_dtype)
 * Limits: M >= 0, K % 32 == 0, M * K <= 2^35; q 4-byte, out 16-byte aligned.
 */
int dequant_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t M, int K, void* out,
                  int out_dtype, void* stream);

/*
 * moe_tile_mxfp4_weights -- MXFP4 weight rows into the tiled order that the
 * products read (offline weight preparation, once per tensor).  With
 * G = ceil(K / 512), block b < rows / 16, super-group g < G, step j < 4 and lane
 * l < 64 (row r = 16 b + l % 16, block of the row c = 16 g + 4 (l / 16) + j):
 *   w [((b G + g) 4 + j) 64 + l]  (16 bytes) = the codes of block c of row r
 *   ws[((b G + g) 64 + l) 4 + j]  (1 byte)   = its scale
 * Blocks past K are codes 0 with scale 127 (the value 0).  A stack [E, N, K] is
 * tiled in one call with rows = E N.
 *
 *   q [rows, K/2], scale [rows, K/32]
 *   w [rows/16 * G * 4096] bytes (out)   ws [rows/16 * G * 256] bytes (out)
 * Limits: rows % 16 == 0, K % 32 == 0, K <= MOEQ_MX_MAX_K, rows/16 * G < 2^24;
 * all but scale 16-byte aligned; outputs do not overlap inputs.
 */
int moe_tile_mxfp4_weights(const uint8_t* q, const uint8_t* scale, int64_t rows, int K, uint8_t* w,
                           uint8_t* ws, void* stream);

/*
 * moe_grouped_gemm_mxfp4 -- grouped GEMM over the routed experts with MXFP4
 * activations and MXFP4 weights.  For sorted row p of expert e (per the plan):
 *   v[p, n] = sum_k A[row(p), k] * W[e, n, k]     (fp32 sums)
 * and the epilogues of moe_grouped_gemm_w4a8:
 *   NONE: out[p, n] = v[p, n]  ([R, N], out_dtype bf16 or fp32)
 *   SILU_MUL: out[p, i] = bf16(silu(v[p, i]) * v[p, N/2 + i])  ([R, N/2], bf16)
 * Rows of experts that the permutation dropped are not written.
 *
 *   a_q, a_s -- MXFP4 rows of K elements.  a_topk = 0: [R] rows in plan order,
 *     row(p) = p.  a_topk = k > 0: [R / k] rows in token order, row(p) =
 *     sorted_rows[p] / k (the k rows of a token read its one row; no gathered
 *     copy is needed)
 *   plan, plan_bytes -- from moe_permute with the same E and R (read only)
 *   w, ws -- [E, N, K] weights in the order of moe_tile_mxfp4_weights
 * Limits: N % 32 == 0, K % 32 == 0, K <= MOEQ_MX_MAX_K, 1 <= E <=
 * MOEQ_MAX_EXPERTS, 0 <= a_topk <= MOEQ_MAX_TOPK, R % a_topk == 0, fewer than 2^24
 * workgroups (with T = ceil(R / 64) + min(E, R) row tiles: T * N / 32 of them at
 * most); a_q, w, ws and out 16-byte, a_s 4-byte aligned.
 */
int moe_grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, int a_topk, const void* plan,
                           size_t plan_bytes, int E, int R, const uint8_t* w, const uint8_t* ws,
                           int N, int K, int epilogue, void* out, int out_dtype, void* stream);

/* Bytes of the workspace of moe_layer_mxfp4_few (0 for sizes it refuses). */
size_t moe_layer_mxfp4_few_ws_size(int T, int k, int H, int I);

/*
 * moe_layer_mxfp4_few -- a whole expert layer for T <= MOEQ_FEW_TOKENS tokens in
 * two kernels, with MXFP4 weights and bf16 activations:
 *   topk_ids, topk_w    as moe_route_topk (logits, bias, k, renormalize)
 *   h_j = silu(Wg_e x_t) * (Wu_e x_t),  e = topk_ids[t, j]   (fp32; bits below 2^-133 are
 *         cut off)
 *   y_t = bf16( sum_j topk_w[t, j] * (W2_e h_j) + shared_t )  (fp32 sums in slot order)
 * Nothing is quantized but the weights; y is rounded once.  Scores of -inf mark masked experts and
 * get weight 0; a token whose k best scores are all -inf gets weights 0 (y_t =
 * shared_t, or 0).  An expert of weight 0 adds nothing, whatever its weights hold.
 * Other scores are finite (with a NaN score the ids stay inside [0, E) and the
 * token's outputs mean nothing).
 *
 *   logits [T, E] fp32, bias [E] fp32 or NULL, x [T, H] bf16
 *   w13, ws13 -- [E, 2I, H] (gate rows, then up rows), w2, ws2 -- [E, H, I], both in
 *     the order of moe_tile_mxfp4_weights, scale bytes at most 252
 *   shared [T, H] bf16 or NULL
 *   topk_ids [T, k] int32 (out), topk_w [T, k] fp32 (out), y [T, H] bf16 (out)
 *   ws -- workspace, contents irrelevant before the call and undefined after it;
 *     calls that may overlap (other streams, concurrently replayed graphs) need
 *     workspaces of their own
 * Limits: 0 <= T <= MOEQ_FEW_TOKENS, H % 32 == 0, I % 32 == 0, H and I <=
 * MOEQ_MX_MAX_K, 1 <= E <= MOEQ_MAX_EXPERTS, 1 <= k <= min(E, MOEQ_MAX_TOPK);
 * ws 256-byte, x, the weights, shared and y 16-byte aligned.
 * MOEQ_ERR_WORKSPACE: ws_bytes < moe_layer_mxfp4_few_ws_size(T, k, H, I).
 */
int moe_layer_mxfp4_few(const float* logits, const float* bias, int T, int E, int k,
                        int renormalize, const uint16_t* x, int H, const uint8_t* w13,
                        const uint8_t* ws13, const uint8_t* w2, const uint8_t* ws2, int I,
                        const uint16_t* shared, int32_t* topk_ids, float* topk_w, uint16_t* y,
                        void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_MX_H */
