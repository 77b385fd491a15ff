/*
 * moeq_lora.h -- the shared experts' projection with low-rank adapters: every
 * row of a batch passes through one shared bf16 weight, and through the adapter
 * of its own request beside it (gfx950).
 *
 * The conventions of moeq.h hold: device pointers, caller-owned buffers,
 * asynchronous work on `stream`, no allocation, no synchronization, the same
 * status codes, arguments checked before any HIP call, deterministic results.
 */
#ifndef MOEQ_LORA_H
#define MOEQ_LORA_H

#include "moeq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest rank of an adapter, and most adapters of a batch. */
#define MOEQ_LORA_MAX_RANK 256
#define MOEQ_MAX_ADAPTERS  (MOEQ_MAX_EXPERTS - 1)

/*
 * moe_adapter_plan -- the rows of a batch grouped by adapter, once per batch; every
 * projection of every layer reads it.  The plan is the one moe_permute would build
 * for k = 1 and L + 1 experts (the layout of moe_plan_size(L + 1, M)), where rows
 * whose id is outside [0, L) form the last group: they have no adapter.
 *
 *   ids [M] int32       plan (out), plan_bytes >= moe_plan_size(L + 1, M)
 * Limits: M >= 0, 1 <= L <= MOEQ_MAX_ADAPTERS, M < 2^24.
 * MOEQ_ERR_WORKSPACE: plan_bytes too small.
 */
int moe_adapter_plan(const int32_t* ids, int M, int L, void* plan, size_t plan_bytes,
                     void* stream);

/* Bytes of the workspace of moe_shared_gemm_lora_bf16 (0 for sizes it refuses). */
size_t moe_shared_gemm_lora_ws_size(int M, int N, int K, int L, int slices, int r);

/*
 * moe_shared_gemm_lora_bf16 -- the shared experts' projection (moe_shared_gemm_bf16)
 * with each row's low-rank adapter.  For row m of adapter l = ids[m], and slice
 * s = n / (N / slices) of output column n:
 *   u[m, s, j] = scale[l] * sum_k a[m, k] * lora_a[l, s, j, k]
 *   v[m, n]    = sum_k a[m, k] * w[n, k] + sum_j u[m, s, j] * lora_b[l, n, j]
 * rows without an adapter: the first sum only.  Epilogues as moe_shared_gemm_bf16:
 *   NONE: out[m, n] = bf16(v[m, n])                               ([M, N])
 *   SILU_MUL: out[m, i] = bf16(silu(v[m, i]) * v[m, N/2 + i])     ([M, N/2])
 * Sums are in fp32; u is carried in two bf16 parts (16 significant bits); out is rounded
 * once.  What an adapter holds reaches the rows of that adapter only.  Two slices are for
 * gate/up weights whose halves have an adapter input (lora_a) each.
 *
 *   a [M, K] bf16, row stride ld_a elements     w [N, K] bf16
 *   lora_a [L, slices, r, K] bf16   lora_b [L, N, r] bf16   scale [L] fp32
 *   plan, plan_bytes -- from moe_adapter_plan with the same M and L (read only)
 *   out [M, N] or [M, N/2] bf16 (out), contiguous
 *   ws -- workspace, contents irrelevant before the call and undefined after it;
 *     calls that may overlap (other streams, concurrently replayed graphs) need
 *     workspaces of their own
 * Limits: 0 <= M < 2^24, K % 8 == 0, K < 2^20, N % 16 == 0 (N % 32 with SILU_MUL or two
 * slices), N <= 2^20, slices 1 or 2, r % 8 == 0, 8 <= r <= MOEQ_LORA_MAX_RANK, 1 <= L <=
 * MOEQ_MAX_ADAPTERS, ld_a >= K, ld_a % 8 == 0, fewer than 2^24 workgroups (M / 64 * N / 64);
 * a, w, lora_a, lora_b, out 16-byte, ws 256-byte aligned; outputs do not overlap inputs.
 * MOEQ_ERR_WORKSPACE: plan_bytes or ws_bytes too small.
 */
int moe_shared_gemm_lora_bf16(const uint16_t* a, int64_t ld_a, const uint16_t* w, int M, int N,
                              int K, const uint16_t* lora_a, const uint16_t* lora_b,
                              const float* scale, int L, int slices, int r, const void* plan,
                              size_t plan_bytes, int epilogue, uint16_t* out, void* ws,
                              size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_LORA_H */
