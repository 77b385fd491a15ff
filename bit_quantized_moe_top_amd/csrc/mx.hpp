// MXFP4 on gfx950: E2M1 codes (two per byte, the low nibble first) with one
// E8M0 scale byte per block of 32 consecutive K.  Device building blocks shared
// by the MXFP4 kernels (mxquant.hip, mxgemm.hip, few.hip).
//
//   value(k) = e2m1(code[k]) * 2^(scale[k / 32] - 127)
//
// Tiled weights.  The matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes
// from lane (r = l % 16, kb = l / 16) 32 consecutive K of row r -- exactly one
// MXFP4 block -- with that block's scale in one byte of a register.  A sum over K
// may take the blocks in any order as long as both operands agree: over a
// super-group of 512 K (16 blocks) step j of four gives lane kb the block
// 4 kb + j.  The scales of a lane's four steps are then four consecutive bytes
// of the row, one dword load per 512 K, and step j reads byte j of it (op_sel).
// Weights are moved once into the order the kernels read (16-row blocks, then
// super-groups, then steps, then lanes):
//   codes  [E N / 16][G][4 steps][64 lanes][16 bytes]
//   scales [E N / 16][G][64 lanes][4 steps]              G = ceil(K / 512)
// so a wave's code load is 1024 contiguous bytes and its scale load 256.  Blocks
// past K are zero codes with scale 1.  Activations stay in rows.
//
// Operand order: weights first, activations second, so the lane (ln, kb) of a
// 16x16 result holds activation row ln and the four consecutive output columns
// 4 kb .. 4 kb + 3: a row leaves in 8-byte (bf16) or 16-byte (fp32) stores.
#pragma once

#include "gemm.hpp"
#include "mx_kernels.hpp"

namespace moeq {

constexpr int kMxBlock = 32;                  // K per scale
constexpr int kMxSuper = 512;                 // K per super-group
constexpr int kMxSteps = 4;                   // matrix steps (128 K each) per super-group
constexpr int kMxCodeBytes = 16 * kMxSuper / 2;       // codes of one 16-row block, one super-group
constexpr int kMxScaleBytes = 16 * kMxSuper / kMxBlock;
constexpr uint32_t kMxOne4 = 0x7F7F7F7Fu;     // four scales of 1

__host__ __device__ inline int mx_supers(int K) { return (K + kMxSuper - 1) / kMxSuper; }

namespace {

typedef int mx_v8i __attribute__((ext_vector_type(8)));
typedef float mx_v4f __attribute__((ext_vector_type(4)));
typedef unsigned mx_v4u __attribute__((ext_vector_type(4)));
typedef __bf16 mx_bf2 __attribute__((ext_vector_type(2)));
typedef float mx_f2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------ quantization
// The E8M0 byte of a block whose largest magnitude has the fp32 exponent field
// f: the power of two floor(log2 amax) - 2 (2 is E2M1's largest exponent), at
// least 2^-127.  f counts from 127, so the byte is f - 2; a zero or subnormal
// amax (f = 0) lies below 2^-126 and takes byte 0.  f = 255 (an infinity or a
// NaN in the block) gives 255, which marks the whole block as NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t f) {
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// the scale as an fp32 operand of the conversions, which read its exponent field
__device__ __forceinline__ float mx_scale_operand(uint32_t byte) { return u2f(byte << 23); }

// 8 E2M1 codes (element 0 in the lowest nibble) of v / scale, rounded to
// nearest even, saturating at 6, sign kept.  A block marked NaN has codes 0.
// (The conversions were checked on the device against the definition, ties,
// subnormals and every scale byte included.)
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float s) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
  return r;
}
__device__ __forceinline__ uint32_t mx_codes8(const uint4& u, float s) {      // 8 bf16
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, u.x), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, u.y), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, u.z), s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, u.w), s, 3);
  return r;
}

// 8 codes times the scale, exact
__device__ __forceinline__ uint4 mx_bf16x8(uint32_t c, float s) {
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3)));
}

// ------------------------------------------------------------------ product
// c + W A over 128 K: w a lane's 32 weight codes, a its 32 activation codes, the
// scales byte J of sw and sa (the hardware's FP4 sums were measured within 1e-7
// of the sum of magnitudes, i.e. fp32 rounding; a scale of 255 gives NaN).
template <int J>
__device__ __forceinline__ mx_v4f mx_mfma(const uint4& w, uint32_t sw, const uint4& a, uint32_t sa,
                                          const mx_v4f& c) {
  const mx_v8i wv = {int(w.x), int(w.y), int(w.z), int(w.w), 0, 0, 0, 0};
  const mx_v8i av = {int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, c, 4, 4, J, int(sw), J, int(sa));
}

// -------------------------------------------------------------- weight loads
// 16 bytes at base + off + lane with cache policy CP (load_weight16), and the
// scale dword beside it
template <int CP>
__device__ __forceinline__ uint32_t load_scale4(const uint8_t* base, int off, uint32_t lane) {
  const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(base), static_cast<short>(0), 0x7FFFFFFF, 0x00020000);
  return __builtin_amdgcn_raw_buffer_load_b32(res, int(lane), off, CP);
}

// one super-group of one operand's 16 rows, as a lane holds it: the codes of its
// four steps and their four scale bytes
struct MxFrag {
  uint4 c[kMxSteps];
  uint32_t s;
};

template <int CP>
__device__ __forceinline__ MxFrag load_weights(const uint8_t* w, const uint8_t* ws, int sg,
                                               int lane) {
  MxFrag f;
#pragma unroll
  for (int j = 0; j < kMxSteps; ++j)
    f.c[j] = load_weight16<CP>(w, (sg * kMxSteps + j) * 1024, uint32_t(lane * 16));
  f.s = load_scale4<CP>(ws, sg * kMxScaleBytes, uint32_t(lane * 4));
  return f;
}

// two fp32 values as bf16 (nearest even; infinities and NaNs kept)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, mx_bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// four consecutive output columns of one row: bf16 (rounded to nearest even) or fp32
__device__ __forceinline__ void store4(void* out, int out_f32, int64_t at, const mx_v4f& v) {
  if (out_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

__device__ __forceinline__ mx_v4f silu_mul4(const mx_v4f& g, const mx_v4f& u) {
  mx_v4f r;
#pragma unroll
  for (int v = 0; v < 4; ++v) r[v] = silu_f32(g[v]) * u[v];
  return r;
}

// Calls fn(integral_constant<int, 0>) ... fn(integral_constant<int, N - 1>).
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& fn) {
  if constexpr (I < N) {
    fn(std::integral_constant<int, I>());
    static_for<N, I + 1>(static_cast<F&&>(fn));
  }
}

}  // namespace

}  // namespace moeq
