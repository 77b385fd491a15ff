// MXFP4 quantization of rows, its inverse, and the move of weights into the
// kernels' tiled order (formats in mx.hpp).  All three are streams bound by HBM.
#include "mx.hpp"

namespace moeq {

namespace {

constexpr int kUnroll = 4;            // 16-byte pieces per thread

// A lane takes 16-byte pieces of x: 8 bf16 elements (4 lanes per block) or 4 fp32
// elements (8 lanes).
template <typename XT>
struct Piece;
template <>
struct Piece<uint16_t> {
  static constexpr int kLanes = 4;
  using Codes = uint32_t;
  // the exponent field of the largest magnitude
  static __device__ __forceinline__ uint32_t amax_field(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7F800000u, w[i] & 0x7F800000u));
    return m >> 23;
  }
  static __device__ __forceinline__ Codes codes(const uint4& v, float s) { return mx_codes8(v, s); }
};
template <>
struct Piece<float> {
  static constexpr int kLanes = 8;
  using Codes = uint16_t;
  static __device__ __forceinline__ uint32_t amax_field(const uint4& v) {
    return (max(max(v.x & 0x7F800000u, v.y & 0x7F800000u),
                max(v.z & 0x7F800000u, v.w & 0x7F800000u))) >> 23;
  }
  static __device__ __forceinline__ Codes codes(const uint4& v, float s) {
    uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, u2f(v.x), u2f(v.y), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, u2f(v.z), u2f(v.w), s, 1);
    return Codes(r);
  }
};

// Consecutive lanes take consecutive pieces, so loads and stores are contiguous;
// the lanes of a block combine the exponent fields of their largest magnitudes with
// DPP moves (only the field matters for the scale, so no floating-point maximum is
// formed).  Piece i of the matrix is piece i of its only "row" when the rows are
// contiguous (the launcher then passes one row); strided rows take one division
// per piece.  x is read once, past the caches' replacement order: 12288 x 2048
// bf16 in 12.0 us (64 MB moved, 5.3 TB/s) against 15.9 us with default loads; turning
// the codes in LDS into 16-byte stores gains nothing on that (12.0 us).
template <typename XT, bool kOneRow>
__global__ void __launch_bounds__(kThreads)
quant_mxfp4_kernel(const XT* __restrict__ x, int64_t pieces, int64_t per_row, int64_t ld,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  using P = Piece<XT>;
  constexpr int kElems = 16 / sizeof(XT);
  const int64_t c0 = int64_t(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (c < pieces) {
      const XT* at = x + c * kElems;
      if constexpr (!kOneRow) {
        const int64_t row = c / per_row;
        at = x + row * ld + (c - row * per_row) * kElems;
      }
      const mx_v4u t = __builtin_nontemporal_load(reinterpret_cast<const mx_v4u*>(at));
      v[u] = make_uint4(t[0], t[1], t[2], t[3]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    uint32_t f = P::amax_field(v[u]);          // (a block's pieces are all inside, or all past the end)
    f = max(f, uint32_t(dpp<kDppQuadSwap1>(int(f), int(f))));
    f = max(f, uint32_t(dpp<kDppQuadSwap2>(int(f), int(f))));
    if (P::kLanes == 8) f = max(f, uint32_t(dpp<kDppRowHalfMirror>(int(f), int(f))));
    const uint32_t byte = mx_scale_byte(f);
    const typename P::Codes codes = P::codes(v[u], mx_scale_operand(byte));
    if (c < pieces) {
      reinterpret_cast<typename P::Codes*>(q)[c] = byte == 255u ? typename P::Codes(0) : codes;
      if (c % P::kLanes == 0) scale[c / P::kLanes] = uint8_t(byte);
    }
  }
}

// The inverse: a thread forms 16-byte pieces of the output, 8 bf16 values from 4
// bytes of codes or 4 fp32 values from 2.
template <typename OT>
__global__ void __launch_bounds__(kThreads)
dequant_mxfp4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                     int64_t pieces, OT* __restrict__ out) {
  using P = Piece<OT>;
  const int64_t c0 = int64_t(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint32_t w[kUnroll], s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c < pieces) {
      w[u] = reinterpret_cast<const typename P::Codes*>(q)[c];
      s[u] = scale[c / P::kLanes];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c >= pieces) continue;
    const float sf = mx_scale_operand(s[u]);
    if constexpr (sizeof(OT) == 2) {
      reinterpret_cast<uint4*>(out)[c] = mx_bf16x8(w[u], sf);
    } else {
      const mx_f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 0);
      const mx_f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 1);
      reinterpret_cast<float4*>(out)[c] = make_float4(a[0], a[1], b[0], b[1]);
    }
  }
}

// One workgroup per (16-row block, super-group): 4 KB of codes, 256 B of scales.
__global__ void __launch_bounds__(kThreads)
tile_mxfp4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale, int K, int G,
                  uint8_t* __restrict__ w, uint8_t* __restrict__ ws) {
  const int64_t unit = blockIdx.x;
  const int64_t blk = unit / G;
  const int sg = int(unit - blk * G);
  const int KB = K / kMxBlock;
  const int t = threadIdx.x, j = t >> 6, lane = t & 63, r = lane & 15, kb = lane >> 4;
  const int64_t row = 16 * blk + r;
  const int b = 16 * sg + 4 * kb + j;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (b < KB) v = *reinterpret_cast<const uint4*>(q + row * (K >> 1) + b * 16);
  reinterpret_cast<uint4*>(w)[unit * kThreads + t] = v;
  if (t < 64) {
    uint32_t s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bi = 16 * sg + 4 * kb + i;
      s |= uint32_t(bi < KB ? scale[row * KB + bi] : 127) << (8 * i);
    }
    reinterpret_cast<uint32_t*>(ws)[unit * 64 + t] = s;
  }
}

}  // namespace

hipError_t launch_quant_mxfp4(const void* x, int x_dtype, int64_t M, int K, int64_t ld_x,
                              uint8_t* q, uint8_t* scale, hipStream_t stream) {
  auto go = [&](auto* xp) {
    using XT = std::remove_const_t<std::remove_pointer_t<decltype(xp)>>;
    const int64_t per_row = K / (16 / int(sizeof(XT))), pieces = M * per_row;
    const dim3 grid(unsigned((pieces + kThreads * kUnroll - 1) / (kThreads * kUnroll)));
    if (ld_x == K || M == 1)
      hipLaunchKernelGGL((quant_mxfp4_kernel<XT, true>), grid, dim3(kThreads), 0, stream, xp,
                         pieces, per_row, ld_x, q, scale);
    else
      hipLaunchKernelGGL((quant_mxfp4_kernel<XT, false>), grid, dim3(kThreads), 0, stream, xp,
                         pieces, per_row, ld_x, q, scale);
  };
  if (x_dtype == MOEQ_BF16) go(static_cast<const uint16_t*>(x));
  else go(static_cast<const float*>(x));
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t M, int K,
                                void* out, int out_dtype, hipStream_t stream) {
  auto go = [&](auto* op) {
    using OT = std::remove_pointer_t<decltype(op)>;
    const int64_t pieces = M * (K / (16 / int(sizeof(OT))));
    const dim3 grid(unsigned((pieces + kThreads * kUnroll - 1) / (kThreads * kUnroll)));
    hipLaunchKernelGGL(dequant_mxfp4_kernel<OT>, grid, dim3(kThreads), 0, stream, q, scale, pieces,
                       op);
  };
  if (out_dtype == MOEQ_BF16) go(static_cast<uint16_t*>(out));
  else go(static_cast<float*>(out));
  return hipGetLastError();
}

hipError_t launch_tile_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t rows, int K,
                             uint8_t* w, uint8_t* ws, hipStream_t stream) {
  const int G = mx_supers(K);
  hipLaunchKernelGGL(tile_mxfp4_kernel, dim3(unsigned(rows / 16 * G)), dim3(kThreads), 0, stream, q,
                     scale, K, G, w, ws);
  return hipGetLastError();
}

}  // namespace moeq
