// MXFP4 quantization of rows, its inverse, and the move of weights into the
// kernels' tiled order (formats in mx.hpp).  All three are streams bound by HBM.
#include "mx.hpp"

namespace moeq {

namespace {

constexpr int kQuantUnroll = 2;       // 16-element chunks per thread
constexpr int kDequantUnroll = 4;     // 8-element chunks per thread

// 16 consecutive elements as loaded
struct Chunk16 {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    lo = q[0];
    hi = q[1];
  }
  // exponent field of the largest magnitude
  __device__ __forceinline__ uint32_t amax_field() const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max((w[i] << 16) & 0x7F800000u, w[i] & 0x7F800000u));
    return m >> 23;
  }
  __device__ __forceinline__ uint2 codes(float s) const {
    return make_uint2(mx_codes8(lo, s), mx_codes8(hi, s));
  }
};
struct Chunk16f {
  float v[2][8];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = reinterpret_cast<const float4*>(p)[2 * h + i];
        v[h][4 * i] = f.x; v[h][4 * i + 1] = f.y; v[h][4 * i + 2] = f.z; v[h][4 * i + 3] = f.w;
      }
  }
  __device__ __forceinline__ uint32_t amax_field() const {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, f2u(v[h][i]) & 0x7F800000u);
    return m >> 23;
  }
  __device__ __forceinline__ uint2 codes(float s) const {
    return make_uint2(mx_codes8(v[0], s), mx_codes8(v[1], s));
  }
};
template <typename XT>
struct ChunkOf { using type = Chunk16; };
template <>
struct ChunkOf<float> { using type = Chunk16f; };

// A thread takes 16 elements, half a block: the pair of lanes (l, l ^ 1) of a
// block exchanges exponent fields with one DPP move.  Only the field of the
// largest magnitude matters for the scale, so no floating-point maximum is
// formed.  Chunk i of the matrix is chunk i of its only "row" when the rows are
// contiguous (the launcher then passes one row); strided rows take one division
// per chunk.
template <typename XT, bool kOneRow>
__global__ void __launch_bounds__(kThreads)
quant_mxfp4_kernel(const XT* __restrict__ x, int64_t chunks, int64_t per_row, int64_t ld,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  using Chunk = typename ChunkOf<XT>::type;
  const int64_t c0 = int64_t(blockIdx.x) * (kThreads * kQuantUnroll) + threadIdx.x;
  Chunk ch[kQuantUnroll];
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c < chunks) {
      if constexpr (kOneRow) {
        ch[u].load(x + c * 16);
      } else {
        const int64_t row = c / per_row;
        ch[u].load(x + row * ld + (c - row * per_row) * 16);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c < chunks) {              // chunks come in pairs: both lanes of a block are here
      const uint32_t f = ch[u].amax_field();
      const uint32_t other = uint32_t(dpp<kDppQuadSwap1>(int(f), int(f)));
      const uint32_t byte = mx_scale_byte(max(f, other));
      const uint2 codes = ch[u].codes(mx_scale_operand(byte));
      const bool nan = byte == 255u;
      reinterpret_cast<uint2*>(q)[c] = nan ? make_uint2(0u, 0u) : codes;
      if ((c & 1) == 0) scale[c >> 1] = uint8_t(byte);
    }
  }
}

// A thread takes 8 codes (4 bytes), a quarter of a block.
template <typename OT>
__global__ void __launch_bounds__(kThreads)
dequant_mxfp4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                     int64_t chunks, OT* __restrict__ out) {
  const int64_t c0 = int64_t(blockIdx.x) * (kThreads * kDequantUnroll) + threadIdx.x;
  uint32_t w[kDequantUnroll], s[kDequantUnroll];
#pragma unroll
  for (int u = 0; u < kDequantUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c < chunks) {
      w[u] = reinterpret_cast<const uint32_t*>(q)[c];
      s[u] = scale[c >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kDequantUnroll; ++u) {
    const int64_t c = c0 + u * kThreads;
    if (c >= chunks) continue;
    const float sf = mx_scale_operand(s[u]);
    if constexpr (sizeof(OT) == 2) {
      reinterpret_cast<uint4*>(out)[c] = mx_bf16x8(w[u], sf);
    } else {
      const mx_f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 0);
      const mx_f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 1);
      const mx_f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 2);
      const mx_f2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], sf, 3);
      reinterpret_cast<float4*>(out)[2 * c] = make_float4(a[0], a[1], b[0], b[1]);
      reinterpret_cast<float4*>(out)[2 * c + 1] = make_float4(d[0], d[1], e[0], e[1]);
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
  const int64_t chunks = M * (K / 16);
  const bool one_row = ld_x == K || M == 1;
  const dim3 grid(unsigned((chunks + kThreads * kQuantUnroll - 1) / (kThreads * kQuantUnroll)));
  auto go = [&](auto* xp) {
    using XT = std::remove_const_t<std::remove_pointer_t<decltype(xp)>>;
    if (one_row)
      hipLaunchKernelGGL((quant_mxfp4_kernel<XT, true>), grid, dim3(kThreads), 0, stream, xp,
                         chunks, chunks, ld_x, q, scale);
    else
      hipLaunchKernelGGL((quant_mxfp4_kernel<XT, false>), grid, dim3(kThreads), 0, stream, xp,
                         chunks, int64_t(K / 16), ld_x, q, scale);
  };
  if (x_dtype == MOEQ_BF16) go(static_cast<const uint16_t*>(x));
  else go(static_cast<const float*>(x));
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t M, int K,
                                void* out, int out_dtype, hipStream_t stream) {
  const int64_t chunks = M * (K / 8);
  const dim3 grid(unsigned((chunks + kThreads * kDequantUnroll - 1) / (kThreads * kDequantUnroll)));
  if (out_dtype == MOEQ_BF16)
    hipLaunchKernelGGL(dequant_mxfp4_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, q, scale,
                       chunks, static_cast<uint16_t*>(out));
  else
    hipLaunchKernelGGL(dequant_mxfp4_kernel<float>, grid, dim3(kThreads), 0, stream, q, scale,
                       chunks, static_cast<float*>(out));
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
