// Grouped GEMM over the routed experts with MXFP4 activations and MXFP4 weights
// (formats, tiled weight order and matrix step in mx.hpp):
//   out[p, n] = epilogue( sum_k A[row(p), k] W[e(p), n, k] ),  fp32 sums
// row(p) = p (activations in plan order) or sorted_rows[p] / topk (activations in
// token order, read in place: no gathered copy of the k rows per token).
//
// K-split kernel: one workgroup per unit (plan tile of <= 64 rows, two 16-row
// weight blocks -- 32 output columns, or 16 gate rows with their 16 up rows);
// wave q sweeps the super-groups of K quarter q, the four partial sums meet in
// LDS in the fixed order s0 + (s1 + (s2 + s3)).
#include "mx.hpp"

namespace moeq {

namespace {

// The activation row of one lane: codes and scales of K / 32 blocks.
struct MxRow {
  const uint8_t* codes;
  const uint8_t* scales;
  bool live;            // a row of the tile (others contribute zeros)
};

// super-group sg of a lane's activation row; blocks past K, and rows past the
// tile, are zeros
__device__ __forceinline__ MxFrag load_act(const MxRow& row, int sg, int kb, int KB) {
  MxFrag f;
  const int b0 = 16 * sg + 4 * kb;
#pragma unroll
  for (int j = 0; j < kMxSteps; ++j) {
    f.c[j] = make_uint4(0u, 0u, 0u, 0u);
    if (row.live && b0 + j < KB) f.c[j] = *reinterpret_cast<const uint4*>(row.codes + (b0 + j) * 16);
  }
  f.s = kMxOne4;
  if (row.live) {
    if ((KB & 3) == 0) {                    // rows of whole dwords
      if (b0 < KB) f.s = *reinterpret_cast<const uint32_t*>(row.scales + b0);
    } else {
      uint32_t s = 0;
#pragma unroll
      for (int j = 0; j < kMxSteps; ++j)
        s |= uint32_t(b0 + j < KB ? row.scales[b0 + j] : 127) << (8 * j);
      f.s = s;
    }
  }
  return f;
}

template <int EPI>
__global__ void __launch_bounds__(kThreads)
gemm_mx_wave_kernel(const uint8_t* a_q, const uint8_t* a_s, int a_topk, const int32_t* plan, int E,
                    int R, const uint8_t* w, const uint8_t* ws, int N, int K, void* out,
                    int out_f32) {
  __shared__ mx_v4f red[4][4][2][kWave];        // [wave][row block][weight block]
  const int lane = threadIdx.x & 63, q = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, kb = lane >> 4;
  const int units = N / 32;
  const int tile = blockIdx.x / units;
  const int u = blockIdx.x - tile * units;
  TileInfo ti;
  if (!tile_info(plan, E, R, tile, ti)) return;         // workgroup-uniform
  const int nrb = (ti.rows + 15) >> 4;
  const int KB = K / kMxBlock, G = mx_supers(K);

  // weight blocks (16 rows each) of the unit
  const int64_t nb = N / 16;
  const int b0 = EPI == MOEQ_EPI_SILU_MUL ? u : 2 * u;
  const int b1 = EPI == MOEQ_EPI_SILU_MUL ? u + N / 32 : 2 * u + 1;
  const uint8_t* w0 = w + (ti.e * nb + b0) * G * int64_t(kMxCodeBytes);
  const uint8_t* w1 = w + (ti.e * nb + b1) * G * int64_t(kMxCodeBytes);
  const uint8_t* s0 = ws + (ti.e * nb + b0) * G * int64_t(kMxScaleBytes);
  const uint8_t* s1 = ws + (ti.e * nb + b1) * G * int64_t(kMxScaleBytes);

  MxRow row[4];
  const PlanView pv = plan_view(const_cast<int32_t*>(plan), E, R);
#pragma unroll
  for (int rb = 0; rb < 4; ++rb) {
    row[rb].live = 16 * rb + ln < ti.rows;
    int64_t r = ti.row0 + (row[rb].live ? 16 * rb + ln : 0);
    if (a_topk && row[rb].live) r = min(max(pv.sorted_rows[r], 0), R - 1) / a_topk;
    row[rb].codes = a_q + r * (K >> 1);
    row[rb].scales = a_s + r * KB;
  }

  mx_v4f acc[4][2];
#pragma unroll
  for (int rb = 0; rb < 4; ++rb)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[rb][j] = mx_v4f{0.f, 0.f, 0.f, 0.f};
  const int g0 = quarter_g0(G, q), gn = g0 + quarter_groups(G, q);
  for (int sg = g0; sg < gn; ++sg) {
    const MxFrag f0 = load_weights<kCpStream>(w0, s0, sg, lane);
    const MxFrag f1 = load_weights<kCpStream>(w1, s1, sg, lane);
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      if (rb < nrb) {
        const MxFrag a = load_act(row[rb], sg, kb, KB);
        static_for<kMxSteps>([&](auto j) {
          acc[rb][0] = mx_mfma<j>(f0.c[j], f0.s, a.c[j], a.s, acc[rb][0]);
          acc[rb][1] = mx_mfma<j>(f1.c[j], f1.s, a.c[j], a.s, acc[rb][1]);
        });
      }
    }
  }
#pragma unroll
  for (int rb = 0; rb < 4; ++rb)
    if (rb < nrb) {
      red[q][rb][0][lane] = acc[rb][0];
      red[q][rb][1][lane] = acc[rb][1];
    }
  __syncthreads();
  // wave q finishes row block q
  if (q >= nrb) return;
  mx_v4f v[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    v[j] = red[0][q][j][lane] + (red[1][q][j][lane] + (red[2][q][j][lane] + red[3][q][j][lane]));
  const int r_in = 16 * q + ln;
  if (r_in >= ti.rows) return;
  const int64_t p = ti.row0 + r_in;
  if constexpr (EPI == MOEQ_EPI_SILU_MUL) {
    store4(out, 0, p * (N >> 1) + 16 * u + 4 * kb, silu_mul4(v[0], v[1]));
  } else {
    store4(out, out_f32, p * N + 32 * u + 4 * kb, v[0]);
    store4(out, out_f32, p * N + 32 * u + 16 + 4 * kb, v[1]);
  }
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, int a_topk,
                                     const void* plan, int E, int R, const uint8_t* w,
                                     const uint8_t* ws, int N, int K, int epilogue, void* out,
                                     int out_dtype, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const int out_f32 = out_dtype == MOEQ_F32 ? 1 : 0;
  const int32_t* p = static_cast<const int32_t*>(plan);
  const dim3 grid(unsigned(int64_t(plan_max_tiles(E, R)) * (N / 32)));
  if (epilogue == MOEQ_EPI_SILU_MUL)
    hipLaunchKernelGGL(gemm_mx_wave_kernel<MOEQ_EPI_SILU_MUL>, grid, dim3(kThreads), 0, stream, a_q,
                       a_s, a_topk, p, E, R, w, ws, N, K, out, out_f32);
  else
    hipLaunchKernelGGL(gemm_mx_wave_kernel<MOEQ_EPI_NONE>, grid, dim3(kThreads), 0, stream, a_q,
                       a_s, a_topk, p, E, R, w, ws, N, K, out, out_f32);
  return hipGetLastError();
}

}  // namespace moeq
