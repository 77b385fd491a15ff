// Grouped GEMM over the routed experts with MXFP4 activations and MXFP4 weights
// (formats, tiled weight order and matrix step in mx.hpp):
//   out[p, n] = epilogue( sum_k A[row(p), k] W[e(p), n, k] ),  fp32 sums
// row(p) = p (activations in plan order) or sorted_rows[p] / topk (activations in
// token order, read in place: no gathered copy of the k rows per token).
//
// Two kernels (which one: mx_shape below):
//  * K-split units, for few rows per expert: one workgroup per (plan tile of <= 64
//    rows, two 16-row weight blocks -- 32 output columns, or 16 gate rows with
//    their 16 up rows); wave q sweeps the super-groups of K quarter q, the four
//    partial sums meet in LDS in the fixed order s0 + (s1 + (s2 + s3)).  Every load
//    goes straight to registers.  Bound by HBM: 4 tokens, top-6 of 256 experts,
//    4096 x 4096 gate/up in 33.6 us, 6.1 TB/s of weights (a pure read: 6.28).
//  * Tiles, for many: 64 plan rows x 64 CB weight rows, activations shared through
//    LDS, weights straight to registers.  2048 tokens, top-6 of 256, 4096 x 4096
//    gate/up in 386 us, 6.0 TB/s of HBM (95% of a pure read); Zipf-popular experts,
//    4096 x 2048 down 237 us, 5.3 TB/s (equal items per XCD, but not equal weight
//    streams).  Experts of hundreds of rows are not bound by HBM: one of 8192 rows
//    105 us, 2.6 PFLOP/s of the 8.0 that the matrix instruction reaches from registers
//    (384 rows each of 256 experts: 2.5).  No unit is full there: matrix units busy
//    0.33, VALU 0.42, L2 to each CU 27 B per clock, waves waiting 0.35 of their time;
//    a weight is used for 64 rows, two waves share a SIMD and meet every 512 K.
#include "front.hpp"
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

// ------------------------------------------------------------- tile kernel
// Work item `idx` of the plan's (row tile, N-tile) pairs, N-tile major and row
// tile minor inside an expert.  The clamps make a plan built for other sizes
// yield wrong rows, never an access outside the buffers.
struct TileItem {
  int e, row0, rows, nt;
  bool shared_w;          // the expert has other row tiles, which read the same weights
};
__device__ __forceinline__ TileItem tile_item(const PlanView& pv, int E, int R, int n_ntiles, int idx) {
  TileItem it;
  const int tb = idx / n_ntiles;
  it.e = min(max(pv.tile_expert[tb], 0), E - 1);
  const int base = min(max(pv.offsets[it.e], 0), R);
  const int end = min(max(pv.offsets[it.e + 1], base), R);
  const int m = max(1, (end - base + MOEQ_TILE_M - 1) / MOEQ_TILE_M);
  const int t0 = tb - min(max((pv.tile_row0[tb] - base) / MOEQ_TILE_M, 0), tb);
  const int local = min(max(idx - t0 * n_ntiles, 0), m * n_ntiles - 1);
  it.nt = local / m;
  it.row0 = min(base + MOEQ_TILE_M * (local - it.nt * m), R);
  it.rows = max(0, min(MOEQ_TILE_M, end - it.row0));
  it.shared_w = m > 1;
  return it;
}

// LDS position of 16-byte piece p of an activation row: pieces are XOR-swizzled so
// that the 16 rows of two values of kb (bit 2 of p) read 32 different 16-byte units
// mod 512 bytes.  (Counters still show 4.6 conflict cycles per read; a swizzle with
// half as many measured the same time on every shape.)
__device__ __forceinline__ int swizzle(int row, int p) {
  const int m = (row & 15) >> 1;
  return p ^ ((m & 3) | ((m & 4) << 1));
}

// One workgroup per work item; XCD x takes a contiguous run of them (workgroups go
// to the XCDs round-robin), so the row tiles that read one weight slice run side by
// side on one XCD and share it through its L2.  Measured and not kept (gate/up of
// 2048 tokens, 390 us): N-tiles dealt over the XCDs, each reading a share of every
// expert, 415; persistent workgroups whose loads run across items, 403.
//
// A wave keeps one super-group of its CB weight blocks in registers (16 KB in flight
// for CB = 4) and reloads a step's registers as soon as its products are issued.
// Two super-groups (CB = 2) cost the third wave per SIMD: 18.6 us against 14.4 at
// 2331 rows of 1440, 12 experts of 1504 columns.
template <int EPI, int CB>
__global__ void __launch_bounds__(kThreads, 2)
gemm_mx_tile_kernel(const uint8_t* a_q, const uint8_t* a_s, int a_topk, const int32_t* plan, int E,
                    int R, const uint8_t* w, const uint8_t* ws, int N, int K, void* out,
                    int out_f32) {
  constexpr int kBlocks = 4 * CB;                       // 16-row weight blocks per workgroup
  constexpr int kRowBytes = kMxSuper / 2;               // codes of one row, one super-group
  __shared__ __align__(16) uint8_t As[2][MOEQ_TILE_M * kRowBytes];
  __shared__ __align__(16) uint32_t Ss[2][MOEQ_TILE_M * 4];

  const PlanView pv = plan_view(const_cast<int32_t*>(plan), E, R);
  const int n_ntiles = (N / 16 + kBlocks - 1) / kBlocks;
  const int n_real = min(max(plan[kPlanTiles], 0), pv.max_tiles);
  const int items = n_real * n_ntiles;
  const int x = int(blockIdx.x) % kXcds, xi = int(blockIdx.x) / kXcds;
  const int per = items / kXcds, rem = items - per * kXcds;
  if (xi >= per + (x < rem ? 1 : 0)) return;            // workgroup-uniform
  const TileItem it = tile_item(pv, E, R, n_ntiles, x * per + min(x, rem) + xi);
  const int nrb = (it.rows + 15) >> 4;

  const auto body = [&](auto cp) {
    constexpr int CP = decltype(cp)::value;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, kb = lane >> 4;
    const int KB = K / kMxBlock, G = mx_supers(K);

    // weight blocks of this wave: CB consecutive ones, or CB / 2 gate blocks and
    // their up blocks; past the last block the last one again (never stored)
    const int nb = N / 16;
    int blk[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      if (EPI == MOEQ_EPI_SILU_MUL)
        blk[j] = min((it.nt * 4 + wave) * (CB / 2) + j % (CB / 2), nb / 2 - 1) + (j < CB / 2 ? 0 : nb / 2);
      else
        blk[j] = min((it.nt * 4 + wave) * CB + j, nb - 1);
    }
    const uint8_t* wb[CB];
    const uint8_t* sb[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int64_t at = (int64_t(it.e) * nb + blk[j]) * G;
      wb[j] = w + at * kMxCodeBytes;
      sb[j] = ws + at * kMxScaleBytes;
    }

    // activation staging: thread t takes piece t % 16 of rows t / 16 + 16 i, and
    // the scale dword t % 4 of row t / 4; rows past the tile repeat its first
    const int sp = tid & 15;
    const auto sorted = [&](int r) {
      const int p = min(it.row0 + (r < it.rows ? r : 0), R - 1);
      return a_topk ? pv.sorted_rows[p] : p;
    };
    const auto source = [&](int row) -> int64_t {
      return a_topk ? min(max(row, 0), R - 1) / a_topk : row;
    };
    int sorted_row[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) sorted_row[i] = sorted(16 * i + (tid >> 4));
    sorted_row[4] = sorted(tid >> 2);

    // the first super-group's weights go out while the rows are looked up
    uint4 wr[kMxSteps][CB];                             // a super-group's codes, step by step
    uint32_t wsc[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) wsc[j] = load_scale4<CP>(sb[j], 0, uint32_t(lane * 4));
#pragma unroll
    for (int s = 0; s < kMxSteps; ++s)
#pragma unroll
      for (int j = 0; j < CB; ++j) wr[s][j] = load_weight16<CP>(wb[j], s * 1024, uint32_t(lane * 16));
    __builtin_amdgcn_sched_barrier(0);

    const uint8_t* arow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) arow[i] = a_q + source(sorted_row[i]) * (K >> 1) + sp * 16;
    const uint8_t* srow = a_s + source(sorted_row[4]) * KB + 4 * (tid & 3);

    uint4 ap[4];
    uint32_t asc;
    auto load_a = [&](int sg) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ap[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < nrb && 16 * sg + sp < KB)
          ap[i] = *reinterpret_cast<const uint4*>(arow[i] + sg * kRowBytes);
      }
      const int b0 = 16 * sg + 4 * (tid & 3);
      asc = kMxOne4;
      if ((KB & 3) == 0) {
        if (b0 < KB) asc = *reinterpret_cast<const uint32_t*>(srow + 16 * sg);
      } else {
        asc = 0;
#pragma unroll
        for (int j = 0; j < kMxSteps; ++j)
          asc |= uint32_t(b0 + j < KB ? srow[16 * sg + j] : 127) << (8 * j);
      }
    };
    auto park_a = [&](int buf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * i + (tid >> 4);
        if (i < nrb) *reinterpret_cast<uint4*>(&As[buf][r * kRowBytes + swizzle(r, sp) * 16]) = ap[i];
      }
      Ss[buf][tid] = asc;
    };

    mx_v4f acc[4][CB];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) acc[i][j] = mx_v4f{0.f, 0.f, 0.f, 0.f};

    // Activations run two super-groups ahead of their use: loaded into registers in
    // one pass of the loop, parked in the free half of LDS at the top of the next,
    // read in the one after.
    load_a(0);
    park_a(0);
    if (G > 1) load_a(1);
    lds_barrier();

    for (int sg = 0; sg < G; ++sg) {
      const int buf = sg & 1;
      const bool more = sg + 1 < G;
      uint32_t nsc[CB];
      if (more) park_a(buf ^ 1);
      if (sg + 2 < G) load_a(sg + 2);
#pragma unroll
      for (int j = 0; j < CB; ++j)
        nsc[j] = more ? load_scale4<CP>(sb[j], (sg + 1) * kMxScaleBytes, uint32_t(lane * 4)) : 0u;
      uint32_t as[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) as[i] = Ss[buf][(16 * i + ln) * 4 + kb];
      static_for<kMxSteps>([&](auto s) {
        const int at = ln * kRowBytes + swizzle(ln, 4 * kb + s) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < nrb) {
            const uint4 a = *reinterpret_cast<const uint4*>(&As[buf][i * 16 * kRowBytes + at]);
#pragma unroll
            for (int j = 0; j < CB; ++j) acc[i][j] = mx_mfma<s>(wr[s][j], wsc[j], a, as[i], acc[i][j]);
          }
        }
        // the step's registers take the next super-group's codes
        __builtin_amdgcn_sched_barrier(0);
        if (more) {
#pragma unroll
          for (int j = 0; j < CB; ++j)
            wr[s][j] = load_weight16<CP>(wb[j], ((sg + 1) * kMxSteps + s) * 1024, uint32_t(lane * 16));
        }
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int j = 0; j < CB; ++j) wsc[j] = nsc[j];
      lds_barrier();
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * i + ln;
      if (r >= it.rows) continue;
      const int64_t p = it.row0 + r;
      if constexpr (EPI == MOEQ_EPI_SILU_MUL) {
#pragma unroll
        for (int j = 0; j < CB / 2; ++j) {
          const int g = (it.nt * 4 + wave) * (CB / 2) + j;
          if (g < nb / 2)
            store4(out, 0, p * (N >> 1) + 16 * g + 4 * kb, silu_mul4(acc[i][j], acc[i][j + CB / 2]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          const int b = (it.nt * 4 + wave) * CB + j;
          if (b < nb) store4(out, out_f32, p * N + 16 * b + 4 * kb, acc[i][j]);
        }
      }
    }
  };
  if (it.shared_w) body(std::integral_constant<int, kCpKeep>());
  else body(std::integral_constant<int, kCpStream>());
}

// Which kernel takes R rows over E experts of N weight rows, and its grid.
//
// Few rows per expert: the K-split units, otherwise the tile kernel.  Measured on
// the gate/up product (K-split against tile kernel, us): E = 256 experts: R = 1536
// rows 350 / 360, 2046 rows 371 / 356; E = 64: 512 rows 26.3 / 27.7, 1024 33.2 / 29.7;
// E = 16: 128 rows 25.6 / 26.4, 256 30.5 / 26.6; E = 4: 128 rows 13.0 / 15.3, 256 22.0 /
// 16.8; E = 1: 128 rows 10.3 / 15.1, 512 26.2 / 17.7.
// Tiles of 256 weight rows if they make two workgroups per CU, which is what fits,
// else of 128: E = 4, 256 rows each: 24.2 us with 256 (320 items), 21.9 with 128;
// E = 1, 2048 rows: 30.2 (528 items) and 41.2.
struct MxShape {
  int cb;               // weight blocks per wave of the tile kernel; 0: K-split units
  int64_t grid;
};
MxShape mx_shape(int E, int R, int N) {
  const int64_t tiles = plan_max_tiles(E, R);
  if (R <= 7 * E || R <= 160) return {0, tiles * (N / 32)};
  const int64_t wide = tiles * ((N + 255) / 256);
  if (wide >= 512) return {4, wide};
  return {2, tiles * ((N + 127) / 128)};
}

}  // namespace

int64_t mxfp4_gemm_grid(int E, int R, int N) { return mx_shape(E, R, N).grid; }

hipError_t launch_grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, int a_topk,
                                     const void* plan, int E, int R, const uint8_t* w,
                                     const uint8_t* ws, int N, int K, int epilogue, void* out,
                                     int out_dtype, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const int out_f32 = out_dtype == MOEQ_F32 ? 1 : 0;
  const int32_t* p = static_cast<const int32_t*>(plan);
  const MxShape shape = mx_shape(E, R, N);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(shape.grid)), dim3(kThreads), 0, stream, a_q, a_s,
                       a_topk, p, E, R, w, ws, N, K, out, out_f32);
  };
  auto go = [&](auto epi) {
    constexpr int EPI = decltype(epi)::value;
    if (shape.cb == 0) launch(gemm_mx_wave_kernel<EPI>);
    else if (shape.cb == 4) launch(gemm_mx_tile_kernel<EPI, 4>);
    else launch(gemm_mx_tile_kernel<EPI, 2>);
  };
  if (epilogue == MOEQ_EPI_SILU_MUL) go(std::integral_constant<int, MOEQ_EPI_SILU_MUL>());
  else go(std::integral_constant<int, MOEQ_EPI_NONE>());
  return hipGetLastError();
}

}  // namespace moeq
