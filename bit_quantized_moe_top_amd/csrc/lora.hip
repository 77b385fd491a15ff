// moe_shared_gemm_lora_bf16: out = epilogue(x W^T + u B_l^T), u = scale_l x A_l^T, l the
// adapter of the row, on v_mfma_f32_16x16x32_bf16 with fp32 sums.
//
// Rows are taken in the plan's order, grouped by adapter, and written back to their own
// place; so a block of rows meets few adapters, and a row tile of the shared product reads
// gathered rows at no extra cost (each lane has its row's address anyway).
//
//   lora_shrink_kernel   u of 16 rows of one adapter x 32 columns: four waves share K.  u is
//                        stored as two bf16 values, hi = bf16(u) and lo = bf16(u - hi), 16
//                        significant bits, since the second product's matrix instruction
//                        takes bf16: the error left, 2^-17 of the adapter's part, is small
//                        against the rounding of out (2^-9).
//   lora_gemm_kernel     64 x 64 tiles of the shared product, then the adapters' part onto
//                        the same accumulators, then the epilogue.
//
// The matrix instruction's lane layout: operand lane (row l % 16, kq = l / 16) holds k = 8 kq
// .. 8 kq + 7; result lane l holds column l % 16 of rows 4 (l / 16) .. 4 (l / 16) + 3.
#include "common.hpp"
#include "lora_kernels.hpp"

namespace moeq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma(const uint4& a, const uint4& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
// 8 elements at k of a row of n (a multiple of 8), 0 past its end
__device__ __forceinline__ uint4 load_k(const uint16_t* row, int k, int n) {
  return k < n ? load16(row + k) : make_uint4(0u, 0u, 0u, 0u);
}

// u of sorted row p, slice s: r hi values, then r lo values
__device__ __forceinline__ int64_t u_at(int64_t p, int s, int slices, int r) {
  return (p * slices + s) * 2 * r;
}

// round to nearest even (NaNs stay NaNs)
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

// f as hi + lo; the largest finite values are cut off instead of rounded up to infinity, and
// an infinity has no rest
__device__ __forceinline__ void split2(float f, uint16_t& hi, uint16_t& lo) {
  hi = to_bf16(f);
  if (fabsf(f) > 0x1.fep127f) hi = uint16_t(f2u(f) >> 16);
  lo = to_bf16(fabsf(f) == INFINITY ? 0.0f : f - bf16_to_f32(hi));
}

// sorted position -> row, inside [0, M) whatever the plan holds
__device__ __forceinline__ int plan_row(const PlanView& pv, int p, int M) {
  return min(max(pv.sorted_rows[min(p, M - 1)], 0), M - 1);
}

// ------------------------------------------------------------------ shrink
constexpr int kShrinkRows = 16, kShrinkCols = 32;

__global__ void __launch_bounds__(256)
lora_shrink_kernel(LoraArgs args, LoraShape s, uint16_t* __restrict__ u) {
  __shared__ v4f red[3][2][kWave];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  // blockIdx.x: plan tile and its 16-row part; blockIdx.y: 32 columns of u
  constexpr int kParts = MOEQ_TILE_M / kShrinkRows;
  const int tile = blockIdx.x / kParts, part = blockIdx.x % kParts;
  if (tile >= min(pv.base[kPlanTiles], pv.max_tiles)) return;
  const int l = pv.tile_expert[tile];
  if (l < 0 || l >= s.L) return;                         // rows without an adapter
  const int p0 = pv.tile_row0[tile] + part * kShrinkRows;
  const int p1 = min(min(pv.offsets[l + 1], s.M), pv.tile_row0[tile] + MOEQ_TILE_M);
  if (p0 < 0 || p0 >= p1) return;
  const int cols = s.slices * s.r, c0 = blockIdx.y * kShrinkCols;
  const uint16_t* x = args.a + int64_t(plan_row(pv, min(p0 + ln, p1 - 1), s.M)) * s.ld_a;
  const uint16_t* arow[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    arow[q] = args.lora_a + (int64_t(l) * cols + min(c0 + 16 * q + ln, cols - 1)) * s.K;
  v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
  for (int k0 = 32 * wave; k0 < s.K; k0 += 128) {
    const int k = k0 + 8 * kq;
    const uint4 xv = load_k(x, k, s.K);
#pragma unroll
    for (int q = 0; q < 2; ++q) acc[q] = mfma(xv, load_k(arow[q], k, s.K), acc[q]);
  }
  if (wave > 0) {
    red[wave - 1][0][lane] = acc[0];
    red[wave - 1][1][lane] = acc[1];
  }
  __syncthreads();
  if (wave > 0) return;
  const float scale = args.scale[l];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const v4f sum = acc[q] + (red[0][q][lane] + (red[1][q][lane] + red[2][q][lane]));
    const int c = c0 + 16 * q + ln;
    if (c >= cols) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int p = p0 + 4 * kq + v;
      if (p >= p1) continue;
      const float f = sum[v] * scale;
      uint16_t* at = u + u_at(p, c / s.r, s.slices, s.r) + c % s.r;
      split2(f, at[0], at[s.r]);
    }
  }
}

// ------------------------------------------------------- the adapters' part
// First adapter (or the last group) with rows past sorted position p.
__device__ __forceinline__ int adapter_at(const PlanView& pv, int L, int p, int lane) {
  int n = 0;
  for (int a0 = 0; a0 <= L; a0 += kWave)
    n += __popcll(__ballot(a0 + lane <= L && pv.offsets[min(a0 + lane, L) + 1] <= p));
  return n;
}

// acc[i][q] += u B_l^T for the wave's rows p0 + 16 i .. and w rows wrow[q] .. + 15.  The
// product of one adapter is formed by itself and added to its own rows only: what another
// adapter holds, infinities and NaN too, does not reach them.
template <int MB, int NQ>
__device__ __forceinline__ void add_adapters(v4f (&acc)[MB][NQ], const PlanView& pv,
                                             const LoraArgs& args, const LoraShape& s,
                                             const uint16_t* u, int p0, const int (&wrow)[NQ],
                                             int lane) {
  const int ln = lane & 15, kq = lane >> 4;
  const int pend = min(p0 + 16 * MB, s.M);
  for (int l = adapter_at(pv, s.L, p0, lane); l < s.L; ++l) {
    const int lo = max(pv.offsets[l], p0), hi = min(pv.offsets[l + 1], pend);
    if (lo >= pend) break;
    if (lo >= hi) continue;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int slice = s.slices == 2 && wrow[q] >= s.N / 2;
      const uint16_t* b = args.lora_b + (int64_t(l) * s.N + wrow[q] + ln) * s.r;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if (p0 + 16 * i >= hi || p0 + 16 * i + 16 <= lo) continue;
        const uint16_t* up = u + u_at(min(p0 + 16 * i + ln, s.M - 1), slice, s.slices, s.r);
        v4f d = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < s.r; k0 += 32) {
          const int k = k0 + 8 * kq;
          const uint4 bv = load_k(b, k, s.r);
          d = mfma(load_k(up, k, s.r), bv, d);
          d = mfma(load_k(up + s.r, k, s.r), bv, d);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int p = p0 + 16 * i + 4 * kq + v;
          acc[i][q][v] += p >= lo && p < hi ? d[v] : 0.0f;
        }
      }
    }
  }
}

// ------------------------------------------------------------- shared product
constexpr int kTile = 64, kStep = 32, kPadRow = kStep + 8;

template <int EPI>
__global__ void __launch_bounds__(256)
lora_gemm_kernel(LoraArgs args, LoraShape s, const uint16_t* __restrict__ u) {
  __shared__ __align__(16) uint16_t As[kTile * kPadRow], Bs[kTile * kPadRow];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  constexpr bool kSilu = EPI == MOEQ_EPI_SILU_MUL;
  const int cols = kSilu ? s.N / 2 : s.N;                // output columns, a multiple of 16
  constexpr int kOutTile = kSilu ? kTile / 2 : kTile;    // output columns per workgroup
  const int ntiles = (cols + kOutTile - 1) / kOutTile;
  const int mt = blockIdx.x / ntiles, nt = blockIdx.x - mt * ntiles;
  const int m0 = mt * kTile, n0 = nt * kOutTile;
  const int wm = wave >> 1, wn = wave & 1;

  // w row of tile row i: 64 columns, or 32 gate and their 32 up rows; past the end the last one
  // again (its results are not stored)
  const auto w_row = [&](int i) {
    if (kSilu) return i < kTile / 2 ? min(n0 + i, cols - 1) : cols + min(n0 + i - kTile / 2, cols - 1);
    return min(n0 + i, cols - 1);
  };
  // the wave's 16-column blocks: two of its half, or one gate block and the matching up block
  const auto block_row = [&](int q) { return kSilu ? q * (kTile / 2) + 16 * wn : 32 * wn + 16 * q; };

  const int sr = tid >> 2, sk = (tid & 3) * 8;
  const uint16_t* xsrc = args.a + int64_t(plan_row(pv, m0 + sr, s.M)) * s.ld_a;
  const uint16_t* wsrc = args.w + int64_t(w_row(sr)) * s.K;
  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) acc[i][q] = v4f{0.f, 0.f, 0.f, 0.f};
  uint4 xv = load_k(xsrc, sk, s.K), wv = load_k(wsrc, sk, s.K);
  for (int k0 = 0; k0 < s.K; k0 += kStep) {
    *reinterpret_cast<uint4*>(&As[sr * kPadRow + sk]) = xv;
    *reinterpret_cast<uint4*>(&Bs[sr * kPadRow + sk]) = wv;
    __syncthreads();
    xv = load_k(xsrc, k0 + kStep + sk, s.K);
    wv = load_k(wsrc, k0 + kStep + sk, s.K);
    uint4 a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = load16(&As[(32 * wm + 16 * i + ln) * kPadRow + 8 * kq]);
#pragma unroll
    for (int q = 0; q < 2; ++q) b[q] = load16(&Bs[(block_row(q) + ln) * kPadRow + 8 * kq]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[i][q] = mfma(a[i], b[q], acc[i][q]);
    __syncthreads();
  }
  // first w row of each column block, kept inside W for blocks past the last column
  int wrow[2], ocol[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    ocol[q] = n0 + (kSilu ? 16 * wn : block_row(q));
    wrow[q] = min(ocol[q], cols - 16) + (kSilu && q ? cols : 0);
  }
  const int p0 = m0 + 32 * wm;
  add_adapters<2, 2>(acc, pv, args, s, u, p0, wrow, lane);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int p = p0 + 16 * i + 4 * kq + v;
      if (p >= s.M) continue;
      uint16_t* o = args.out + int64_t(plan_row(pv, p, s.M)) * cols;
      if (kSilu) {
        if (ocol[0] < cols) o[ocol[0] + ln] = to_bf16(silu_f32(acc[i][0][v]) * acc[i][1][v]);
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (ocol[q] < cols) o[ocol[q] + ln] = to_bf16(acc[i][q][v]);
      }
    }
  }
}

// ------------------------------------------------------------------ few rows
// Up to 64 rows: bound by the stream of W.  One launch multiplies (64 w rows x all rows x a
// range of K per workgroup, fp32 parts to the workspace) and, in its first workgroups, forms u,
// which does not depend on the product; a second one adds the parts and the adapters, and
// applies the epilogue.
//
// The product's workgroup takes K in pieces of 512: each wave holds its 16 w rows' piece in
// registers, 16 loads of 16 bytes per lane that go out at once (two consecutive ones fill whole
// 128-byte lines), while the x rows' piece is staged in LDS, which the four waves share.  16-byte
// piece c of LDS row r sits at c ^ 2 (r % 16): the 16 rows x 2 pieces that 32 lanes of an operand
// read take are then 32 different 16-byte slots of 512 bytes.
//
// Parts are stored as the matrix instruction leaves them: 16 bytes per lane, 1 KB per block.
constexpr int kFewRows = 64, kFewPiece = 512, kFewCols = 64;
constexpr int kFewSteps = kFewPiece / 32;

__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}

// the plan's tiles by lane (at most 64 of up to 64 rows), and the adapter of a sorted row
struct FewPlan {
  int n, row0, expert;
  __device__ __forceinline__ FewPlan(const PlanView& pv, int lane) {
    n = min(min(pv.base[kPlanTiles], pv.max_tiles), kWave);
    row0 = pv.tile_row0[min(lane, pv.max_tiles - 1)];
    expert = pv.tile_expert[min(lane, pv.max_tiles - 1)];
  }
  // the plan tile of sorted row p (-1: none)
  __device__ __forceinline__ int tile(int p, int lane) const {
    return __popcll(__ballot(lane < n && row0 <= p)) - 1;
  }
};

// u (fp32) of up to 16 rows of one adapter x 32 columns: block `b` of the list of 16-row pieces
__device__ __forceinline__ void few_shrink(const LoraArgs& args, const LoraShape& s, float* u, int b,
                                           int c0, v4f* red) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const FewPlan fp(pv, lane);
  // rows of each tile, and the 16-row pieces before it
  const int next = __shfl_down(fp.row0, 1);
  const int end = min(lane + 1 < fp.n ? next : s.M, s.M);
  const bool has = lane < fp.n && fp.expert >= 0 && fp.expert < s.L && fp.row0 >= 0;
  const int rows = has ? min(max(end - fp.row0, 0), MOEQ_TILE_M) : 0;
  const int pieces = (rows + 15) / 16;
  const int before = wave_inclusive_scan(pieces) - pieces;
  const uint64_t mine = __ballot(pieces > 0 && b >= before && b < before + pieces);
  if (mine == 0) return;
  const int t = __ffsll(static_cast<unsigned long long>(mine)) - 1;
  const int l = readlane(fp.expert, t);
  const int p0 = readlane(fp.row0, t) + 16 * (b - readlane(before, t));
  const int p1 = min(p0 + 16, readlane(fp.row0, t) + readlane(rows, t));
  const int cols = s.slices * s.r;
  const uint16_t* x = args.a + int64_t(plan_row(pv, min(p0 + ln, p1 - 1), s.M)) * s.ld_a;
  const uint16_t* arow[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    arow[q] = args.lora_a + (int64_t(l) * cols + min(c0 + 16 * q + ln, cols - 1)) * s.K;
  v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
  constexpr int kU = 4;
  for (int k0 = 32 * kU * wave; k0 < s.K; k0 += 32 * kU * 4) {
    uint4 xv[kU], av[2][kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int k = k0 + 32 * j + 8 * kq;
      xv[j] = load_k(x, k, s.K);
      av[0][j] = load_k(arow[0], k, s.K);
      av[1][j] = load_k(arow[1], k, s.K);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      acc[0] = mfma(xv[j], av[0][j], acc[0]);
      acc[1] = mfma(xv[j], av[1][j], acc[1]);
    }
  }
  if (wave > 0) {
    red[((wave - 1) * 2) * kWave + lane] = acc[0];
    red[((wave - 1) * 2 + 1) * kWave + lane] = acc[1];
  }
  __syncthreads();
  if (wave > 0) return;
  const float scale = args.scale[l];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const v4f sum = acc[q] + (red[q * kWave + lane] + (red[(2 + q) * kWave + lane] + red[(4 + q) * kWave + lane]));
    const int c = c0 + 16 * q + ln;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int p = p0 + 4 * kq + v;
      if (c < cols && p < p1) u[int64_t(p) * cols + c] = sum[v] * scale;
    }
  }
}

template <int MB>
__global__ void __launch_bounds__(256, 2)
lora_few_kernel(LoraArgs args, LoraShape s, float* __restrict__ u, v4f* __restrict__ parts,
                int shrink_blocks, int shrink_cols, int pieces_per_split) {
  extern __shared__ __align__(16) uint8_t lds[];
  if (int(blockIdx.x) < shrink_blocks) {
    few_shrink(args, s, u, blockIdx.x / shrink_cols, (blockIdx.x % shrink_cols) * 32,
               reinterpret_cast<v4f*>(lds));
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const int ntiles = (s.N + kFewCols - 1) / kFewCols;
  const int b = blockIdx.x - shrink_blocks;
  const int split = b / ntiles, nt = b - split * ntiles;
  const int n0 = nt * kFewCols + 16 * wave;
  const uint16_t* wsrc = args.w + int64_t(min(n0 + ln, s.N - 1)) * s.K;
  const int pieces = (s.K + kFewPiece - 1) / kFewPiece;
  const int c0 = split * pieces_per_split, c1 = min(c0 + pieces_per_split, pieces);

  uint4 wv[kFewSteps];
  auto load_w = [&](int c) {
#pragma unroll
    for (int j = 0; j < kFewSteps; ++j) {
      const int k = c * kFewPiece + 32 * j + 8 * kq;
      const uint4 v = load_stream(wsrc + min(k, s.K - 8));
      wv[j] = k < s.K ? v : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // x: thread -> piece tid % 64 of rows tid / 64, + 4, ...
  const uint16_t* xsrc[4 * MB];
#pragma unroll
  for (int i = 0; i < 4 * MB; ++i)
    xsrc[i] = args.a + int64_t(plan_row(pv, wave + 4 * i, s.M)) * s.ld_a;
  load_w(c0);
  v4f acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; ++c) {
    uint4 xv[4 * MB];
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) xv[i] = load_k(xsrc[i], c * kFewPiece + 8 * lane, s.K);
    if (c > c0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) {
      const int row = wave + 4 * i;
      *reinterpret_cast<uint4*>(lds + row * (2 * kFewPiece) + ((lane ^ (2 * (row & 15))) * 16)) = xv[i];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kFewSteps; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const uint4 a = *reinterpret_cast<const uint4*>(
            lds + (16 * i + ln) * (2 * kFewPiece) + (((4 * j + kq) ^ (2 * ln)) * 16));
        acc[i] = mfma(a, wv[j], acc[i]);
      }
    if (c + 1 < c1) load_w(c + 1);
  }
  if (n0 >= s.N) return;
  const int nb = s.N / 16;
#pragma unroll
  for (int i = 0; i < MB; ++i)
    if (16 * i < s.M) parts[((int64_t(split) * ((s.M + 15) / 16) + i) * nb + n0 / 16) * kWave + lane] = acc[i];
}

// parts and adapters joined: a wave forms 16 rows x 16 output columns (of the gate and the up
// half with SILU_MUL).  Lane l has column l % 16 of rows 4 (l / 16) .. + 3, whose adapters may all
// differ: it reads their B rows for its column (r consecutive values) and u, and sums r products in
// fp32 for each.  All of these loads are independent.
template <int EPI>
__global__ void __launch_bounds__(256)
lora_join_kernel(LoraArgs args, LoraShape s, const float* __restrict__ u,
                 const v4f* __restrict__ parts, int splits) {
  constexpr bool kSilu = EPI == MOEQ_EPI_SILU_MUL;
  constexpr int kHalves = kSilu ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const int cols = kSilu ? s.N / 2 : s.N;
  const int cblocks = cols / 16, mblocks = (s.M + 15) / 16, nb = s.N / 16;
  const int item = blockIdx.x * 4 + wave;
  if (item >= cblocks * mblocks) return;
  const int mb = item / cblocks, cb = item - mb * cblocks;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const FewPlan fp(pv, lane);
  v4f acc[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    const v4f* at = parts + (int64_t(mb) * nb + cb + h * cblocks) * kWave + lane;
    acc[h] = at[0];
    for (int i = 1; i < splits; ++i) acc[h] = acc[h] + at[int64_t(i) * mblocks * nb * kWave];
  }
  // lane i < 16: the adapter of row 16 mb + i (-1: none)
  int adapter = -1;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int p = 16 * mb + i;
    const int t = fp.tile(p, lane);
    const int e = readlane(fp.expert, max(t, 0));
    if (lane == i && t >= 0 && p < s.M && e >= 0 && e < s.L) adapter = e;
  }
  const int ucols = s.slices * s.r;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int l = __shfl(adapter, 4 * kq + v);
    if (l < 0) continue;
    const float* ur = u + int64_t(16 * mb + 4 * kq + v) * ucols;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int n = (cb + h * cblocks) * 16 + ln;
      const uint16_t* br = args.lora_b + (int64_t(l) * s.N + n) * s.r;
      const float* us = ur + (s.slices == 2 && n >= s.N / 2 ? s.r : 0);
      float d = 0.0f;
      for (int j = 0; j < s.r; j += 8) {
        float bv[8];
        bf16x8_to_f32(load16(br + j), bv);
        const float4 u0 = *reinterpret_cast<const float4*>(us + j);
        const float4 u1 = *reinterpret_cast<const float4*>(us + j + 4);
        d = fmaf(u0.x, bv[0], d); d = fmaf(u0.y, bv[1], d);
        d = fmaf(u0.z, bv[2], d); d = fmaf(u0.w, bv[3], d);
        d = fmaf(u1.x, bv[4], d); d = fmaf(u1.y, bv[5], d);
        d = fmaf(u1.z, bv[6], d); d = fmaf(u1.w, bv[7], d);
      }
      acc[h][v] += d;
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int p = 16 * mb + 4 * kq + v;
    if (p >= s.M) continue;
    const float f = kSilu ? silu_f32(acc[0][v]) * acc[kHalves - 1][v] : acc[0][v];
    args.out[int64_t(plan_row(pv, p, s.M)) * cols + cb * 16 + ln] = to_bf16(f);
  }
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// splits of K of the few-row product: about 512 workgroups, whole pieces of K each
struct FewSplit {
  int splits, per_split;
};
FewSplit few_split(const LoraShape& s) {
  const int ntiles = (s.N + kFewCols - 1) / kFewCols, pieces = (s.K + kFewPiece - 1) / kFewPiece;
  int want = (512 + ntiles - 1) / ntiles;
  if (want > pieces) want = pieces;
  const int per = (pieces + want - 1) / want;
  return {(pieces + per - 1) / per, per};
}
size_t few_u_bytes(const LoraShape& s) { return align256(size_t(s.M) * s.slices * s.r * sizeof(float)); }

template <int MB>
hipError_t launch_few(const LoraArgs& args, const LoraShape& s, hipStream_t stream) {
  const FewSplit fs = few_split(s);
  float* u = static_cast<float*>(args.ws);
  v4f* parts = reinterpret_cast<v4f*>(static_cast<uint8_t*>(args.ws) + few_u_bytes(s));
  const int reached = s.L < s.M ? s.L : s.M;             // adapters that have rows, at most
  const int row_pieces = reached + s.M / 16 < s.M ? reached + s.M / 16 : s.M;
  const int shrink_cols = (s.slices * s.r + 31) / 32, shrink = row_pieces * shrink_cols;
  const int ntiles = (s.N + kFewCols - 1) / kFewCols;
  const unsigned lds = 16 * MB * 2 * kFewPiece;          // at least the 6 KB of few_shrink
  hipLaunchKernelGGL(lora_few_kernel<MB>, dim3(unsigned(shrink + ntiles * fs.splits)), dim3(256), lds,
                     stream, args, s, u, parts, shrink, shrink_cols, fs.per_split);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const bool silu = s.epilogue == MOEQ_EPI_SILU_MUL;
  const int items = (silu ? s.N / 2 : s.N) / 16 * ((s.M + 15) / 16);
  const auto join = silu ? lora_join_kernel<MOEQ_EPI_SILU_MUL> : lora_join_kernel<MOEQ_EPI_NONE>;
  hipLaunchKernelGGL(join, dim3(unsigned((items + 3) / 4)), dim3(256), 0, stream, args, s, u, parts,
                     fs.splits);
  return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(const LoraShape& s) {
  if (s.M <= kFewRows)
    return few_u_bytes(s) + align256(size_t(few_split(s).splits) * ((s.M + 15) / 16) * s.N * 16 * sizeof(float)) + 256;
  return align256(size_t(s.M) * s.slices * 2 * s.r * sizeof(uint16_t));
}

hipError_t launch_shared_gemm_lora(const LoraArgs& args, const LoraShape& s, hipStream_t stream) {
  if (s.M == 0) return hipSuccess;
  if (s.M <= 16) return launch_few<1>(args, s, stream);
  if (s.M <= 32) return launch_few<2>(args, s, stream);
  if (s.M <= kFewRows) return launch_few<4>(args, s, stream);
  uint16_t* u = static_cast<uint16_t*>(args.ws);
  const dim3 sgrid(unsigned(plan_max_tiles(s.L + 1, s.M)) * (MOEQ_TILE_M / kShrinkRows),
                   unsigned((s.slices * s.r + kShrinkCols - 1) / kShrinkCols));
  hipLaunchKernelGGL(lora_shrink_kernel, sgrid, dim3(256), 0, stream, args, s, u);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const bool silu = s.epilogue == MOEQ_EPI_SILU_MUL;
  const int cols = silu ? s.N / 2 : s.N, out_tile = silu ? kTile / 2 : kTile;
  const int64_t blocks = int64_t((s.M + kTile - 1) / kTile) * ((cols + out_tile - 1) / out_tile);
  if (silu)
    hipLaunchKernelGGL(lora_gemm_kernel<MOEQ_EPI_SILU_MUL>, dim3(unsigned(blocks)), dim3(256), 0, stream,
                       args, s, u);
  else
    hipLaunchKernelGGL(lora_gemm_kernel<MOEQ_EPI_NONE>, dim3(unsigned(blocks)), dim3(256), 0, stream,
                       args, s, u);
  return hipGetLastError();
}

}  // namespace moeq
