// moe_shared_gemm_lora_bf16: out = epilogue(x W^T + u B_l^T), u = scale_l x A_l^T, l the
// adapter of the row, on v_mfma_f32_16x16x32_bf16 with fp32 sums.
//
// Rows are taken in the plan's order, grouped by adapter, and written back to their own
// place; so a block of rows meets few adapters, and a row tile of the shared product reads
// gathered rows at no extra cost (each lane has its row's address anyway).
//
// u is summed in fp32, in parts over shares of K that the reader adds in their order.  For the
// second product, whose matrix instruction takes bf16, it is split into hi = bf16(u) and lo =
// bf16(u - hi), 16 significant bits: the error left, 2^-17 of the adapter's part, is small against
// the rounding of out (2^-8).
//
// Up to 64 rows the stream of W bounds the call: lora_few_kernel forms parts of the product over
// shares of K next to the parts of u, lora_join_kernel adds them, the adapters' product and the
// epilogue.  More rows: lora_gemm_kernel, in tiles, with the adapters' product onto the tile's
// accumulators; u by lora_shrink_kernel ahead of it, or, where tiles are too few for the card, K is
// split over workgroups too and u's parts are formed by the same launch, and a second one joins.
// Small problems of short K: lora_short_kernel, everything in one launch.
//
//   8192 x 4096, 16 rows on 32 adapters of rank 16: 19.5 us, 74 MB read (3.8 TB/s; W's stream alone
//   10.7 at the 6.3 TB/s that a plain read reaches); 1 row 18.1.  2048 rows: 122 to 133 us from card to
//   card, 1.04 to 1.14 PFLOP/s (a library product of these sizes without adapters: 107 us, 1.29).
//
// The matrix instruction's lane layout: operand lane (row l % 16, kq = l / 16) holds k = 8 kq
// .. 8 kq + 7; result lane l holds column l % 16 of rows 4 (l / 16) .. 4 (l / 16) + 3.
#include <algorithm>
#include <type_traits>

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
// 8 elements at k of a row of n (a multiple of 8), 0 past its end: read inside the row by load_in,
// and dropped by keep.  (A branch would keep the loads around it from being in flight together.)
__device__ __forceinline__ uint4 load_in(const uint16_t* row, int k, int n) { return load16(row + min(k, n - 8)); }
__device__ __forceinline__ uint4 keep(const uint4& v, bool in) {
  return make_uint4(in ? v.x : 0u, in ? v.y : 0u, in ? v.z : 0u, in ? v.w : 0u);
}
__device__ __forceinline__ uint4 load_k(const uint16_t* row, int k, int n) { return keep(load_in(row, k, n), k < n); }

// round to nearest even (NaNs stay NaNs)
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

// f as hi + lo; the largest finite values are cut off instead of rounded up to infinity, and
// an infinity has no rest
__device__ __forceinline__ void split2(float f, uint16_t& hi, uint16_t& lo) {
  hi = to_bf16(f);
  if (fabsf(f) > 0x1.fep127f) hi = uint16_t(f2u(f) >> 16);
  lo = to_bf16(fabsf(f) == INFINITY ? 0.0f : f - bf16_to_f32(hi));
}

// Lane l of a quad holds f of four rows in column l, and leaves with row l of the four columns in bf16:
// one place and one store of 8 bytes a lane, instead of four and four of 2.  (All lanes take part.)
__device__ __forceinline__ uint2 quad_rows(const float (&f)[4], int lane) {
  const uint32_t a = to_bf16(f[0]) | uint32_t(to_bf16(f[1])) << 16, b = to_bf16(f[2]) | uint32_t(to_bf16(f[3])) << 16;
  // rows of the lane's own parity, from it and its neighbour
  const uint32_t sel = lane & 1 ? 0x03020706u : 0x05040100u;
  const uint32_t p0 = __builtin_amdgcn_perm(uint32_t(dpp<kDppQuadSwap1>(0, int(a))), a, sel);
  const uint32_t p1 = __builtin_amdgcn_perm(uint32_t(dpp<kDppQuadSwap1>(0, int(b))), b, sel);
  const bool up = lane & 2;
  const uint32_t other = uint32_t(dpp<kDppQuadSwap2>(0, int(up ? p0 : p1)));
  return up ? make_uint2(other, p1) : make_uint2(p0, other);
}

// sorted position -> row, inside [0, M) whatever the plan holds
__device__ __forceinline__ int plan_row(const PlanView& pv, int p, int M) {
  return min(max(pv.sorted_rows[min(p, M - 1)], 0), M - 1);
}

// ------------------------------------------------------------------ shrink
// Parts of u: 32 rows of one adapter x 32 columns x a share of K per workgroup, summed over its
// four waves, [split][M][columns] in fp32.  A wave takes K in pieces of 128, all of a piece's loads
// in flight at once: the launch is a chain of memory latencies, not of work (2048 rows x 32 columns,
// K = 4096: 11.3 us, 17 MB; 777 x 24, K = 1448: 4.7).
constexpr int kShrinkRows = 32, kShrinkCols = 32;
constexpr int kShrinkSteps = kShrinkPiece / 32;

// Workgroups of one launch: (plan tile and its 32-row part, 32 columns, split of K)
struct ShrinkGrid {
  int parts, cols, splits;
  __host__ __device__ int blocks() const { return parts * cols * splits; }
};

// workgroup b of the grid; red: 16 KB of LDS
__device__ __forceinline__ void shrink(const LoraArgs& args, const LoraShape& s, float* u,
                                       const ShrinkGrid& grid, int b, v4f (*red)[4][kWave]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const int split = b / (grid.parts * grid.cols), at = b - split * grid.parts * grid.cols;
  const int cblock = at / grid.parts, piece = at - cblock * grid.parts;
  constexpr int kParts = MOEQ_TILE_M / kShrinkRows;
  const int tile = piece / kParts, part = piece % kParts;
  // (the plan's words in as few dependent loads as they take: adapter and first row of the tile, then
  // the end of the adapter's rows and the rows' places, then the rows)
  const int n_tiles = pv.base[kPlanTiles], l = pv.tile_expert[tile], row0 = pv.tile_row0[tile];
  if (tile >= n_tiles || l < 0 || l >= s.L || row0 < 0 || row0 >= s.M) return;
  const int p0 = row0 + part * kShrinkRows;
  const int end = pv.offsets[l + 1];
  const int cols = s.slices * s.r, c0 = cblock * kShrinkCols;
  const uint16_t *x[2], *a[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    x[q] = args.a + int64_t(plan_row(pv, p0 + 16 * q + ln, s.M)) * s.ld_a;
    a[q] = args.lora_a + (int64_t(l) * cols + min(c0 + 16 * q + ln, cols - 1)) * s.K;
  }
  const int p1 = min(min(end, s.M), row0 + MOEQ_TILE_M);
  if (p0 >= p1) return;
  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int c = (4 * split + wave) * kShrinkPiece; c < s.K; c += 4 * grid.splits * kShrinkPiece) {
    uint4 xv[2][kShrinkSteps], av[2][kShrinkSteps];
#pragma unroll
    for (int j = 0; j < kShrinkSteps; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) av[q][j] = load_in(a[q], c + 32 * j + 8 * kq, s.K);
#pragma unroll
    for (int j = 0; j < kShrinkSteps; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) xv[q][j] = load_in(x[q], c + 32 * j + 8 * kq, s.K);
    __builtin_amdgcn_sched_barrier(0);                   // all of them in flight
#pragma unroll
    for (int j = 0; j < kShrinkSteps; ++j) {
      const bool in = c + 32 * j + 8 * kq < s.K;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i >> 1][i & 1] = mfma(keep(xv[i >> 1][j], in), keep(av[i & 1][j], in), acc[i >> 1][i & 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i][lane] = acc[i >> 1][i & 1];
  __syncthreads();
  // wave w adds and stores block w: rows 16 (w / 2) .., columns 16 (w % 2) ..
  const v4f sum = (red[0][wave][lane] + red[1][wave][lane]) + (red[2][wave][lane] + red[3][wave][lane]);
  const int col = c0 + 16 * (wave & 1) + ln;
  const float scale = args.scale[l];
  u += int64_t(split) * s.M * cols;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int p = p0 + 16 * (wave >> 1) + 4 * kq + v;
    if (p < p1 && col < cols) u[int64_t(p) * cols + col] = sum[v] * scale;
  }
}

__global__ void __launch_bounds__(256)
lora_shrink_kernel(LoraArgs args, LoraShape s, float* __restrict__ u, ShrinkGrid grid) {
  __shared__ v4f red[4][4][kWave];
  shrink(args, s, u, grid, blockIdx.x, red);
}

// ------------------------------------------------------- the adapters' part
// First adapter (or the last group) with rows past sorted position p.
__device__ __forceinline__ int adapter_at(const PlanView& pv, int L, int p, int lane) {
  int n = 0;
  for (int a0 = 0; a0 <= L; a0 += kWave)
    n += __popcll(__ballot(a0 + lane <= L && pv.offsets[min(a0 + lane, L) + 1] <= p));
  return n;
}

// ------------------------------------------------------- operands through LDS
// Rows of 64 K, one 128-byte line each, loaded straight into LDS.
constexpr int kRowB = 2 * kSlotK;

// Position of 16-byte chunk c of a 128-byte LDS row r: c ^ swz(r).  The 16 rows x 2 chunks that
// 32 lanes of an operand read take are then 32 different 16-byte slots modulo 512 bytes.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// s_waitcnt vmcnt(n), the other counters unconstrained
template <int n>
__device__ __forceinline__ void wait_vmem() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}
// every wave's LDS reads so far are done, without a wait for loads still in flight
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes per lane straight into LDS, lane l's at dst + 16 l (dst a wave-uniform LDS offset).
// Written in assembly: the compiler, which counts such a load as a write of all of LDS, would wait
// for every one in flight ahead of the next LDS read; here the ring's own waits order them.  (No
// register receives the data, so nothing the compiler allocates is written behind its back; m0,
// which names the LDS address, is used by nothing else in these kernels.)
template <bool kOnce>                                    // read once: non-temporal
__device__ __forceinline__ void load_lds(const uint16_t* src, uint32_t dst) {
  if constexpr (kOnce)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt"
                 :: "v"(src), "s"(dst) : "memory");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(src), "s"(dst) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const uint8_t* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p));
}

// ------------------------------------------------------------- shared product
// BM x BN tiles by G groups of kWM x kWN waves, each wave BM / kWM rows x BN / kWN columns.  A group has a
// ring of its own and a G-th of K; the groups' sums meet in LDS.  The ring holds units: the 128-byte
// pieces (64 K) of the tile's w rows or of its x rows, in turn (w first: it comes from farther and has
// half a slot more time).  The first kUnits - 1 go out up front.  A slot (a w unit and the x unit after
// it) is multiplied in two halves of 32 K, row block by row block.  A row block's x operand is read
// anew, for the next half, as soon as its products are issued, so it has a half's time to arrive and
// needs no second register; the w operands, used by all row blocks, have two sets.  The ring moves on
// after kOpen row blocks of the second half of slot st: by then its operands are in registers
// (lgkmcnt(0), which waits for nothing), and this wave's loads of slot st + 1 have landed (all but those
// of the kUnits - 4 units issued after them); after the barrier the same holds for every wave, so slot
// st + 1 can be read, and the next two units take slot st's places.
// The 256 x 256 tile has all of its 256 registers in use: 20 (SILU_MUL) or 24 are kept in scratch memory
// before and after the slots' loop, none within it, 72 or 84 bytes a lane (9.4 or 11 MB of 256 workgroups).
template <int BM_, int BN_, int G>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, kGroups = G;
  static constexpr int kWM = BM > BN ? 4 : 2, kWN = BN == 256 ? 4 : 2, kGroupWaves = kWM * kWN;
  static constexpr int kRows = BM / kWM, kCols = BN / kWN, kM = kRows / 16, kN = kCols / 16;
  static constexpr int kEndM = kM / G;                   // row blocks that a wave finishes
  static constexpr int kXB = BM * kRowB, kWB = BN * kRowB;               // bytes of a unit
  static constexpr int kLX = BM / 8 / kGroupWaves, kLW = BN / 8 / kGroupWaves;   // and loads of a wave
  // a CU's 160 KB for one workgroup of 256 rows or of two groups, half of them for the others
  static constexpr int kRoom = BM == 256 ? 160 * 1024 : 80 * 1024;
  static constexpr int kUnits = BM == BN ? kRoom / kXB : kRoom / (kXB + kWB) * 2;
  static constexpr int kRingB = BM == BN ? kUnits * kXB : kUnits / 2 * (kXB + kWB);
  static constexpr int kLds = G * kRingB, kThreads = 64 * kGroupWaves * G;
  static_assert(kUnits >= 4, "two slots");
  static_assert((G == 1 ? 0 : BM * BN * 4) + BM * (2 * 2 * 128 + 16) <= kLds, "the exchange, and 64 ranks of u");
  // where unit j (j < kUnits) lies; loads of units from .. to - 1 (even: w)
  static __device__ __forceinline__ int place(int j) {
    return BM == BN ? j * kXB : (j >> 1) * (kXB + kWB) + (j & 1) * kWB;
  }
  static constexpr int loads(int from, int to) {
    int n = 0;
    for (int j = from; j < to; ++j) n += j & 1 ? kLX : kLW;
    return n;
  }
};

// acc[i][q] += u B_l^T, i < kEndM, for the rows p0 + 16 i .. and w rows wrow[q] .. + 15, by all waves of
// the workgroup together.  The tile's u, its parts summed, goes to LDS in two bf16 values, 64
// ranks of every slice at a time, [row][slice][hi, lo]; B comes from memory.  The product of one
// adapter is formed by itself and added to its own rows only: what another adapter holds, infinities
// and NaN too, does not reach them.
template <typename T>
__device__ __forceinline__ void add_adapters(v4f (&acc)[T::kM][T::kN], const PlanView& pv,
                                             const LoraArgs& args, const LoraShape& s, const float* u,
                                             int u_splits, uint8_t* lds, int m0, int p0,
                                             const int (&wrow)[T::kN], int lane) {
  constexpr int kM = T::kEndM, kN = T::kN;
  const int ln = lane & 15, kq = lane >> 4;
  const int pend = min(p0 + 16 * kM, s.M);
  // the adapters of the wave's rows: the first, and the offsets of 64 groups from there
  const int first = p0 < s.M ? adapter_at(pv, s.L, p0, lane) : s.L;
  int window = first;
  int off = pv.offsets[min(window + lane, s.L + 1)];
  const auto offset = [&](int l) {
    if (l < window || l - window >= kWave) {
      window = l;
      off = pv.offsets[min(window + lane, s.L + 1)];
    }
    return readlane(off, l - window);
  };
  // the next adapter with rows from l on (s.L: none)
  int lo = 0, hi = 0;
  const auto next_adapter = [&](int l) {
    for (; l < s.L; ++l) {
      lo = max(offset(l), p0);
      hi = min(offset(l + 1), pend);
      if (lo < hi) return l;
      if (lo >= pend) break;
    }
    return s.L;
  };
  const int cols = s.slices * s.r;
  // ranks k0 .. + 63 (or the rest), in steps of 32: one (up to 32 ranks), or two
  const auto pass = [&](int k0, auto n_steps) {
    constexpr int kSteps = decltype(n_steps)::value, kOnce = T::kRows == 128 ? 1 : 16 / (kN * kSteps);
    const int kc = kSteps == 2 && s.r - k0 > 32 ? 64 : 32;               // ranks in LDS, zeros past r
    const int plane = 2 * kc, row_bytes = s.slices * 2 * plane + 16;
    // kOnce adapters' B at a time: what the registers hold
    int id[kOnce], from[kOnce], to[kOnce];
    uint4 b[kOnce][kSteps][kN];
    const auto load_b = [&](int l) {
#pragma unroll
      for (int a = 0; a < kOnce; ++a) {
        l = next_adapter(l);
        id[a] = l;
        from[a] = lo;
        to[a] = hi;
        l = min(l + 1, s.L);
      }
#pragma unroll
      for (int a = 0; a < kOnce; ++a) {
        if (id[a] >= s.L) break;
#pragma unroll
        for (int q = 0; q < kN; ++q) {
          const uint16_t* at = args.lora_b + (int64_t(id[a]) * s.N + wrow[q] + ln) * s.r;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) b[a][j][q] = load_in(at, k0 + 32 * j + 8 * kq, s.r);
        }
      }
    };
    load_b(first);
    if (k0 > 0) __syncthreads();                         // the ranks before are done with
    // u's elements, four at a time, those of kU quads in flight together
    constexpr int kU = T::kRows == 128 ? 1 : 2;          // (what the registers hold)
    const int rows = min(T::BM, s.M - m0), quads = min(s.r - k0, kc) / 4, pads = kc / 4 - quads;
    const int n = rows * s.slices * quads;
    const int64_t u_stride = int64_t(s.M) * cols;
    const auto place = [&](int i, int per, int& k) {     // quad i of rows x slices x `per` quads
      const int at = i / per, row = s.slices == 2 ? at >> 1 : at;
      k = 4 * (i - at * per);
      return lds + row * row_bytes + (s.slices == 2 ? at & 1 : 0) * 2 * plane;
    };
    for (int i0 = threadIdx.x; i0 < n; i0 += kU * T::kThreads) {
      v4f v[kU][4];
#pragma unroll
      for (int a = 0; a < kU; ++a) {
        const int i = min(i0 + a * T::kThreads, n - 1), at = i / quads;
        const float* src = u + int64_t(m0) * cols + int64_t(at) * s.r + k0 + 4 * (i - at * quads);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < u_splits) v[a][j] = *reinterpret_cast<const v4f*>(src + j * u_stride);
      }
#pragma unroll
      for (int a = 0; a < kU; ++a) {
        if (i0 + a * T::kThreads >= n) break;
        v4f f = v[a][0];
#pragma unroll
        for (int j = 1; j < 4; ++j)
          if (j < u_splits) f = f + v[a][j];
        uint16_t h[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(f[j], h[j], o[j]);
        int k;
        uint8_t* to = place(i0 + a * T::kThreads, quads, k) + 2 * k;
        *reinterpret_cast<uint2*>(to) = make_uint2(h[0] | uint32_t(h[1]) << 16, h[2] | uint32_t(h[3]) << 16);
        *reinterpret_cast<uint2*>(to + plane) = make_uint2(o[0] | uint32_t(o[1]) << 16, o[2] | uint32_t(o[3]) << 16);
      }
    }
    for (int i = threadIdx.x; i < rows * s.slices * pads; i += T::kThreads) {
      int k;
      uint8_t* to = place(i, pads, k) + 2 * (k + 4 * quads);
      *reinterpret_cast<uint2*>(to) = *reinterpret_cast<uint2*>(to + plane) = make_uint2(0u, 0u);
    }
    __syncthreads();
    while (id[0] < s.L) {
#pragma unroll
      for (int a = 0; a < kOnce; ++a) {
        if (id[a] >= s.L) break;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
          for (int q = 0; q < kN; ++q) b[a][j][q] = keep(b[a][j][q], k0 + 32 * j + 8 * kq < s.r);
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          const int pi = p0 + 16 * i;
          if (pi < to[a] && pi + 16 > from[a]) {
            bool mine[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) mine[v] = pi + 4 * kq + v >= from[a] && pi + 4 * kq + v < to[a];
            const uint8_t* at = lds + (pi - m0 + ln) * row_bytes + 16 * kq;
#pragma unroll
            for (int q = 0; q < kN; ++q) {
              const int slice = s.slices == 2 && wrow[q] >= s.N / 2 ? 2 * plane : 0;
              v4f d = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                if (j == 1 && kc == 32) break;
                d = mfma(*reinterpret_cast<const uint4*>(at + slice + 64 * j), b[a][j][q], d);
                d = mfma(*reinterpret_cast<const uint4*>(at + slice + plane + 64 * j), b[a][j][q], d);
              }
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[i][q][v] += mine[v] ? d[v] : 0.0f;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      load_b(min(id[kOnce - 1] + 1, s.L));
    }
  };
  for (int k0 = 0; k0 < s.r; k0 += 64) {
    // (the 256 tile's accumulators leave no room for both)
    if (T::kRows == 128 || s.r - k0 > 32) pass(k0, std::integral_constant<int, 2>());
    else pass(k0, std::integral_constant<int, 1>());
  }
}

// What a launch of the tile kernel does: the whole projection; a split of K of the product, to parts
// (with the shrink); or the join of the parts, the adapters and the epilogue.
enum TileMode { kWhole, kParts, kJoin };

template <int EPI, typename T, TileMode MODE>
__global__ void __launch_bounds__(T::kThreads, 2)
lora_gemm_kernel(LoraArgs args, LoraShape s, float* __restrict__ u, v4f* __restrict__ parts, int splits,
                 ShrinkGrid sgrid) {
  static_assert(MODE != kParts || EPI == MOEQ_EPI_NONE, "parts are of W's own columns");
  static_assert(MODE == kWhole || T::kGroups == 1, "groups are for whole tiles");
  constexpr int kM = T::kM, kN = T::kN, kG = T::kGroups;       // kM x kN blocks of 16 x 16 per wave
  constexpr int BM = T::BM, BN = T::BN, kLX = T::kLX, kLW = T::kLW, kEndM = T::kEndM;
  constexpr bool kSilu = EPI == MOEQ_EPI_SILU_MUL;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4, lr = lane >> 3;
  const int group = kG == 1 ? 0 : wave / T::kGroupWaves, gw = kG == 1 ? wave : wave % T::kGroupWaves;
  const int wm = gw / T::kWN, wn = gw % T::kWN;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const int cols = kSilu ? s.N / 2 : s.N;                // output columns, a multiple of 16
  constexpr int kOut = kSilu ? BN / 2 : BN;                // output columns per workgroup
  // Workgroups go round the XCDs: each takes a run of tiles, all row tiles of a column tile before
  // the next one, so that an XCD's tiles share their w rows in its L2.
  int block = blockIdx.x, blocks = gridDim.x;
  if constexpr (MODE == kParts) {
    // (the shrink's workgroups last: ahead of the product's they kept half of those waiting for LDS)
    blocks -= sgrid.blocks();
    if (block >= blocks) {
      shrink(args, s, u, sgrid, block - blocks, reinterpret_cast<v4f (*)[4][kWave]>(lds));
      return;
    }
  }
  const int mtiles = (s.M + BM - 1) / BM;
  const int xcd = block & 7;
  int tile = xcd * (blocks >> 3) + min(xcd, blocks & 7) + (block >> 3), split = 0;
  if constexpr (MODE == kParts) {                        // the splits of a tile follow each other
    split = tile % splits;
    tile /= splits;
  }
  const int nt = tile / mtiles, mt = tile - nt * mtiles;
  const int m0 = mt * BM, n0 = nt * kOut;

  // w row of tile row i: BN columns, or BN/2 gate and their BN/2 up rows; past the end the last one
  // again (its results are not stored)
  const auto w_row = [&](int i) {
    if (kSilu) return i < BN / 2 ? min(n0 + i, cols - 1) : cols + min(n0 + i - BN / 2, cols - 1);
    return min(n0 + i, cols - 1);
  };
  // tile row of the wave's 16-column block q: gate blocks, then the matching up blocks
  const auto block_row = [&](int q) {
    return kSilu ? (q < kN / 2 ? 0 : BN / 2) + (T::kCols / 2) * wn + 16 * (q % (kN / 2))
                 : T::kCols * wn + 16 * q;
  };

  // loads: wave v of a group moves rows 8 (its loads v + g) + lr, lane's chunk (lane % 8) ^ swz(row)
  const uint16_t *xsrc[kLX], *wsrc[kLW];
#pragma unroll
  for (int g = 0; g < kLX; ++g) {
    const int row = 8 * (kLX * gw + g) + lr;
    xsrc[g] = args.a + int64_t(plan_row(pv, m0 + row, s.M)) * s.ld_a + ((lane & 7) ^ swz(row & 15)) * 8;
  }
#pragma unroll
  for (int g = 0; g < kLW; ++g) {
    const int row = 8 * (kLW * gw + g) + lr;
    wsrc[g] = args.w + int64_t(w_row(row)) * s.K + ((lane & 7) ^ swz(row & 15)) * 8;
  }
  const uint8_t* const ring = lds + group * T::kRingB;
  const uint32_t ring0 = lds_offset(ring);
  // this group's (or launch's) slots of 64 K: first, number
  const int all_slots = s.K / kSlotK;
  const int s0 = MODE == kParts ? int(int64_t(all_slots) * split / splits) : group * (all_slots / kG);
  const int slots = MODE == kParts ? int(int64_t(all_slots) * (split + 1) / splits) - s0
                                   : MODE == kJoin ? 0 : all_slots / kG;
  // load g of unit `unit` (2 st: w, 2 st + 1: x of slot st); past the last slot, the last again
  const auto issue = [&](bool is_w, int g, int unit) {
    const int k = (s0 + min(unit >> 1, slots - 1)) * kSlotK;
    const int row = 8 * ((is_w ? kLW : kLX) * gw + g);
    load_lds<false>((is_w ? wsrc[is_w ? g : 0] : xsrc[is_w ? 0 : g]) + k,
                    ring0 + uint32_t(T::place(unit % T::kUnits) + row * kRowB));
  };

  v4f acc[kM][kN];
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int q = 0; q < kN; ++q) acc[i][q] = v4f{0.f, 0.f, 0.f, 0.f};
  const int rd[2] = {ln * kRowB + ((kq ^ swz(ln)) * 16), ln * kRowB + (((4 + kq) ^ swz(ln)) * 16)};
  uint4 xa[kM], wb[2][kN];
  const auto read_x = [&](int i, const uint8_t* buf, int h) {
    xa[i] = *reinterpret_cast<const uint4*>(buf + (T::kRows * wm + 16 * i) * kRowB + rd[h]);
  };
  const auto read_w = [&](const uint8_t* buf, int h) {
#pragma unroll
    for (int q = 0; q < kN; ++q) wb[h][q] = *reinterpret_cast<const uint4*>(buf + block_row(q) * kRowB + rd[h]);
  };
  const auto multiply = [&](int i, int h) {
#pragma unroll
    for (int q = 0; q < kN; ++q) acc[i][q] = mfma(xa[i], wb[h][q], acc[i][q]);
  };
  constexpr int kOpen = kM / 4;

  if (slots > 0) {
#pragma unroll
    for (int unit = 0; unit + 1 < T::kUnits; ++unit)
#pragma unroll
      for (int g = 0; g < (unit & 1 ? kLX : kLW); ++g) issue(!(unit & 1), g, unit);
    wait_vmem<T::loads(2, T::kUnits - 1)>();
    ring_barrier();
    int px = 1, pw = 0;                                  // ring places of the slot's units
    read_w(ring, 0);
#pragma unroll
    for (int i = 0; i < kM; ++i) read_x(i, ring + T::place(1), 0);
    // unit `unit`'s loads, spread over the rows from `first` on
    const auto issue_row = [&](int i, int first, int unit, bool is_w) {
      const int n = is_w ? kLW : kLX, rows = kM - first, per = (n + rows - 1) / rows;
#pragma unroll
      for (int j = 0; j < n; ++j)
        if (i >= first && j / per == i - first) issue(is_w, j, unit);
    };
    const auto first_half = [&](int st) {
      read_w(ring + T::place(pw), 1);
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        multiply(i, 0);
        read_x(i, ring + T::place(px), 1);
        issue_row(i, 0, 2 * st + T::kUnits - 1, T::kUnits & 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int st = 0; st + 1 < slots; ++st) {
      first_half(st);
      px = px + 2 >= T::kUnits ? px + 2 - T::kUnits : px + 2;
      pw = pw + 2 >= T::kUnits ? pw + 2 - T::kUnits : pw + 2;
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        if (i == kOpen) {
          wait_vmem<T::loads(4, T::kUnits)>();
          ring_barrier();
          read_w(ring + T::place(pw), 0);
#pragma unroll
          for (int j = 0; j < kOpen; ++j) read_x(j, ring + T::place(px), 0);
        }
        multiply(i, 1);
        if (i >= kOpen) {
          read_x(i, ring + T::place(px), 0);
          issue_row(i, kOpen, 2 * st + T::kUnits, !(T::kUnits & 1));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    first_half(slots - 1);
#pragma unroll
    for (int i = 0; i < kM; ++i) multiply(i, 1);
    wait_vmem<0>();                                      // the loads past the last slot
  }
  // K past the groups' slots, zeros after its end: by the first group
  if (MODE == kWhole || (MODE == kParts && split == splits - 1)) {
#pragma unroll
    for (int rest = 0; rest < kG; ++rest) {
      const int k0 = (all_slots / kG * kG + rest) * kSlotK;
      if (k0 >= s.K) break;
      ring_barrier();
      for (int i = tid; i < (BM + BN) * 8; i += T::kThreads) {
        const int row = i >> 3, c = i & 7;
        const uint16_t* src = row < BM ? args.a + int64_t(plan_row(pv, m0 + row, s.M)) * s.ld_a
                                       : args.w + int64_t(w_row(row - BM)) * s.K;
        *reinterpret_cast<uint4*>(lds + row * kRowB + ((c ^ swz(row & 15)) * 16)) = load_k(src, k0 + 8 * c, s.K);
      }
      __syncthreads();
      if (group > 0) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        read_w(lds + BM * kRowB, h);
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          read_x(i, lds, h);
          multiply(i, h);
        }
      }
    }
  }

  // first w row of each column block, kept inside W for blocks past the last column
  int wrow[kN], ocol[kN];
#pragma unroll
  for (int q = 0; q < kN; ++q) {
    const bool up = kSilu && q >= kN / 2;
    ocol[q] = n0 + block_row(q) - (up ? BN / 2 : 0);
    wrow[q] = min(ocol[q], cols - 16) + (up ? cols : 0);
  }
  const int p0 = m0 + T::kRows * wm + 16 * kEndM * group;
  if constexpr (MODE != kWhole) {                        // blocks [split][16 rows][16 w rows][lane]
    const int mblocks = (s.M + 15) / 16, nb = s.N / 16;
    const int64_t stride = int64_t(mblocks) * nb * kWave;
    const auto part = [&](int i, int q) {
      return parts + (int64_t(min(p0 / 16 + i, mblocks - 1)) * nb + wrow[q] / 16) * kWave + lane;
    };
    if constexpr (MODE == kParts) {
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int q = 0; q < kN; ++q)
          if (p0 / 16 + i < mblocks && ocol[q] < cols) part(i, q)[split * stride] = acc[i][q];
    } else {
      v4f v[kMaxSplits][kM][kN];                         // all loads at once
#pragma unroll
      for (int j = 0; j < kMaxSplits; ++j)
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
          for (int q = 0; q < kN; ++q)
            if (j < splits) v[j][i][q] = part(i, q)[j * stride];
#pragma unroll
      for (int j = 0; j < kMaxSplits; ++j)
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
          for (int q = 0; q < kN; ++q)
            if (j < splits) acc[i][q] = acc[i][q] + v[j][i][q];
    }
    if constexpr (MODE == kParts) return;
  }
  ring_barrier();                                        // the ring's LDS is free
  constexpr int kMeet = kG == 1 ? 0 : BM * BN * 4;       // LDS of the groups' exchange: half of either's sums
  if constexpr (kG > 1) {
    // group g finishes row blocks g kEndM ...: it leaves its sums of the others to their group
    static_assert(kG == 2, "one other group");
    v4f* const meet = reinterpret_cast<v4f*>(lds) + lane;
#pragma unroll
    for (int i = 0; i < kEndM; ++i)
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        meet[((wave * kEndM + i) * kN + q) * kWave] = group ? acc[i][q] : acc[kEndM + i][q];
        acc[i][q] = group ? acc[kEndM + i][q] : acc[i][q];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEndM; ++i)
#pragma unroll
      for (int q = 0; q < kN; ++q)
        acc[i][q] = acc[i][q] + meet[(((wave ^ T::kGroupWaves) * kEndM + i) * kN + q) * kWave];
  }
  add_adapters<T>(acc, pv, args, s, u, sgrid.splits, lds + kMeet, m0, p0, wrow, lane);
#pragma unroll
  for (int i = 0; i < kEndM; ++i) {
    // (a row block at a time: the rows' places hoisted together would take the accumulators' registers)
    __builtin_amdgcn_sched_barrier(0);
    const int p = p0 + 16 * i + 4 * kq + (ln & 3);
    uint16_t* o = args.out + int64_t(plan_row(pv, p, s.M)) * cols + (ln & 12);
#pragma unroll
    for (int q = 0; q < (kSilu ? kN / 2 : kN); ++q) {
      float f[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        f[v] = kSilu ? silu_f32(acc[i][q][v]) * acc[i][q + (kSilu ? kN / 2 : 0)][v] : acc[i][q][v];
      const uint2 four = quad_rows(f, lane);
      if (p < s.M && ocol[q] < cols) *reinterpret_cast<uint2*>(o + ocol[q]) = four;
    }
  }
}

// ------------------------------------------------------------------ few rows
// Up to 64 rows: bound by the stream of W.  One launch multiplies (64 w rows x all rows x a
// range of K per workgroup, fp32 parts to the workspace) and, in its first workgroups, forms
// u's parts, which do not depend on the product; a second one adds the parts and the adapters,
// and applies the epilogue.
//
// Parts are stored as the matrix instruction leaves them: 16 bytes per lane, 1 KB per block.

// u parts: a wave takes 16 rows of one adapter x 16 columns x a piece of 512 K (several, if there
// are more than 16)
constexpr int kUSteps = kUPiece / 32;

// the plan's tiles by lane: all of them (at most 64 of up to 64 rows), or those from sorted row p0's on
struct FewPlan {
  int n, row0, expert;
  __device__ __forceinline__ FewPlan(const PlanView& pv, int lane) {
    n = min(min(pv.base[kPlanTiles], pv.max_tiles), kWave);
    row0 = pv.tile_row0[min(lane, pv.max_tiles - 1)];
    expert = pv.tile_expert[min(lane, pv.max_tiles - 1)];
  }
  __device__ __forceinline__ FewPlan(const PlanView& pv, int p0, int lane) {
    const int tiles = min(pv.base[kPlanTiles], pv.max_tiles);
    constexpr int kAhead = 5;                            // the tiles of 256 rows at once
    int before = 0;                                      // tiles that begin at or before p0
    for (int t0 = 0; t0 < tiles; t0 += kAhead * kWave) {
      int first[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) first[i] = pv.tile_row0[min(t0 + i * kWave + lane, pv.max_tiles - 1)];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        before += __popcll(__ballot(t0 + i * kWave + lane < tiles && first[i] <= p0));
    }
    const int t = max(before - 1, 0);
    n = min(tiles - t, kWave);
    row0 = pv.tile_row0[min(t + lane, pv.max_tiles - 1)];
    expert = pv.tile_expert[min(t + lane, pv.max_tiles - 1)];
  }
  // adapter of sorted row p0 + lane, lane < 16 (the tile that holds it; -1: none)
  __device__ __forceinline__ int adapter16(int p0, int lane) const {
    const int base = __popcll(__ballot(lane < n && row0 <= p0)) - 1;
    const int at = row0 - p0;
    const uint32_t bit = lane < n && at > 0 && at < 16 ? 1u << at : 0u;
    const uint32_t starts = uint32_t(wave_reduce(int(bit), [](int a, int b) { return a | b; }, 0));
    const int t = base + __popc(starts & ((2u << (lane & 15)) - 1u));
    const int e = __shfl(expert, max(t, 0));
    return t >= 0 ? e : -1;
  }
};

// One wave: scale * x A_l^T over pieces c0 .. c1 - 1 of K, for 16-row piece `b` of the adapters'
// rows and columns 16 cb .. + 15, into u [M][columns].  All loads of a piece go out at once: this
// is a chain of memory latencies next to the stream of W, so it has to be short.
__device__ __forceinline__ void few_shrink(const LoraArgs& args, const LoraShape& s, float* u, int b,
                                           int cb, int c0, int c1, int lane) {
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
  const uint16_t* arow = args.lora_a + (int64_t(l) * cols + min(16 * cb + ln, cols - 1)) * s.K;
  const uint16_t* x = args.a + int64_t(plan_row(pv, min(p0 + ln, p1 - 1), s.M)) * s.ld_a;
  const float scale = args.scale[l];
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; ++c) {
    uint4 av[kUSteps], xv[kUSteps];
#pragma unroll
    for (int j = 0; j < kUSteps; ++j) av[j] = load_in(arow, c * kUPiece + 32 * j + 8 * kq, s.K);
#pragma unroll
    for (int j = 0; j < kUSteps; ++j) xv[j] = load_in(x, c * kUPiece + 32 * j + 8 * kq, s.K);
    __builtin_amdgcn_sched_barrier(0);                   // all of them in flight
#pragma unroll
    for (int j = 0; j < kUSteps; ++j) {
      const bool in = c * kUPiece + 32 * j + 8 * kq < s.K;
      acc = mfma(keep(xv[j], in), keep(av[j], in), acc);
    }
  }
  const int col = 16 * cb + ln;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int p = p0 + 4 * kq + v;
    if (col < cols && p < p1) u[int64_t(p) * cols + col] = acc[v] * scale;
  }
}

template <int MB>
constexpr int few_slot_bytes() { return (kFewCols + 16 * MB) * kRowB; }
// slots of the ring: what three workgroups of a CU can have in its 160 KB
template <int MB>
constexpr int few_ring() { return 160 * 1024 / 3 / few_slot_bytes<MB>(); }

// The product.  Both operands reach LDS by loads that write LDS directly, whole 128-byte lines, no
// staging registers, a ring of slots of 64 K deep in flight.  A wave loads the 16 w rows whose
// columns it computes and its share of the x rows.
template <int MB>
__global__ void __launch_bounds__(256, 3)
lora_few_kernel(LoraArgs args, LoraShape s, float* __restrict__ u, v4f* __restrict__ parts,
                int shrink_items, int u_cols, int u_splits, int u_per_split, int slots_per_split) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int shrink_blocks = (shrink_items + 3) / 4;
  if (int(blockIdx.x) < shrink_blocks) {
    const int item = blockIdx.x * 4 + wave;              // (row piece, K split, 16 columns)
    if (item >= shrink_items) return;
    const int cb = item % u_cols, rest = item / u_cols;
    const int sp = rest % u_splits, pieces = (s.K + kUPiece - 1) / kUPiece;
    few_shrink(args, s, u + int64_t(sp) * s.M * s.slices * s.r, rest / u_splits, cb, sp * u_per_split,
               min((sp + 1) * u_per_split, pieces), lane);
    return;
  }
  constexpr int kSlots = few_ring<MB>(), kSlotB = few_slot_bytes<MB>();
  constexpr int kXLoads = MB == 4 ? 2 : 1;               // x: 16 MB rows over four waves
  constexpr int kXRows = 4 * MB;                         // x rows per wave
  constexpr int kLoads = 2 + kXLoads;
  const int ln = lane & 15, kq = lane >> 4;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const int ntiles = (s.N + kFewCols - 1) / kFewCols, all_slots = s.K / kSlotK;
  const int b = blockIdx.x - shrink_blocks, splits = (gridDim.x - shrink_blocks) / ntiles;
  // (neighbouring workgroups take neighbouring ranges of the same rows)
  const int nt = b / splits, split = b - nt * splits;
  const int n0 = nt * kFewCols + 16 * wave;
  const int s0 = split * slots_per_split, n_slots = min(slots_per_split, all_slots - s0);

  const int lr = lane >> 3;
  const uint16_t* wsrc[2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
    wsrc[g] = args.w + int64_t(min(n0 + 8 * g + lr, s.N - 1)) * s.K + s0 * kSlotK +
              (((lane & 7) ^ swz(8 * g + lr)) * 8);
  const uint16_t* xsrc[kXLoads];
#pragma unroll
  for (int g = 0; g < kXLoads; ++g) {
    // (the rows are read at wave-uniform addresses, through the scalar cache: a vector load's result
    // could only be waited for together with the w loads issued before it is needed)
    const int first = kXRows * wave + 8 * g;
    int row = 0;
#pragma unroll
    for (int i = 0; i < (MB == 1 ? 4 : 8); ++i) {
      const int at = plan_row(pv, first + i, s.M);
      row = lr == i ? at : row;
    }
    xsrc[g] = args.a + int64_t(row) * s.ld_a + s0 * kSlotK + (((lane & 7) ^ swz((first + lr) & 15)) * 8);
  }
  // slot st of this range; past the last one, the last again (into a buffer that is not read)
  const uint32_t lds0 = lds_offset(lds);
  auto issue = [&](int st) {
    const uint32_t buf = lds0 + (st % kSlots) * kSlotB;
    const int k = min(st, n_slots - 1) * kSlotK;
#pragma unroll
    for (int g = 0; g < 2; ++g) load_lds<true>(wsrc[g] + k, buf + (16 * wave + 8 * g) * kRowB);
#pragma unroll
    for (int g = 0; g < kXLoads; ++g)
      if (MB > 1 || lane < 32)
        load_lds<false>(xsrc[g] + k, buf + (kFewCols + kXRows * wave + 8 * g) * kRowB);
  };
  v4f acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int rd[2] = {ln * kRowB + ((kq ^ swz(ln)) * 16), ln * kRowB + (((4 + kq) ^ swz(ln)) * 16)};
  auto multiply = [&](const uint8_t* buf) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 wv = *reinterpret_cast<const uint4*>(buf + 16 * wave * kRowB + rd[h]);
#pragma unroll
      for (int i = 0; i < MB; ++i)
        acc[i] = mfma(*reinterpret_cast<const uint4*>(buf + (kFewCols + 16 * i) * kRowB + rd[h]), wv, acc[i]);
    }
  };
  if (n_slots > 0) {
#pragma unroll
    for (int st = 0; st < kSlots; ++st) issue(st);
    wait_vmem<(kSlots - 1) * kLoads>();
    ring_barrier();
    for (int st = 0; st < n_slots; ++st) {
      multiply(lds + (st % kSlots) * kSlotB);
      if (st + 1 == n_slots) break;
      wait_vmem<(kSlots - 2) * kLoads>();                // this wave's loads of slot st + 1 have landed
      ring_barrier();                                    // ... every wave's, and slot st is read
      issue(st + kSlots);
    }
    wait_vmem<0>();
  }
  const int tail = s.K - all_slots * kSlotK;          // K past whole slots, zeros after it
  if (tail > 0 && split == splits - 1) {
    ring_barrier();
    const int k0 = all_slots * kSlotK;
    for (int i = tid; i < (kFewCols + 16 * MB) * 8; i += 256) {
      const int row = i >> 3, c = i & 7;
      const uint16_t* src = row < kFewCols
          ? args.w + int64_t(min(nt * kFewCols + row, s.N - 1)) * s.K
          : args.a + int64_t(plan_row(pv, row - kFewCols, s.M)) * s.ld_a;
      *reinterpret_cast<uint4*>(lds + row * kRowB + ((c ^ swz(row & 15)) * 16)) = load_k(src, k0 + 8 * c, s.K);
    }
    __syncthreads();
    multiply(lds);
  }
  if (n0 >= s.N) return;
  const int nb = s.N / 16, mblocks = (s.M + 15) / 16;
#pragma unroll
  for (int i = 0; i < MB; ++i)
    if (i < mblocks) parts[((int64_t(split) * mblocks + i) * nb + n0 / 16) * kWave + lane] = acc[i];
}

// at[0] + at[stride] + ... (n of them, in this order), kAhead loads at a time; the first ones go out in
// load(), well ahead of sum()
template <int kAhead>
struct PartSum {
  v4f v[kAhead];
  __device__ __forceinline__ void load(const v4f* at, int64_t stride, int i0, int n) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i] = at[min(i0 + i, n - 1) * stride];
  }
  __device__ __forceinline__ v4f sum(const v4f* at, int64_t stride, int n) {
    v4f acc = v[0];
#pragma unroll
    for (int i = 1; i < kAhead; ++i)
      if (i < n) acc = acc + v[i];
    for (int i0 = kAhead; i0 < n; i0 += kAhead) {
      load(at, stride, i0, n);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < n) acc = acc + v[i];
    }
    return acc;
  }
};

// bytes of LDS for u of 16 rows in two bf16 parts, each slice padded to whole steps of 32
__host__ __device__ inline int join_u_row(int slices, int r) { return slices * ((r + 31) / 32 * 32) * 4 + 16; }

// parts and adapters joined: a workgroup forms 16 rows x 16 output columns (of the gate and the up
// half with SILU_MUL).  For each adapter among the 16 rows, its B rows of these columns times all
// 16 rows' u, kept for the adapter's own rows: each B value is read once, in half lines that the
// two steps of a pair complete.  (A lane that read the B rows of its own column for its four rows,
// and summed without the matrix instruction, used 16 bytes of each line at a time and read lines
// over: 11.7 us for 64 rows of rank 64 x 4096 columns.)  This launch is latency: everything but B
// is loaded at once, B as soon as the rows' adapters are known, and the adapters, up to 16, are
// dealt over the four waves, so that none loads twice (four columns' worth per workgroup and all
// adapters in each wave: 9.3 us instead of 4.8 for 16 rows x 8192).  So are the parts, which keeps
// registers at four workgroups a CU up to rank 32: 64 rows of gate/up 8192 are then one go (the call
// 27.5 us; all parts in the first wave, two workgroups a CU, 30.3).
template <int EPI, bool kFew, int kSteps>                // kSteps: steps of 32 ranks at a time
__global__ void __launch_bounds__(256, kSteps == 1 ? 4 : 3)
lora_join_kernel(LoraArgs args, LoraShape s, const float* __restrict__ u,
                 const v4f* __restrict__ parts, int splits, int u_splits) {
  extern __shared__ __align__(16) uint8_t us[];          // u: [16 rows][slice][hi, lo][r to 32]
  __shared__ v4f red[3][2][kWave];
  constexpr bool kSilu = EPI == MOEQ_EPI_SILU_MUL;
  constexpr int kHalves = kSilu ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const int cols = kSilu ? s.N / 2 : s.N;
  const int cblocks = cols / 16, mblocks = (s.M + 15) / 16, nb = s.N / 16;
  const int mb = blockIdx.y, cb = blockIdx.x;
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  const FewPlan fp = kFew ? FewPlan(pv, lane) : FewPlan(pv, 16 * mb, lane);
  const int rows = min(16, s.M - 16 * mb);
  const int64_t part_stride = int64_t(mblocks) * nb * kWave, u_stride = int64_t(s.M) * s.slices * s.r / 4;
  const v4f* pat[kHalves];
  // the product's parts are dealt over the waves too: up to 8 of up to 64 rows, else up to 4
  PartSum<kFew ? 2 : 1> ps[kHalves];
  const int n_parts = (splits - wave + 3) / 4;
  PartSum<kFew ? 8 : kMaxSplits> pu;
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    pat[h] = parts + wave * part_stride + (int64_t(mb) * nb + cb + h * cblocks) * kWave + lane;
    if (n_parts > 0) ps[h].load(pat[h], 4 * part_stride, 0, n_parts);
  }
  // u's elements, four at a time: thread i takes quads i, i + 256, ... of [row][slice][r to 32]
  const int r32 = (s.r + 31) / 32 * 32, quads = s.slices * (r32 / 4), row_bytes = join_u_row(s.slices, s.r);
  const auto u_quad = [&](int i, int& row, int& slice, int& k) {
    row = i / quads;
    const int c = i - row * quads;
    slice = c / (r32 / 4);
    k = 4 * (c - slice * (r32 / 4));
    return reinterpret_cast<const v4f*>(
        u + (int64_t(16 * mb + min(row, rows - 1)) * s.slices + slice) * s.r + min(k, s.r - 4));
  };
  int urow, uslice, uk;
  const v4f* uat = u_quad(min(tid, 16 * quads - 1), urow, uslice, uk);
  pu.load(uat, u_stride, 0, u_splits);
  const int out_row = plan_row(pv, 16 * mb + 4 * kq + (ln & 3), s.M);

  // lane i < 16: the adapter of row 16 mb + i (-1: none).  Rows are sorted by adapter, so each
  // adapter's rows follow its first one.
  int adapter = fp.adapter16(16 * mb, lane);
  if (lane >= rows || adapter >= s.L || adapter < 0) adapter = -1;
  const uint32_t with = uint32_t(__ballot(adapter >= 0));
  const int before = __shfl_up(adapter, 1);
  uint32_t firsts = uint32_t(__ballot(adapter >= 0 && (lane == 0 || before != adapter)));
  // first w row of the block's halves, and their slice of u
  int wrow[kHalves], slice[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    wrow[h] = (cb + h * cblocks) * 16;
    slice[h] = s.slices == 2 && wrow[h] >= s.N / 2;
  }
  constexpr int kMine = 4;                               // adapters of a wave
  uint32_t of[kMine];                                    // their rows, one bit each
  int id[kMine], n_mine = 0;
  for (int i = 0; i < wave; ++i) firsts &= firsts - 1;
#pragma unroll
  for (int a = 0; a < kMine; ++a) {                      // every fourth of the list
    const int i = firsts ? __ffs(firsts) - 1 : 0;
    const uint32_t rest = firsts & (firsts - 1);
    // the bits from this first row up to the next one
    of[a] = firsts ? with & (~0u << i) & (rest ? (rest & -rest) - 1 : ~0u) : 0u;
    id[a] = max(readlane(adapter, i), 0);
    n_mine += firsts != 0;
    firsts = rest;
    for (int j = 0; j < 3; ++j) firsts &= firsts - 1;
  }
  uint4 b[kMine][kSteps][kHalves];
  auto load_b = [&](int k0) {
#pragma unroll
    for (int a = 0; a < kMine; ++a)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint16_t* at = args.lora_b + (int64_t(id[a]) * s.N + wrow[h] + ln) * s.r;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) b[a][j][h] = load16(at + min(k0 + 32 * j + 8 * kq, s.r - 8));
      }
  };
  if (n_mine > 0) load_b(0);
  v4f acc[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
    acc[h] = n_parts > 0 ? ps[h].sum(pat[h], 4 * part_stride, n_parts) : v4f{0.f, 0.f, 0.f, 0.f};
  for (int i = tid; i < 16 * quads; i += 256) {
    if (i >= 256) {
      uat = u_quad(i, urow, uslice, uk);
      pu.load(uat, u_stride, 0, u_splits);
    }
    const v4f f = pu.sum(uat, u_stride, u_splits);
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(uk < s.r ? f[j] : 0.0f, hi[j], lo[j]);
    uint8_t* to = us + urow * row_bytes + (uslice * 2 * r32 + uk) * 2;
    *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | uint32_t(hi[1]) << 16, hi[2] | uint32_t(hi[3]) << 16);
    *reinterpret_cast<uint2*>(to + 2 * r32) =
        make_uint2(lo[0] | uint32_t(lo[1]) << 16, lo[2] | uint32_t(lo[3]) << 16);
  }
  __syncthreads();                                       // u is in LDS
  for (int k0 = 0; n_mine > 0 && k0 < s.r; k0 += 32 * kSteps) {
    uint4 hi[kSteps][kHalves], lo[kSteps][kHalves];
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int k = min(k0 + 32 * j, r32 - 32) + 8 * kq;   // (a step past r is not used)
        const uint8_t* at = us + ln * row_bytes + (slice[h] * 2 * r32 + k) * 2;
        hi[j][h] = *reinterpret_cast<const uint4*>(at);
        lo[j][h] = *reinterpret_cast<const uint4*>(at + 2 * r32);
      }
    if (k0 > 0) load_b(k0);
#pragma unroll
    for (int a = 0; a < kMine; ++a)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const bool in = k0 + 32 * j + 8 * kq < s.r;
          const uint4 w = b[a][j][h];
          const uint4 bv = make_uint4(in ? w.x : 0u, in ? w.y : 0u, in ? w.z : 0u, in ? w.w : 0u);
          if (j == 0 || k0 + 32 < s.r) {
            d = mfma(hi[j][h], bv, d);
            d = mfma(lo[j][h], bv, d);
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[h][v] += of[a] >> (4 * kq + v) & 1 ? d[v] : 0.0f;
      }
  }
  if (wave > 0) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) red[wave - 1][h][lane] = acc[h];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
    acc[h] = acc[h] + (red[0][h][lane] + (red[1][h][lane] + red[2][h][lane]));
  float f[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) f[v] = kSilu ? silu_f32(acc[0][v]) * acc[kHalves - 1][v] : acc[0][v];
  const uint2 four = quad_rows(f, lane);
  if (4 * kq + (ln & 3) < rows)
    *reinterpret_cast<uint2*>(args.out + int64_t(out_row) * cols + cb * 16 + (ln & 12)) = four;
}

// ------------------------------------------------------------------ short K
// Everything in one launch: a workgroup forms 16 rows x 64 output columns, a wave 16 of them (of the gate
// and the up half with SILU_MUL) over all of K, whose operands go out at once.  u of the 16 rows is formed
// by every workgroup that needs it, the adapters' pieces of 16 ranks dealt over its waves.
template <int EPI>
__global__ void __launch_bounds__(256)
lora_short_kernel(LoraArgs args, LoraShape s) {
  extern __shared__ __align__(16) uint8_t us[];          // u as in lora_join_kernel
  constexpr bool kSilu = EPI == MOEQ_EPI_SILU_MUL;
  constexpr int kHalves = kSilu ? 2 : 1, KS = kShortK / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kq = lane >> 4;
  const int cols = kSilu ? s.N / 2 : s.N;
  const int n0 = 64 * blockIdx.x + 16 * wave, p0 = 16 * blockIdx.y, rows = min(16, s.M - p0);
  const PlanView pv = plan_view(args.plan, s.L + 1, s.M);
  int wrow[kHalves], slice[kHalves];
  uint4 wv[kHalves][KS];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    wrow[h] = min(n0, cols - 16) + h * cols;
    slice[h] = s.slices == 2 && wrow[h] >= s.N / 2;
    const uint16_t* w = args.w + int64_t(wrow[h] + ln) * s.K;
#pragma unroll
    for (int j = 0; j < KS; ++j) wv[h][j] = load_in(w, 32 * j + 8 * kq, s.K);
  }
  const uint16_t* x = args.a + int64_t(plan_row(pv, p0 + ln, s.M)) * s.ld_a;
  // lane i < 16: the adapter of row p0 + i (-1: none), the groups that end at or before it
  int adapter = 0;
  for (int a0 = 0; a0 < s.L; a0 += kWave) {
    const int end = pv.offsets[min(a0 + lane + 1, s.L)];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = __popcll(__ballot(a0 + lane < s.L && end <= p0 + i));
      adapter += lane == i ? n : 0;
    }
  }
  if (lane >= rows || adapter >= s.L) adapter = -1;
  uint4 xv[KS];
#pragma unroll
  for (int j = 0; j < KS; ++j) xv[j] = load_in(x, 32 * j + 8 * kq, s.K);
#pragma unroll
  for (int j = 0; j < KS; ++j) xv[j] = keep(xv[j], 32 * j + 8 * kq < s.K);
  // rows are sorted by adapter: those of one follow its first, up to the next first
  const uint32_t with = uint32_t(__ballot(adapter >= 0));
  const int before = __shfl_up(adapter, 1);
  const uint32_t firsts = uint32_t(__ballot(adapter >= 0 && (lane == 0 || before != adapter)));
  const auto rows_of = [&](uint32_t left) {              // ... of the lowest bit of `left`
    const uint32_t rest = left & (left - 1);
    return with & ~((left & -left) - 1) & (rest ? (rest & -rest) - 1 : ~0u);
  };
  const int r32 = (s.r + 31) / 32 * 32, row_bytes = join_u_row(s.slices, s.r), ucols = s.slices * s.r;
  for (int i = tid; i < 16 * s.slices * (r32 - s.r); i += 256) {         // ranks past r
    const int at = i / (r32 - s.r), row = s.slices == 2 ? at >> 1 : at, k = s.r + i - at * (r32 - s.r);
    uint8_t* to = us + row * row_bytes + ((s.slices == 2 ? at & 1 : 0) * 2 * r32 + k) * 2;
    *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<uint16_t*>(to + 2 * r32) = 0;
  }
  const int blocks = (ucols + 15) / 16;
  int at = 0;
  for (uint32_t left = firsts; left; left &= left - 1) {
    const int l = readlane(adapter, __ffs(left) - 1);
    const uint32_t mine = rows_of(left);
    for (int cb = 0; cb < blocks; ++cb, ++at) {
      if ((at & 3) != wave) continue;
      const int col = 16 * cb + ln;
      const uint16_t* arow = args.lora_a + (int64_t(l) * ucols + min(col, ucols - 1)) * s.K;
      uint4 av[KS];
#pragma unroll
      for (int j = 0; j < KS; ++j) av[j] = load_in(arow, 32 * j + 8 * kq, s.K);
      const float scale = args.scale[l];
      v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KS; ++j)
        if (32 * j < s.K) d = mfma(xv[j], keep(av[j], 32 * j + 8 * kq < s.K), d);
      const int sl = col >= s.r ? 1 : 0;
      uint8_t* to = us + (sl * 2 * r32 + col - sl * s.r) * 2;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (col < ucols && mine >> (4 * kq + v) & 1) {
          uint16_t hi, lo;
          split2(d[v] * scale, hi, lo);
          *reinterpret_cast<uint16_t*>(to + (4 * kq + v) * row_bytes) = hi;
          *reinterpret_cast<uint16_t*>(to + (4 * kq + v) * row_bytes + 2 * r32) = lo;
        }
    }
  }
  v4f acc[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    acc[h] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (32 * j < s.K) acc[h] = mfma(xv[j], keep(wv[h][j], 32 * j + 8 * kq < s.K), acc[h]);
  }
  __syncthreads();                                       // u is in LDS
  if (n0 >= cols) return;
  for (uint32_t left = firsts; left;) {                  // four adapters' B at a time
    constexpr int kOnce = 4;
    uint32_t of[kOnce];
    int id[kOnce];
#pragma unroll
    for (int a = 0; a < kOnce; ++a) {
      of[a] = left ? rows_of(left) : 0u;
      id[a] = left ? readlane(adapter, __ffs(left) - 1) : 0;
      left &= left - 1;
    }
    for (int k0 = 0; k0 < s.r; k0 += 32) {
      uint4 b[kOnce][kHalves];
#pragma unroll
      for (int a = 0; a < kOnce; ++a)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          b[a][h] = load_in(args.lora_b + (int64_t(id[a]) * s.N + wrow[h] + ln) * s.r, k0 + 8 * kq, s.r);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint8_t* from = us + ln * row_bytes + (slice[h] * 2 * r32 + k0 + 8 * kq) * 2;
        const uint4 hi = *reinterpret_cast<const uint4*>(from), lo = *reinterpret_cast<const uint4*>(from + 2 * r32);
#pragma unroll
        for (int a = 0; a < kOnce; ++a) {
          if (of[a] == 0) continue;
          const uint4 bv = keep(b[a][h], k0 + 8 * kq < s.r);
          v4f d = mfma(hi, bv, v4f{0.f, 0.f, 0.f, 0.f});
          d = mfma(lo, bv, d);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[h][v] += of[a] >> (4 * kq + v) & 1 ? d[v] : 0.0f;
        }
      }
    }
  }
  float f[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) f[v] = kSilu ? silu_f32(acc[0][v]) * acc[kHalves - 1][v] : acc[0][v];
  const uint2 four = quad_rows(f, lane);
  const int p = 4 * kq + (ln & 3);
  if (p < rows)
    *reinterpret_cast<uint2*>(args.out + int64_t(plan_row(pv, p0 + p, s.M)) * cols + n0 + (ln & 12)) = four;
}

hipError_t launch_short(const LoraArgs& args, const LoraShape& s, hipStream_t stream) {
  const bool silu = s.epilogue == MOEQ_EPI_SILU_MUL;
  const int cols = silu ? s.N / 2 : s.N;
  const auto fn = silu ? lora_short_kernel<MOEQ_EPI_SILU_MUL> : lora_short_kernel<MOEQ_EPI_NONE>;
  hipLaunchKernelGGL(fn, dim3(unsigned((cols + 63) / 64), unsigned((s.M + 15) / 16)), dim3(256),
                     unsigned(16 * join_u_row(s.slices, s.r)), stream, args, s);
  return hipGetLastError();
}

template <bool kFew>
hipError_t launch_join(const LoraArgs& args, const LoraShape& s, const float* u, const v4f* parts, int splits,
                       int u_splits, hipStream_t stream) {
  const bool silu = s.epilogue == MOEQ_EPI_SILU_MUL;
  const int cblocks = (silu ? s.N / 2 : s.N) / 16;
  const auto join = s.r <= 32 ? (silu ? lora_join_kernel<MOEQ_EPI_SILU_MUL, kFew, 1> : lora_join_kernel<MOEQ_EPI_NONE, kFew, 1>)
                              : (silu ? lora_join_kernel<MOEQ_EPI_SILU_MUL, kFew, 2> : lora_join_kernel<MOEQ_EPI_NONE, kFew, 2>);
  hipLaunchKernelGGL(join, dim3(unsigned(cblocks), unsigned((s.M + 15) / 16)), dim3(256),
                     unsigned(16 * join_u_row(s.slices, s.r)), stream, args, s, u, parts, splits, u_splits);
  return hipGetLastError();
}

template <int MB>
hipError_t launch_few(const LoraArgs& args, const LoraShape& s, const LoraPath& path, float* u, v4f* parts,
                      hipStream_t stream) {
  const int reached = s.L < s.M ? s.L : s.M;             // adapters that have rows, at most
  const int row_pieces = reached + s.M / 16 < s.M ? reached + s.M / 16 : s.M;
  const int u_cols = (s.slices * s.r + 15) / 16, items = row_pieces * u_cols * path.u_splits;
  const int ntiles = (s.N + kFewCols - 1) / kFewCols;
  const unsigned lds = few_ring<MB>() * few_slot_bytes<MB>();
  static_assert(few_ring<MB>() * few_slot_bytes<MB>() <= 64 * 1024, "no attribute needed");
  hipLaunchKernelGGL(lora_few_kernel<MB>, dim3(unsigned((items + 3) / 4 + ntiles * path.splits)), dim3(256),
                     lds, stream, args, s, u, parts, items, u_cols, path.u_splits, path.u_pieces, path.slots);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  return launch_join<true>(args, s, u, parts, path.splits, path.u_splits, stream);
}

ShrinkGrid shrink_grid(const LoraShape& s, const LoraPath& path) {
  return {plan_max_tiles(s.L + 1, s.M) * (MOEQ_TILE_M / kShrinkRows),
          (s.slices * s.r + kShrinkCols - 1) / kShrinkCols, path.u_splits};
}

template <int EPI, typename T, TileMode MODE>
hipError_t launch_tile_kernel(const LoraArgs& args, const LoraShape& s, const LoraPath& path, float* u,
                              v4f* parts, hipStream_t stream) {
  const auto fn = lora_gemm_kernel<EPI, T, MODE>;
  const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
  if (err != hipSuccess) return err;
  const ShrinkGrid sgrid = shrink_grid(s, path);
  const int64_t tiles = tiles_of(s, T::BM, T::BN),
                blocks = MODE == kParts ? sgrid.blocks() + tiles * path.splits : tiles;
  hipLaunchKernelGGL(fn, dim3(unsigned(blocks)), dim3(T::kThreads), T::kLds, stream, args, s, u, parts,
                     path.splits, sgrid);
  return hipGetLastError();
}
template <typename T, TileMode MODE>
hipError_t launch_tiles(const LoraArgs& args, const LoraShape& s, const LoraPath& path, float* u, v4f* parts,
                        hipStream_t stream) {
  return s.epilogue == MOEQ_EPI_SILU_MUL
             ? launch_tile_kernel<MOEQ_EPI_SILU_MUL, T, MODE>(args, s, path, u, parts, stream)
             : launch_tile_kernel<MOEQ_EPI_NONE, T, MODE>(args, s, path, u, parts, stream);
}

}  // namespace

hipError_t launch_shared_gemm_lora(const LoraArgs& args, const LoraShape& s, hipStream_t stream) {
  if (s.M == 0) return hipSuccess;
  const LoraPath path = lora_path(s);
  if (path.one_launch) return launch_short(args, s, stream);
  float* u = static_cast<float*>(args.ws);
  v4f* parts = reinterpret_cast<v4f*>(static_cast<uint8_t*>(args.ws) + path.u_bytes);
  if (path.few) {
    static_assert(kFewRows <= 64, "four blocks of 16 rows");
    return s.M <= 16 ? launch_few<1>(args, s, path, u, parts, stream)
                     : s.M <= 32 ? launch_few<2>(args, s, path, u, parts, stream)
                                 : launch_few<4>(args, s, path, u, parts, stream);
  }
  hipError_t err;
  if (path.splits > 1) {
    err = path.bm == 128
              ? launch_tile_kernel<MOEQ_EPI_NONE, Tile<128, 128, 1>, kParts>(args, s, path, u, parts, stream)
              : launch_tile_kernel<MOEQ_EPI_NONE, Tile<64, 64, 1>, kParts>(args, s, path, u, parts, stream);
    if (err != hipSuccess) return err;
    return path.join_rows ? launch_join<false>(args, s, u, parts, path.splits, path.u_splits, stream)
                          : launch_tiles<Tile<64, 64, 1>, kJoin>(args, s, path, u, parts, stream);
  }
  const ShrinkGrid sgrid = shrink_grid(s, path);
  hipLaunchKernelGGL(lora_shrink_kernel, dim3(unsigned(sgrid.blocks())), dim3(256), 0, stream, args, s, u,
                     sgrid);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  if (path.bn == 256) return launch_tiles<Tile<256, 256, 1>, kWhole>(args, s, path, u, parts, stream);
  if (path.bm == 256) return launch_tiles<Tile<256, 128, 1>, kWhole>(args, s, path, u, parts, stream);
  if (path.bm == 64) return launch_tiles<Tile<64, 64, 1>, kWhole>(args, s, path, u, parts, stream);
  if (path.groups == 2) return launch_tiles<Tile<128, 128, 2>, kWhole>(args, s, path, u, parts, stream);
  return launch_tiles<Tile<128, 128, 1>, kWhole>(args, s, path, u, parts, stream);
}

}  // namespace moeq
