// A whole MoE layer for at most 16 tokens in two kernels, with MXFP4 expert
// weights and bf16 activations (weight-only quantization: a few tokens are bound
// by the weight stream, so 16-bit activations cost nothing and spare the layer
// their rounding to 4 bits):
//   few_gate_up_kernel  s = logits + bias, top-k, weights;  h = silu(Wg x) * (Wu x)
//   few_down_kernel     o_j = W2 h_j;  y = sum_j w_j o_j (+ shared)
//
// Sums: W = e2m1 * 2^s converts exactly to bf16 (2 significant bits), products
// and sums run in fp32 on v_mfma_f32_16x16x32_bf16.  h enters the second product as
// the sum of three bf16 values, 8 of fp32's 24 significant bits each, so nothing of
// it is rounded away (split_bf16): the matrix units have the time, and the weights
// are converted once for all three.  o stays fp32; y is rounded once.  (Two values,
// 16 bits, took 0.2 us less at one token and 0.4 at four, and cost y a bf16 step in
// one element of some hundreds.)
//
// Work units.  A workgroup belongs to one routed row r = t k + j and a run of
// column units.  In the gate/up kernel it finds its row's expert and the other
// tokens' rows of that expert from the scores themselves (4 T E bytes, from L2), so
// no launch is spent on routing; in the down kernel from the ids the first wrote.
// The lowest row of an expert owns it and computes all of them (at most one per
// token, so at most 16: one 16-column MFMA block); the other rows' workgroups leave
// at once.  No plan is built or read.
//
// Joining the experts' outputs without a third launch: the down kernel's
// workgroups store their fp32 o columns past the caches, then count up one
// arrival counter per column unit; the one that arrives last has all T k rows of
// its 32 columns and forms y in slot order j, so results do not depend on the
// arrival order.  Nobody waits for anybody.  The gate/up kernel clears the
// counters, so a call leaves no state that the next one needs.  (The stores are
// agent-scope atomic stores, written through to where every XCD sees them; the wave
// waits for them before it counts, so a count that completes a unit stands for
// finished stores.  A release fence instead would write back an XCD's whole L2 in
// every workgroup.)
//
// Bound by HBM plus some 4 us per kernel that no load covers (launch, routing or
// ids, first bytes; reduction, join).  4096 x 2048, top-6 of 256 experts, gate/up +
// down in us, against the weights at the 6.28 TB/s of a pure read: one token 13.9 +
// 8.8 (8.5 + 4.3), four tokens 37.7 + 21.3 (32.8 + 16.4), sixteen 105 + 70 (114 +
// 57; some of the weights still lie in the memory-side cache).  Where tokens share
// experts the reads of their activations bind: sixteen tokens, top-2 of 8 experts,
// 33.6 + 29.6 (11.2 + 5.6).  On the way: routing
// every token in every workgroup 55.9 (four tokens, gate/up) -> ranks instead of k
// argmax rounds 53.4 -> unconditional LDS reads and no register spills 36.9.
#include "front.hpp"
#include "mx.hpp"

namespace moeq {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewMaxRows = 2 * kWave;        // routed rows: 16 tokens x 8 experts
static_assert(kFewTokens * MOEQ_MAX_TOPK <= kFewMaxRows, "two ballots cover the routed rows");
// Activation rows staged in LDS: at most four, in at most 17 KB for T <= 4 tokens
// (two rows of 4096 elements of x, one of 2048 of h in three planes), 25 KB above; a
// single row may take 40 KB.  More would leave fewer workgroups on a CU for rows that
// are rarely there; an expert with more rows reads them from memory.  Measured, us:
//   4096 x 2048, top-6 of 256 experts, gate/up with 17, 25, 33 KB: four tokens 37.6,
//   38.1, 40.7; sixteen 108.2, 105.1, 107.9; down with 17, 25 KB: four tokens 21.2,
//   22.4; with 25, 37 KB: eight 39.2, 46.7; sixteen 74.4, 73.8
//   one row in 17, 25, 40, 65 KB: h of 2880, one token 12.4, 9.9, 10.1, 9.7; of 6144
//   18.0, 18.1, 14.0, 13.9; of 8192, eight tokens 72.8, 71.4, 71.9, 79.8
constexpr int kStageRows = 4;
constexpr int few_stage_limit(int T) { return (T > 4 ? 25 : 17) << 10; }
constexpr int kStageOne = 40 << 10;
constexpr int kTurnBytes = 4096;              // LDS per wave for rows read from memory (MemoryAct)

constexpr int kDppRowRor8 = 0x128;            // lane i of 16 takes lane (i + 8) % 16
constexpr int kDppRowRor12 = 0x12C;           // ... lane (i + 4) % 16
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ mx_v4f mfma_bf16(const uint4& w, const uint4& a, const mx_v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, w),
                                                 __builtin_bit_cast(bf8, a), c, 0, 0, 0);
}

// v as the sum of three bf16 values: the top 8 significant bits (cut off, so the
// largest finite values do not round up to infinity), the next 8, the last 8.  Each
// difference is exact.  Bits below 2^-133, bf16's smallest step, are cut off.  The
// rest of an infinity is 0 (not inf - inf), that of a NaN a NaN.
constexpr int kHPlanes = 3;
__device__ __forceinline__ void split_bf16(float v, uint32_t (&p)[kHPlanes]) {
  p[0] = f2u(v) & 0xFFFF0000u;
  const float r = fabsf(v) == INFINITY ? 0.0f : v - u2f(p[0]);
  p[1] = f2u(r) & 0xFFFF0000u;
  p[2] = f2u(r - u2f(p[1]));
#pragma unroll
  for (int i = 0; i < kHPlanes; ++i) p[i] >>= 16;
}

// rows of one expert among the routed rows: the routed row of activation row n
// in `rows`, their number, and whether routed row r is the lowest of them
struct FewRows {
  int n;
  bool owner;
};
// (ids of one token differ, so there are at most T; the bounds keep ids that something
// else wrote from leaving the array)
__device__ __forceinline__ FewRows find_rows(int e_lo, int e_hi, int T, int R, int r, int lane,
                                             int* rows) {
  const int e = r < kWave ? readlane(e_lo, r & 63) : readlane(e_hi, r & 63);
  const uint64_t lo = __ballot(lane < R && e_lo == e);
  const uint64_t hi = __ballot(lane + kWave < R && e_hi == e);
  FewRows f;
  f.n = min(__popcll(lo) + __popcll(hi), T);
  f.owner = (lo ? __ffsll(static_cast<unsigned long long>(lo)) - 1
                : kWave + __ffsll(static_cast<unsigned long long>(hi)) - 1) == r;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int at_lo = __popcll(lo & below), at_hi = __popcll(lo) + __popcll(hi & below);
  if ((lo >> lane & 1) && at_lo < kFewTokens) rows[at_lo] = lane;
  if ((hi >> lane & 1) && at_hi < kFewTokens) rows[at_hi] = lane + kWave;
  return f;
}

// The activation rows of an expert: row i is row rows[i] of src, kPlanes planes of
// K bf16 elements each whose sum is the row's value.  In LDS plane p of row i lies at
// (i kPlanes + p) * plane_bytes, padded to whole super-groups and 16 bytes.
template <int kPlanes>
struct FewStage {
  const uint16_t* src;
  const int* rows;
  uint8_t* lds;
  int n, K, per_plane, plane_bytes;
  __device__ __forceinline__ FewStage(const uint16_t* src, const int* rows, uint8_t* lds, int K)
      : src(src), rows(rows), lds(lds), n(0), K(K), per_plane(mx_supers(K) * (kMxSuper / 8)),
        plane_bytes(per_plane * 16 + 16) {}
  // piece p (8 elements) of a plane of source row `row`; pieces past K are 0
  __device__ __forceinline__ uint4 piece(int row, int plane, int p) const {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (p * 8 < K)
      v = *reinterpret_cast<const uint4*>(src + (int64_t(row) * kPlanes + plane) * K + p * 8);
    return v;
  }
  __device__ __forceinline__ void put(int i, int plane, int p, const uint4& v) const {
    *reinterpret_cast<uint4*>(lds + (i * kPlanes + plane) * plane_bytes + p * 16) = v;
  }
  // copies pieces first, first + kFewThreads, ... of row i's planes
  __device__ __forceinline__ void copy(int i, int row, int first) const {
    for (int p = first; p < per_plane; p += kFewThreads) {
      uint4 v[kPlanes];
#pragma unroll
      for (int plane = 0; plane < kPlanes; ++plane) v[plane] = piece(row, plane, p);
#pragma unroll
      for (int plane = 0; plane < kPlanes; ++plane) put(i, plane, p, v[plane]);
    }
  }
};

// A row whose index is known ahead of the expert's others (the workgroup's own
// row, which is activation row 0 when the workgroup owns its expert): its first
// pieces are loaded at the top of the kernel and parked in LDS later.
template <int kPlanes>
struct EarlyRow {
  static constexpr int kEarly = 2;            // pieces per thread and plane
  uint4 v[kPlanes][kEarly];
  __device__ __forceinline__ void load(const FewStage<kPlanes>& st, int row, int tid) {
#pragma unroll
    for (int plane = 0; plane < kPlanes; ++plane)
#pragma unroll
      for (int i = 0; i < kEarly; ++i)
        if (tid + i * kFewThreads < st.per_plane) v[plane][i] = st.piece(row, plane, tid + i * kFewThreads);
  }
  __device__ __forceinline__ void store(const FewStage<kPlanes>& st, int row, int tid) const {
#pragma unroll
    for (int plane = 0; plane < kPlanes; ++plane)
#pragma unroll
      for (int i = 0; i < kEarly; ++i)
        if (tid + i * kFewThreads < st.per_plane) st.put(0, plane, tid + i * kFewThreads, v[plane][i]);
    st.copy(0, row, tid + kEarly * kFewThreads);
  }
};

// the two 16-row weight blocks of column unit u of one expert, and the K quarter
// of this wave
template <typename BlkF>
struct FewWeights {
  const uint8_t *w, *ws;
  BlkF blk;
  int G, g0, gn;
  __device__ __forceinline__ FewWeights(const uint8_t* w, const uint8_t* ws, int64_t e, int64_t blocks,
                                        int K, int q, BlkF blk)
      : blk(blk), G(mx_supers(K)), g0(quarter_g0(G, q)), gn(quarter_groups(G, q)) {
    this->w = w + e * blocks * G * kMxCodeBytes;
    this->ws = ws + e * blocks * G * kMxScaleBytes;
  }
  __device__ __forceinline__ void load(int u, int i, int lane, MxFrag (&f)[2]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t at = int64_t(blk(u, b)) * G;
      f[b] = load_weights<kCpStream>(w + at * kMxCodeBytes, ws + at * kMxScaleBytes, g0 + i, lane);
    }
  }
};

// Activations of one super-group as the 16 columns of the products take them: lane
// (ln, kb) holds column ln's blocks 4 kb .. 4 kb + 3 (256 consecutive bytes), step j
// and quarter m of it 16 bytes.  kSets columns sets share the weights.
//
// From LDS, where the rows are staged: one set, `at` the lane's column and kb.
struct StagedAct {
  static constexpr int kSets = 1;
  const uint8_t* at;
  uint4 v[1][4];
  __device__ __forceinline__ void load(int sg, int j) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
      v[0][m] = *reinterpret_cast<const uint4*>(at + sg * 1024 + j * 64 + m * 16);
  }
};
// From memory.  A load takes 64 consecutive bytes (one block) of 16 columns, lane l
// piece l % 4 of column l / 4, so that it touches 16 lines and not 64; 4 KB of LDS
// that belong to the wave turn the pieces round.  (`at`: the lane's column l / 4 of
// each set, `turn`: the wave's LDS, XOR-swizzled so that the 16 columns of one kb
// read different banks.)  Blocks past K are 0.  Down product, 4096 x 2048, 16 tokens,
// in us: top-8 of 8 experts 80.4 with each lane loading its own pieces, 45.6 turned;
// top-2 of 8 37.3, 29.6.
template <int kColumnSets>
struct MemoryAct {
  static constexpr int kSets = kColumnSets;
  const uint8_t* at[kSets];
  uint8_t* turn;
  int blocks, lane;
  uint4 v[kSets][4];
  __device__ __forceinline__ void load(int sg, int j) {
#pragma unroll
    for (int p = 0; p < kSets; ++p)
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const int b = 16 * sg + 4 * kb + j;
        v[p][kb] = make_uint4(0u, 0u, 0u, 0u);
        if (b < blocks) v[p][kb] = *reinterpret_cast<const uint4*>(at[p] + b * 64);
      }
    const int wc = lane >> 2, wm = lane & 3, ln = lane & 15, kb = lane >> 4;
#pragma unroll
    for (int p = 0; p < kSets; ++p) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<uint4*>(turn + ((b * 16 + wc) * 4 + (wm ^ (wc >> 2))) * 16) = v[p][b];
      lds_wave_sync();
#pragma unroll
      for (int m = 0; m < 4; ++m)
        v[p][m] = *reinterpret_cast<const uint4*>(turn + ((kb * 16 + ln) * 4 + (m ^ (ln >> 2))) * 16);
      lds_wave_sync();
    }
  }
};

// acc += W A over one super-group
template <typename ActT>
__device__ __forceinline__ void few_mac(const MxFrag (&f)[2], ActT& act, int sg, mx_v4f (&acc)[2]) {
  static_for<kMxSteps>([&](auto j) {
    float sc[2];                              // byte j of the scale dword in the exponent field
#pragma unroll
    for (int b = 0; b < 2; ++b)
      sc[b] = u2f((j < 3 ? f[b].s << (j < 3 ? 23 - 8 * j : 0) : f[b].s >> 1) & 0x7F800000u);
    act.load(sg, j);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t c = m == 0 ? f[b].c[j].x : m == 1 ? f[b].c[j].y : m == 2 ? f[b].c[j].z : f[b].c[j].w;
        const uint4 wv = mx_bf16x8(c, sc[b]);
#pragma unroll
        for (int p = 0; p < ActT::kSets; ++p) acc[b] = mfma_bf16(wv, act.v[p][m], acc[b]);
      }
  });
}

// The column units u0 .. u1 - 1 of one expert.  A unit is a product of two 16-row
// weight blocks with the rows' activations; wave q sweeps K quarter q, the
// quarters meet in LDS in the fixed order s0 + (s1 + (s2 + s3)), and wave 0 calls
// done(u, sums).  The sweep runs over items (unit, super-group of the quarter)
// with two register sets, so the next item's weights are in flight while one is
// multiplied; the first item's are already in `f0`.
//
// kStaged: the rows are in LDS, otherwise they are read from memory.  Columns past
// the last row read the last one (their results are never used).  kGrouped (at most
// kStageRows rows, which leaves columns free): the planes share one product, columns
// 4 p .. 4 p + 3 read plane p of rows 0 .. 3 (the last four the last plane once more,
// unused) and the groups are added at the end.  Otherwise a product per plane.
template <bool kStaged, bool kGrouped, int kPlanes, typename WeightsT, typename DoneF>
__device__ __forceinline__ void few_units(const WeightsT& wt, int u0, int u1, const FewStage<kPlanes>& st,
                                          MxFrag (&f0)[2], mx_v4f* red, DoneF&& done) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int q = __builtin_amdgcn_readfirstlane(tid >> 6);
  static_assert(kStageRows <= 4 && (kPlanes == 1 || kPlanes == 3), "four of the 16 columns per plane");
  static_assert(!kStaged || kGrouped || kPlanes == 1, "staged rows are few");
  constexpr bool kGroups = kGrouped && kPlanes > 1;
  const int ln = lane & 15, kb = lane >> 4;
  const auto col_row = [&](int c) { return min(kGroups ? c & 3 : c, st.n - 1); };
  const auto col_plane = [&](int c) { return kGroups ? min(c >> 2, kPlanes - 1) : 0; };
  std::conditional_t<kStaged, StagedAct, MemoryAct<kGroups ? 1 : kPlanes>> act;
  if constexpr (kStaged) {
    act.at = st.lds + (col_row(ln) * kPlanes + col_plane(ln)) * st.plane_bytes + kb * 256;
  } else {
    const int c = lane >> 2;
#pragma unroll
    for (int p = 0; p < act.kSets; ++p)
      act.at[p] = reinterpret_cast<const uint8_t*>(
          st.src + (int64_t(st.rows[col_row(c)]) * kPlanes + col_plane(c) + p) * st.K + (lane & 3) * 8);
    act.turn = st.lds + q * kTurnBytes;
    act.blocks = st.K / kMxBlock;
    act.lane = lane;
  }
  const int per_unit = max(wt.gn, 1);                   // a wave without K still joins the sums
  const int items = (u1 - u0) * per_unit;
  mx_v4f acc[2] = {mx_v4f{0.f, 0.f, 0.f, 0.f}, mx_v4f{0.f, 0.f, 0.f, 0.f}};
  int u = u0, i = 0;                                    // the current item
  int lu = u0, li = 0;                                  // the last item loaded

  auto load_next = [&](MxFrag (&f)[2]) {
    if (++li == per_unit) { li = 0; ++lu; }
    if (lu < u1 && wt.gn > 0) wt.load(lu, li, lane, f);
  };
  auto step = [&](MxFrag (&f)[2]) {
    if (wt.gn > 0) few_mac(f, act, wt.g0 + i, acc);
    if (++i < per_unit) return;
    // one half of red per unit parity: a unit's sums are read before the barrier
    // of the next, and overwritten after it
    mx_v4f* half = red + (u & 1) * (3 * 2 * kWave);
    if (q > 0) {
      half[((q - 1) * 2) * kWave + lane] = acc[0];
      half[((q - 1) * 2 + 1) * kWave + lane] = acc[1];
    }
    lds_barrier();
    if (q == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[j] = acc[j] + (half[j * kWave + lane] +
                           (half[(2 + j) * kWave + lane] + half[(4 + j) * kWave + lane]));
      if (kGroups) {                                    // columns n + 4 and n + 8 to column n
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[j][v] += dpp<kDppRowRor12>(acc[j][v], acc[j][v]) + dpp<kDppRowRor8>(acc[j][v], acc[j][v]);
      }
      done(u, acc);
    }
    acc[0] = acc[1] = mx_v4f{0.f, 0.f, 0.f, 0.f};
    i = 0;
    ++u;
  };
  if constexpr (kStaged) {
    MxFrag f1[2];
    load_next(f1);
    for (int it = 0; it < items; it += 2) {
      step(f0);
      if (it + 1 == items) break;
      load_next(f0);
      step(f1);
      load_next(f1);
    }
  } else {
    // one register set, loaded anew: activations straight from memory take the room
    // of the second, and the first item's early copy need not stay live for this path
    MxFrag f[2];
    li = -1;
    for (int it = 0; it < items; ++it) {
      load_next(f);
      step(f);
    }
  }
}

// Stages the rows after row 0 (which is in LDS) if all fit, and runs the units.
template <int kPlanes, typename WeightsT, typename DoneF>
__device__ __forceinline__ void few_run(const WeightsT& wt, int u0, int u1, const FewStage<kPlanes>& st,
                                        int stage_rows, MxFrag (&f0)[2], mx_v4f* red, DoneF&& done) {
  if (st.n <= stage_rows) {
    if (st.n > 1) {
      for (int i = 1; i < st.n; ++i) st.copy(i, st.rows[i], threadIdx.x);
      lds_barrier();
    }
    few_units<true, true>(wt, u0, u1, st, f0, red, done);
  } else if (kPlanes > 1 && st.n <= kStageRows) {
    few_units<false, true>(wt, u0, u1, st, f0, red, done);
  } else {
    few_units<false, false>(wt, u0, u1, st, f0, red, done);
  }
}

// -------------------------------------------------------------- kernel 1
// One token's biased scores as order-preserving keys (front.hpp), expert e in lane
// e % 64, slot e / 64; 0 past E and at least 1 before it (one NaN has key 0), so that
// every expert has a rank and at_rank and rank_of invert each other whatever the
// scores hold: each routed row is computed by exactly one workgroup per unit.
template <int NS>
struct Scores {
  uint32_t key[NS];
  __device__ __forceinline__ void load(const float* row, const float* bias, int E, int lane) {
    float s[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = row[min(i * kWave + lane, E - 1)];
    if (bias) {
#pragma unroll
      for (int i = 0; i < NS; ++i) s[i] = s[i] + bias[min(i * kWave + lane, E - 1)];
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) key[i] = i * kWave + lane < E ? max(score_key(s[i]), 1u) : 0u;
  }
  // the expert of rank j (0 the best): j + 1 rounds of a wave-wide argmax, as in
  // route_token_values
  __device__ __forceinline__ int at_rank(int j, int lane) const {
    uint32_t rest[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) rest[i] = key[i];
    int e = 0;
    for (int round = 0; round <= j; ++round) {
      uint32_t ck = 0, bk;
      int ci = 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (rest[i] > ck) { ck = rest[i]; ci = i * kWave + lane; }
      e = wave_best(ck, ci, &bk);
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i * kWave + lane == e) rest[i] = 0u;
    }
    return __builtin_amdgcn_readfirstlane(e);
  }
  // the rank of expert e: the number of experts ahead of it in the same order
  __device__ __forceinline__ int rank_of(int e, int lane) const {
    uint32_t ke = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i == (e >> 6)) ke = uint32_t(readlane(int(key[i]), e & 63));
    int n = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      n += __popcll(__ballot(key[i] > ke || (key[i] == ke && i * kWave + lane < e)));
    return n;
  }
};

template <int NS>
__global__ void __launch_bounds__(kFewThreads, NS > 8 ? 2 : 4)    // waves per SIMD
few_gate_up_kernel(const float* logits, const float* bias, int T, int E, int k, int renormalize,
                   const uint16_t* x, int H, const uint8_t* w13, const uint8_t* ws13, int I,
                   int units_per_wg, int stage_rows, int32_t* ids, float* topk_w, uint16_t* h,
                   uint32_t* counters, int n_counters) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ mx_v4f red[2 * 3 * 2 * kWave];
  __shared__ int ranks[kFewTokens], rows[kFewTokens], tokens[kFewTokens];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int units = I / 16;
  const int runs = (units + units_per_wg - 1) / units_per_wg;
  const int r = blockIdx.x / runs, run = blockIdx.x - r * runs;
  const int u0 = run * units_per_wg, u1 = min(u0 + units_per_wg, units);
  const int t = r / k, j = r - t * k;

  // one workgroup per token writes its weights
  constexpr int kWaves = kFewThreads / kWave, kMine = kFewTokens / kWaves;
  if (run == 0 && j == 0 && wave == kWaves - 1) {
    float w;
    route_token_values<NS>(logits + int64_t(t) * E, bias, E, k, renormalize, lane, w);
    if (lane < k) topk_w[t * k + lane] = w;
  }

  // Routing.  The row's expert is the j-th best of its token (each wave finds it);
  // wave w then ranks it among the scores of tokens w, w + 4, ...: another token
  // has a row for it exactly if its rank there is below k.  (Ranking costs a few
  // ballots, against k argmax rounds for routing every token.)  The token's own
  // row of x is read alongside, and the expert's first weights go out as soon as
  // the expert is known, ahead of the rest: a workgroup that then turns out not to
  // own its expert has read one item in vain.
  Scores<NS> own, mine[kMine];
  own.load(logits + int64_t(t) * E, bias, E, lane);
  FewStage<1> st(x, tokens, lds, H);
  EarlyRow<1> early;
  if (stage_rows > 0) early.load(st, t, tid);
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (wave + i * kWaves < T) mine[i].load(logits + int64_t(wave + i * kWaves) * E, bias, E, lane);
  const int e = own.at_rank(j, lane);
  if (run == 0 && tid == 0) ids[r] = e;
  auto blk = [I](int u, int b) { return u + b * (I / 16); };
  const FewWeights<decltype(blk)> wt(w13, ws13, e, (2 * I) / 16, H, wave, blk);
  MxFrag f0[2];
  if (wt.gn > 0) wt.load(u0, 0, lane, f0);
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (wave + i * kWaves < T) {
      const int rank = mine[i].rank_of(e, lane);
      if (lane == 0) ranks[wave + i * kWaves] = rank;
    }
  if (stage_rows > 0) early.store(st, t, tid);
  if (blockIdx.x == 0)
    for (int i = tid; i < n_counters; i += kFewThreads) counters[i] = 0;
  lds_barrier();
  const int rank = ranks[min(lane, T - 1)];
  const uint64_t members = __ballot(lane < T && rank < k);
  if (__ffsll(static_cast<unsigned long long>(members)) - 1 != t) return;   // workgroup-uniform
  const int n = __popcll(members);
  if (members >> lane & 1) {                            // (every wave writes the same)
    const int at = __popcll(members & ((uint64_t(1) << lane) - 1));
    tokens[at] = lane;
    rows[at] = lane * k + rank;
  }
  if (n > 1) lds_barrier();
  st.n = n;
  const int ln = lane & 15, kb = lane >> 4;
  auto done = [&](int u, const mx_v4f (&v)[2]) {
    if (ln >= n) return;
    const mx_v4f hv = silu_mul4(v[0], v[1]);
    uint32_t p[4][kHPlanes];
#pragma unroll
    for (int c = 0; c < 4; ++c) split_bf16(hv[c], p[c]);
    uint16_t* at = h + int64_t(rows[ln]) * kHPlanes * I + 16 * u + 4 * kb;
#pragma unroll
    for (int i = 0; i < kHPlanes; ++i)
      *reinterpret_cast<uint2*>(at + i * I) =
          make_uint2(p[0][i] | p[1][i] << 16, p[2][i] | p[3][i] << 16);
  };
  few_run(wt, u0, u1, st, stage_rows, f0, red, done);
}

// -------------------------------------------------------------- kernel 2
// 8 bytes past the caches (agent scope: other XCDs' L2s do not see this one's)
__device__ __forceinline__ void store_through(float* p, float a, float b) {
  const uint64_t v = uint64_t(f2u(a)) | (uint64_t(f2u(b)) << 32);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_through(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(u2f(uint32_t(v)), u2f(uint32_t(v >> 32)));
}

__global__ void __launch_bounds__(kFewThreads, 4)
few_down_kernel(const int32_t* ids, const float* topk_w, const uint16_t* h, int T, int E, int k,
                const uint8_t* w2, const uint8_t* ws2, int H, int I, int units_per_wg,
                int stage_rows, float* o, uint32_t* counters, const uint16_t* shared, uint16_t* y) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ mx_v4f red[2 * 3 * 2 * kWave];
  __shared__ int rows[kFewTokens];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k;
  const int units = H / 32;
  const int runs = (units + units_per_wg - 1) / units_per_wg;
  const int r = blockIdx.x / runs;
  const int u0 = (blockIdx.x - r * runs) * units_per_wg, u1 = min(u0 + units_per_wg, units);
  const int e_lo = ids[min(lane, R - 1)], e_hi = ids[min(lane + kWave, R - 1)];
  FewStage<kHPlanes> st(h, rows, lds, I);
  EarlyRow<kHPlanes> early;
  if (stage_rows > 0) early.load(st, r, tid);
  // (ids come from the first kernel of the call; clamped all the same)
  const int e = min(max(__builtin_amdgcn_readfirstlane(ids[r]), 0), E - 1);
  auto blk = [](int u, int b) { return 2 * u + b; };
  const FewWeights<decltype(blk)> wt(w2, ws2, e, H / 16, I, wave, blk);
  MxFrag f0[2];
  if (wt.gn > 0) wt.load(u0, 0, lane, f0);
  if (stage_rows > 0) early.store(st, r, tid);
  const FewRows f = find_rows(e_lo, e_hi, T, R, r, lane, rows);
  const int ln = lane & 15, kb = lane >> 4;

  // Wave 0, after its stores: one arrival per unit of the run, then y where this
  // was the last one (T tokens x 8 column quads per unit).
  auto arrive = [&]() {
    // the stores have reached memory before the arrivals are counted
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    uint32_t before = 0;
    if (lane < u1 - u0)
      before = __hip_atomic_fetch_add(counters + u0 + lane, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
    uint64_t last = __ballot(lane < u1 - u0 && before + 1 == uint32_t(R));
    asm volatile("" ::: "memory");
    for (; last; last &= last - 1) {
      const int u = u0 + __ffsll(static_cast<unsigned long long>(last)) - 1;
      for (int i = lane; i < T * 8; i += kWave) {
        const int t = i >> 3, c = 32 * u + 4 * (i & 7);
        float2 p[MOEQ_MAX_TOPK][2];
        float wt[MOEQ_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOEQ_MAX_TOPK; ++j) {
          const int s = t * k + min(j, k - 1);
          p[j][0] = load_through(o + int64_t(s) * H + c);
          p[j][1] = load_through(o + int64_t(s) * H + c + 2);
          wt[j] = topk_w[s];
        }
        mx_v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < MOEQ_MAX_TOPK; ++j) {
          // (a weight of 0, a masked expert's, adds nothing whatever its row holds)
          if (j < k && wt[j] != 0.0f) {
            acc[0] = fmaf(wt[j], p[j][0].x, acc[0]);
            acc[1] = fmaf(wt[j], p[j][0].y, acc[1]);
            acc[2] = fmaf(wt[j], p[j][1].x, acc[2]);
            acc[3] = fmaf(wt[j], p[j][1].y, acc[3]);
          }
        }
        if (shared) {
          const uint2 sh = *reinterpret_cast<const uint2*>(shared + int64_t(t) * H + c);
          acc[0] += u2f(sh.x << 16);
          acc[1] += u2f(sh.x & 0xFFFF0000u);
          acc[2] += u2f(sh.y << 16);
          acc[3] += u2f(sh.y & 0xFFFF0000u);
        }
        store4(y, 0, int64_t(t) * H + c, acc);
      }
    }
  };

  if (!f.owner) {                               // its expert's rows are another workgroup's
    if (wave == 0) arrive();
    return;
  }
  lds_barrier();
  st.n = f.n;
  auto done = [&](int u, const mx_v4f (&v)[2]) {
    if (ln < f.n) {
      float* p = o + int64_t(rows[ln]) * H + 32 * u + 4 * kb;
      store_through(p, v[0][0], v[0][1]);
      store_through(p + 2, v[0][2], v[0][3]);
      store_through(p + 16, v[1][0], v[1][1]);
      store_through(p + 18, v[1][2], v[1][3]);
    }
  };
  few_run(wt, u0, u1, st, stage_rows, f0, red, done);
  if (wave == 0) arrive();
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// rows staged in LDS for rows of `planes` planes of K elements, and their bytes
int few_row_bytes(int planes, int K) { return planes * (mx_supers(K) * (kMxSuper * 2) + 16); }
int few_stage_rows(int T, int planes, int K) {
  const int fit = few_stage_limit(T) / few_row_bytes(planes, K);
  const int n = T < kStageRows ? T : kStageRows;
  if (fit == 0) return few_row_bytes(planes, K) <= kStageOne ? 1 : 0;
  return n < fit ? n : fit;
}
// LDS of a launch: the staged rows, or what reading them from memory takes if an
// expert may have more
unsigned few_lds_bytes(int T, int planes, int K) {
  const int rows = few_stage_rows(T, planes, K);
  const int staged = rows * few_row_bytes(planes, K), turn = kTurnBytes * (kFewThreads / kWave);
  return unsigned(rows < T && staged < turn ? turn : staged);
}

// Column units per workgroup.  One unit each lets the dispatcher balance the CUs,
// several spread the routing and the joins over more weights; a launch is to hold
// about `launch` workgroups (some rounds of the four that fit a CU).  Measured at 4096
// x 2048, top-6 of 256 experts (gate/up, down; us): one token 13.8, 8.3 with one unit,
// 14.8, 10.2 with two; four 36.9, 20.6 with one, 37.5, 22.2 with two, 37.9, 24.6 with
// four; sixteen 142.5, 83.0 with one, 115.3, 71.8 with two, 110.6, 70.6 with three,
// 105.8, 73.4 with four, 112.5, 84.2 with six.
// R counts every routed row, those that leave at once too: they route before they
// leave.  Sized by the rows that can stay, min(R, E): sixteen tokens, top-8 of 8,
// 4096 x 2048, 102, 86 against 40, 46; top-4 of 32, 2880 x 2880, 88, 60 against 64, 60.
// Launches of 1500 and 2048: sixteen tokens, top-2 of 8, 26.5, 25.8 against 33.5, 29.7,
// but eight, top-6 of 256, 67.5, 42.6 against 67.0, 39.6.
int few_units_per_wg(int R, int units, int launch) {
  const int64_t n = int64_t(R) * units / launch;
  return n < 1 ? 1 : n > 4 ? 4 : int(n);
}

}  // namespace

size_t few_ws_bytes(int T, int k, int H, int I) {
  const size_t R = size_t(T) * k;
  return align256(size_t(H / 32) * 4) + align256(R * I * (2 * kHPlanes)) + align256(R * H * 4);
}

hipError_t launch_layer_mxfp4_few(const float* logits, const float* bias, int T, int E, int k,
                                  int renormalize, const uint16_t* x, int H, const uint8_t* w13,
                                  const uint8_t* ws13, const uint8_t* w2, const uint8_t* ws2, int I,
                                  const uint16_t* shared, int32_t* ids, float* topk_w, uint16_t* y,
                                  void* ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int R = T * k;
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint32_t* counters = reinterpret_cast<uint32_t*>(base);
  uint16_t* h = reinterpret_cast<uint16_t*>(base + align256(size_t(H / 32) * 4));
  float* o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(h) + align256(size_t(R) * I * (2 * kHPlanes)));
  const int upw1 = few_units_per_wg(R, I / 16, 3000), upw2 = few_units_per_wg(R, H / 32, 4096);
  const int runs1 = (I / 16 + upw1 - 1) / upw1, runs2 = (H / 32 + upw2 - 1) / upw2;
  with_route_slots(E, [&](auto ns) {
    hipLaunchKernelGGL((few_gate_up_kernel<decltype(ns)::value>), dim3(unsigned(R * runs1)),
                       dim3(kFewThreads), few_lds_bytes(T, 1, H), stream, logits, bias, T, E, k,
                       renormalize, x, H, w13, ws13, I, upw1, few_stage_rows(T, 1, H), ids, topk_w, h,
                       counters, H / 32);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(few_down_kernel, dim3(unsigned(R * runs2)), dim3(kFewThreads),
                     few_lds_bytes(T, kHPlanes, I), stream, ids, topk_w, h, T, E, k, w2, ws2, H, I, upw2,
                     few_stage_rows(T, kHPlanes, I), o, counters, shared, y);
  return hipGetLastError();
}

}  // namespace moeq
