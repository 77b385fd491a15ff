// A whole MoE layer for at most 16 tokens in two kernels, with MXFP4 expert
// weights and bf16 activations (weight-only quantization: a few tokens are bound
// by the weight stream, so 16-bit activations cost nothing and spare the layer
// their rounding to 4 bits):
//   few_gate_up_kernel  s = logits + bias, top-k, weights;  h = silu(Wg x) * (Wu x)
//   few_down_kernel     o_j = W2 h_j;  y = sum_j w_j o_j (+ shared)
//
// Sums: W = e2m1 * 2^s converts exactly to bf16 (2 significant bits), products
// and sums run in fp32 on v_mfma_f32_16x16x32_bf16.  h is rounded once to bf16,
// the second product's operand type (2^-9 of each element, uncorrelated over the
// I summands; the layer's 8-bit and 16-bit paths round h the same way).  o stays
// fp32; y is rounded once.
//
// Work units.  A workgroup belongs to one routed row r = t k + j and a run of
// column units.  It routes all T tokens itself (gate/up; 4 T E bytes from L2), so
// no launch is spent on routing, then finds with two ballots which rows share its
// row's expert: the lowest of them owns the expert and computes all of them (an
// expert has at most one row per token, so at most 16: one 16-column MFMA block),
// the others' workgroups leave at once.  No plan is built or read.
//
// Joining the experts' outputs without a third launch: the down kernel's
// workgroups store their fp32 o columns past the caches, then count up one
// arrival counter per column unit; the one that arrives last has all T k rows of
// its 32 columns and forms y in slot order j, so results do not depend on the
// arrival order.  Nobody waits for anybody.  The gate/up kernel clears the
// counters, so a call leaves no state that the next one needs.
#include "front.hpp"
#include "mx.hpp"

namespace moeq {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewMaxRows = 2 * kWave;        // routed rows: 16 tokens x 8 experts
static_assert(kFewTokens * MOEQ_MAX_TOPK <= kFewMaxRows, "two ballots cover the routed rows");
constexpr int kStageRows = 4;                 // rows of activations staged in LDS

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ mx_v4f mfma_bf16(const uint4& w, const uint4& a, const mx_v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, w),
                                                 __builtin_bit_cast(bf8, a), c, 0, 0, 0);
}

// rows of one expert among the routed rows: the routed row of activation row n
// in `rows`, their number, and whether routed row r is the lowest of them
struct FewRows {
  int n;
  bool owner;
};
__device__ __forceinline__ FewRows find_rows(int e_lo, int e_hi, int R, int r, int lane, int* rows) {
  const int e = r < kWave ? readlane(e_lo, r & 63) : readlane(e_hi, r & 63);
  const uint64_t lo = __ballot(lane < R && e_lo == e);
  const uint64_t hi = __ballot(lane + kWave < R && e_hi == e);
  FewRows f;
  f.n = __popcll(lo) + __popcll(hi);
  f.owner = (lo ? __ffsll(static_cast<unsigned long long>(lo)) - 1
                : kWave + __ffsll(static_cast<unsigned long long>(hi)) - 1) == r;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  if (lo >> lane & 1) rows[__popcll(lo & below)] = lane;
  if (hi >> lane & 1) rows[__popcll(lo) + __popcll(hi & below)] = lane + kWave;
  return f;
}

// The activations of an expert's rows as the second operand: from LDS (rows
// staged by the workgroup) or from memory (more than the staged rows).
struct FewAct {
  const uint8_t* lds;       // this lane's row in LDS (bytes), rows G * 1024 + 16 apart
  const uint16_t* mem;      // this lane's row in memory
  bool staged, live;
  int K;
  // 8 elements m of block b (32 b + 8 m)
  __device__ __forceinline__ uint4 get(int b, int m) const {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (!live) return v;
    if (staged) v = *reinterpret_cast<const uint4*>(lds + b * 64 + m * 16);
    else if (b * kMxBlock < K) v = *reinterpret_cast<const uint4*>(mem + b * kMxBlock + m * 8);
    return v;
  }
};

// acc += W A over one super-group
__device__ __forceinline__ void few_mac(const MxFrag& f0, const MxFrag& f1, const FewAct& act,
                                        int sg, int kb, mx_v4f (&acc)[2]) {
  static_for<kMxSteps>([&](auto j) {
    const float sc0 = u2f((f0.s << (23 - 8 * j > 0 ? 23 - 8 * j : 0) >> (8 * j > 23 ? 8 * j - 23 : 0)) & 0x7F800000u);
    const float sc1 = u2f((f1.s << (23 - 8 * j > 0 ? 23 - 8 * j : 0) >> (8 * j > 23 ? 8 * j - 23 : 0)) & 0x7F800000u);
    const uint32_t c0[4] = {f0.c[j].x, f0.c[j].y, f0.c[j].z, f0.c[j].w};
    const uint32_t c1[4] = {f1.c[j].x, f1.c[j].y, f1.c[j].z, f1.c[j].w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint4 a = act.get(16 * sg + 4 * kb + j, m);
      acc[0] = mfma_bf16(mx_bf16x8(c0[m], sc0), a, acc[0]);
      acc[1] = mfma_bf16(mx_bf16x8(c1[m], sc1), a, acc[1]);
    }
  });
}

// 16-byte pieces of the expert's activation rows into LDS: piece c of the
// flattened (row, piece of a row padded to G super-groups); pieces past K are 0
struct FewStage {
  const uint16_t* src;      // [.., K] rows
  const int* rows;          // row of src of each activation row
  int n, K, per_row, row_bytes;
  __device__ __forceinline__ bool load(int c, uint4& v) const {
    const int row = c / per_row, p = c - row * per_row;
    v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= n) return false;
    if (p * 8 < K) v = *reinterpret_cast<const uint4*>(src + int64_t(rows[row]) * K + p * 8);
    return true;
  }
  __device__ __forceinline__ void store(uint8_t* lds, int c, const uint4& v) const {
    const int row = c / per_row, p = c - row * per_row;
    *reinterpret_cast<uint4*>(lds + row * row_bytes + p * 16) = v;
  }
};

// The column units u0 .. u1 - 1 of one expert: unit u multiplies the 16-row
// weight blocks blk0(u), blk1(u) by the rows' activations; wave q sweeps K quarter
// q, the quarters meet in LDS in the fixed order s0 + (s1 + (s2 + s3)), and wave 0
// calls done(u, sums) (every wave calls done; only wave 0's sums are whole).
// The next item's weights are loaded before this one's are used.
template <typename BlkF, typename DoneF>
__device__ __forceinline__ void few_units(const uint8_t* w, const uint8_t* ws, int K, int u0,
                                          int u1, const FewStage& st, uint8_t* lds, bool staged,
                                          mx_v4f* red, BlkF&& blk, DoneF&& done) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int q = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, kb = lane >> 4;
  const int G = mx_supers(K);
  const int g0 = quarter_g0(G, q), gn = quarter_groups(G, q);

  auto load = [&](int u, int sg, MxFrag& f0, MxFrag& f1) {
    const int64_t b0 = blk(u, 0), b1 = blk(u, 1);
    f0 = load_weights<kCpStream>(w + b0 * G * kMxCodeBytes, ws + b0 * G * kMxScaleBytes, sg, lane);
    f1 = load_weights<kCpStream>(w + b1 * G * kMxCodeBytes, ws + b1 * G * kMxScaleBytes, sg, lane);
  };

  // the first pieces of the activations go out ahead of the weights, and are
  // written to LDS while those are in flight
  constexpr int kAhead = 4;
  uint4 piece[kAhead];
  bool have[kAhead];
  if (staged) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) have[i] = st.load(tid + i * kFewThreads, piece[i]);
  }
  MxFrag f0, f1;
  if (gn > 0) load(u0, g0, f0, f1);
  if (staged) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (have[i]) st.store(lds, tid + i * kFewThreads, piece[i]);
    uint4 v;
    for (int c = tid + kAhead * kFewThreads; c < st.n * st.per_row; c += kFewThreads)
      if (st.load(c, v)) st.store(lds, c, v);
  }
  lds_barrier();
  FewAct act;
  act.live = ln < st.n;
  act.staged = staged;
  act.K = K;
  act.lds = lds + (act.live ? ln : 0) * st.row_bytes;
  act.mem = st.src + int64_t(st.rows[act.live ? ln : 0]) * K;

  for (int u = u0; u < u1; ++u) {
    mx_v4f acc[2] = {mx_v4f{0.f, 0.f, 0.f, 0.f}, mx_v4f{0.f, 0.f, 0.f, 0.f}};
    for (int i = 0; i < gn; ++i) {
      MxFrag n0 = f0, n1 = f1;
      const bool more = i + 1 < gn;
      if (more || u + 1 < u1) load(more ? u : u + 1, more ? g0 + i + 1 : g0, n0, n1);
      few_mac(f0, f1, act, g0 + i, kb, acc);
      f0 = n0;
      f1 = n1;
    }
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
      done(u, acc);
    }
  }
}

// -------------------------------------------------------------- kernel 1
template <int NS>
__global__ void __launch_bounds__(kFewThreads)
few_gate_up_kernel(const float* logits, const float* bias, int T, int E, int k, int renormalize,
                   const uint16_t* x, int H, const uint8_t* w13, const uint8_t* ws13, int I,
                   int units_per_wg, int stage_rows, int32_t* ids, float* topk_w, uint16_t* h,
                   uint32_t* counters, int n_counters) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ mx_v4f red[2 * 3 * 2 * kWave];
  __shared__ int sel[kFewMaxRows];
  __shared__ int rows[kFewTokens], tokens[kFewTokens];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k;

  for (int t = wave; t < T; t += kFewThreads / kWave) {
    float wt;
    const int e = route_token_values<NS>(logits + int64_t(t) * E, bias, E, k, renormalize, lane, wt);
    if (lane < k) {
      sel[t * k + lane] = e;
      if (blockIdx.x == 0) {
        // a token whose best score is -inf has no weights (0/0): it gets zeros
        const int best = readlane(e, 0);
        const float s0 = logits[int64_t(t) * E + best] + (bias ? bias[best] : 0.0f);
        ids[t * k + lane] = e;
        topk_w[t * k + lane] = s0 == -INFINITY ? 0.0f : wt;
      }
    }
  }
  if (blockIdx.x == 0)
    for (int i = tid; i < n_counters; i += kFewThreads) counters[i] = 0;
  lds_barrier();
  const int units = I / 16;
  const int runs = (units + units_per_wg - 1) / units_per_wg;
  const int r = blockIdx.x / runs;
  const int u0 = (blockIdx.x - r * runs) * units_per_wg, u1 = min(u0 + units_per_wg, units);
  const int e_lo = sel[min(lane, R - 1)], e_hi = sel[min(lane + kWave, R - 1)];
  const FewRows f = find_rows(e_lo, e_hi, R, r, lane, rows);    // (every wave writes the same)
  if (!f.owner) return;                                         // workgroup-uniform
  const int e = __builtin_amdgcn_readfirstlane(sel[r]);
  if (lane < f.n) tokens[lane] = rows[lane] / k;
  lds_barrier();

  FewStage st;
  st.src = x;
  st.rows = tokens;
  st.n = f.n;
  st.K = H;
  st.per_row = mx_supers(H) * (kMxSuper / 8);
  st.row_bytes = st.per_row * 16 + 16;
  const int64_t blocks = int64_t(2 * I) / 16, G = mx_supers(H);
  const int ln = lane & 15, kb = lane >> 4;
  few_units(w13 + e * blocks * G * kMxCodeBytes, ws13 + e * blocks * G * kMxScaleBytes, H, u0, u1,
            st, lds, f.n <= stage_rows, red,
            [&](int u, int j) { return u + j * (I / 16); },
            [&](int u, const mx_v4f (&v)[2]) {
              if (ln >= f.n) return;
              const mx_v4f hv = silu_mul4(v[0], v[1]);
              store4(h, 0, int64_t(rows[ln]) * I + 16 * u + 4 * kb, hv);
            });
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

__global__ void __launch_bounds__(kFewThreads)
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
  const FewRows f = find_rows(e_lo, e_hi, R, r, lane, rows);
  const int ln = lane & 15, kb = lane >> 4;

  // The wave that completes unit u forms y there: T tokens x 8 column quads.
  auto arrive = [&](int u) {
    // this wave's stores have reached memory before its arrival does
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    uint32_t before = 0;
    if (lane == 0)
      before = __hip_atomic_fetch_add(counters + u, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    before = __builtin_amdgcn_readfirstlane(before);
    asm volatile("" ::: "memory");
    if (before + 1 != uint32_t(R)) return;
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
        if (j < k) {
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
  };

  if (!f.owner) {                               // its expert's rows are another workgroup's
    if (wave == 0)
      for (int u = u0; u < u1; ++u) arrive(u);
    return;
  }
  // (ids come from the first kernel of the call; clamped all the same)
  const int e = __builtin_amdgcn_readfirstlane(min(max(ids[r], 0), E - 1));
  lds_barrier();

  FewStage st;
  st.src = h;
  st.rows = rows;
  st.n = f.n;
  st.K = I;
  st.per_row = mx_supers(I) * (kMxSuper / 8);
  st.row_bytes = st.per_row * 16 + 16;
  const int64_t blocks = H / 16, G = mx_supers(I);
  few_units(w2 + e * blocks * G * kMxCodeBytes, ws2 + e * blocks * G * kMxScaleBytes, I, u0, u1, st,
            lds, f.n <= stage_rows, red, [&](int u, int j) { return 2 * u + j; },
            [&](int u, const mx_v4f (&v)[2]) {
              if (ln < f.n) {
                float* p = o + int64_t(rows[ln]) * H + 32 * u + 4 * kb;
                store_through(p, v[0][0], v[0][1]);
                store_through(p + 2, v[0][2], v[0][3]);
                store_through(p + 16, v[1][0], v[1][1]);
                store_through(p + 18, v[1][2], v[1][3]);
              }
              arrive(u);
            });
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// rows staged in LDS for rows of K elements, and the bytes they take
int few_stage_rows(int T, int K) {
  const int row_bytes = mx_supers(K) * (kMxSuper * 2) + 16;
  const int fit = (64 << 10) / row_bytes;
  int n = T < kStageRows ? T : kStageRows;
  return n < fit ? n : fit;
}
unsigned few_stage_bytes(int T, int K) {
  return unsigned(few_stage_rows(T, K) * (mx_supers(K) * (kMxSuper * 2) + 16));
}

}  // namespace

size_t few_ws_bytes(int T, int k, int H, int I) {
  const size_t R = size_t(T) * k;
  return align256(size_t(H / 32) * 4) + align256(R * I * 2) + align256(R * H * 4);
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
  float* o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(h) + align256(size_t(R) * I * 2));
  const int upw1 = 1, upw2 = 1;
  const int runs1 = (I / 16 + upw1 - 1) / upw1, runs2 = (H / 32 + upw2 - 1) / upw2;
  with_route_slots(E, [&](auto ns) {
    hipLaunchKernelGGL((few_gate_up_kernel<decltype(ns)::value>), dim3(unsigned(R * runs1)),
                       dim3(kFewThreads), few_stage_bytes(T, H), stream, logits, bias, T, E, k,
                       renormalize, x, H, w13, ws13, I, upw1, few_stage_rows(T, H), ids, topk_w, h,
                       counters, H / 32);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(few_down_kernel, dim3(unsigned(R * runs2)), dim3(kFewThreads),
                     few_stage_bytes(T, I), stream, ids, topk_w, h, T, E, k, w2, ws2, H, I, upw2,
                     few_stage_rows(T, I), o, counters, shared, y);
  return hipGetLastError();
}

}  // namespace moeq
