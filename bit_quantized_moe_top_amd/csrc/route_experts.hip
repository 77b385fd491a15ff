// moe_route_experts: a token takes 64 or 16 lanes of a wave.
//
// Layout.  A group of experts lies on whole lanes, a power of two of them: with Gp the groups rounded
// up to a power of two, lane l of the token's holds experts sub C .. sub C + C - 1 of group l / (lanes /
// Gp), sub = l % (lanes / Gp), C = the group's experts per lane.  Lanes ascend with the expert index,
// so the lowest tied lane (then the lowest slot of it) is the lowest tied expert.  Without a group step
// (all groups stay) there is one group.
//
// Choice.  The order wanted is that of the real numbers c = s + bias.
//  * No bias: s grows with the logit, so experts are ordered by their logits, exactly.
//  * Bias: c is formed in fp32 within an error of tol / 2 (below).  The fp32 order of the k picks stands
//    if neighbours among them, and the last pick and every expert left, are at least tol apart or are
//    the same number (equal logit and equal bias, hence a tie that the index decides).  Otherwise the
//    experts within tol of the last pick or above it, the only ones the true choice can be among, are
//    ranked by their c in 64 bits.  Likewise for groups.  (Of random logits of unit variance
//    some 3 to 15 tokens in 10000; how many depends on the values, see WideChoice.)
//
// tol: with u = 2^-24, exp by the hardware's 2^x is within (1.5 |x| + 2) u of its value (the product
// with log2 e, its rounding, 1 ulp).  Sigmoid: s (1 - s) |l| < 0.23, so |ds| <= (0.9 + 1 + 2) u with the
// sum and the reciprocal.  Softmax: p |l - max| <= 0.37 pmax, pmax the largest score; its denominator's
// relative error is the p-weighted mean of (2.5 |x| + 2) u, |x| <= 7 on average for 1024 experts, plus
// NS + 6 roundings: |dp| <= 60 u pmax.  The sum with the bias: u |c|.  Twice that, and some: 2^-17 smax +
// 2^-22 |c| with smax = pmax, or 1/8 for sigmoid.
//
// Bound by VALU issue, a token's scores, sorts and k rounds against 2 or 4 E bytes read: 16384 tokens of
// 256 experts in 8 groups 14.1 us (17.8 MB, 1.3 TB/s; some 1300 vector instructions a wave of four
// tokens), 4096 of 1024 experts with a bias 13.3 us (0.65 TB/s; 1160 a wave of one, and the choice in 64
// bits at the end; without a bias 9.2), 64 of 256 3.8 us, a launch.
#include <algorithm>

#include "front.hpp"
#include "serve_kernels.hpp"

namespace moeq {

namespace {

constexpr int kRouteWaves = 4;                 // waves per workgroup
static_assert(MOEQ_MAX_TOPK <= 16, "a token's picks lie in the first 16 lanes");
constexpr int kDppRowShl1 = 0x101;             // lane i takes lane i + 1 of its 16
constexpr int kDppRowRor = 0x120;              // + n: lane i takes lane (i - n) % 16

// natural exponential by the hardware's 2^x
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
// key of a score (as score_key), at least 1 (one NaN's is 0) so that 0 marks "no candidate"
__device__ __forceinline__ uint32_t slot_key(float v) { return umax(score_key(v), 1u); }
__device__ __forceinline__ uint64_t wide_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t k = b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
  return k ? k : 1ull;
}
__device__ __forceinline__ uint64_t shfl64(uint64_t v, int from) {
  const int lo = __shfl(int(uint32_t(v)), from), hi = __shfl(int(uint32_t(v >> 32)), from);
  return uint64_t(uint32_t(lo)) | (uint64_t(uint32_t(hi)) << 32);
}
__device__ __forceinline__ double shfl64(double v, int from) {
  return __builtin_bit_cast(double, shfl64(__builtin_bit_cast(uint64_t, v), from));
}

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int from) {
  return uint64_t(uint32_t(readlane(int(uint32_t(v)), from))) |
         (uint64_t(uint32_t(readlane(int(uint32_t(v >> 32)), from))) << 32);
}

// score of a logit in fp32: softmax relative to `top`, times 1 / denominator
__device__ __forceinline__ float fast_score(float l, bool softmax, float top, float rden) {
  return softmax ? exp_fast(l - top) * rden : __builtin_amdgcn_rcpf(1.0f + exp_fast(-l));
}

// ---------------------------------------------------- the choice in 64 bits
// One token by a whole wave.  Rare, but a wave that comes here ends last: experts are read four a lane at
// a time and the candidates, taken from the sorted lists, are ranked side by side (4096 tokens of 1024
// experts, some six of them here: 13.3 us; with the candidates found by another pass over the row 15.3,
// one expert a lane at a time and a pass for each pick 18.5).  Few registers, for these are the whole
// kernel's: the row kept in them cost 16384 tokens of 256 experts a fifth.
template <typename LT>
struct WideChoice {
  const LT* row;
  const float* bias;
  const RouteShape& p;
  int lane;
  bool softmax;
  double top, den;                                       // softmax

  __device__ __forceinline__ WideChoice(const LT* row, const float* bias, const RouteShape& p, int lane,
                                        float ftop)
      : row(row), bias(bias), p(p), lane(lane), softmax(p.scoring == MOEQ_SCORE_SOFTMAX), top(ftop), den(1.0) {
    if (!softmax) return;
    den = 0.0;
    each(lane, kWave, p.E, [&](int, float l, float) { den += exp(double(l) - top); });
    for (int i = 1; i < kWave; i <<= 1) den += shfl64(den, lane ^ i);
  }
  // fn(expert, logit, bias) for the experts first, first + step, ... below end; past it the logit is
  // -inf, so that the wave's lanes stay together
  template <typename Fn>
  __device__ __forceinline__ void each(int first, int step, int end, Fn fn) const {
#pragma unroll 1
    for (int e0 = first; __ballot(e0 < end); e0 += 4 * step) {
      float l[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = min(e0 + step * j, p.E - 1);
        l[j] = load1(row + e);
        b[j] = bias ? bias[e] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = e0 + step * j;
        fn(e, e < end ? l[j] : -INFINITY, b[j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __device__ __forceinline__ double c(float l, float b) const {
    if (l == -INFINITY) return -INFINITY;
    return (softmax ? exp(double(l) - top) / den : 1.0 / (1.0 + exp(-double(l)))) + double(b);
  }

  // bit g: group g stays.  Groups lie on whole lanes, 2^shift of them.
  __device__ __forceinline__ uint64_t groups(int shift) const {
    const int S = p.E / p.n_group, C = (S + (1 << shift) - 1) >> shift;
    const int g = lane >> shift, at = (lane & ((1 << shift) - 1)) * C;
    const int first = g * S + at;
    double b1 = -INFINITY, b2 = -INFINITY;
    each(first, 1, g < p.n_group ? min(first + C, (g + 1) * S) : 0, [&](int, float l, float b) {
      const double x = c(l, b);
      b2 = fmax(b2, fmin(b1, x));
      b1 = fmax(b1, x);
    });
    for (int i = 0; i < shift; ++i) {
      const double o1 = shfl64(b1, lane ^ 1 << i), o2 = shfl64(b2, lane ^ 1 << i);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const uint64_t value = wide_key(p.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1);
    const uint64_t mine = shfl64(value, lane << shift & 63);             // lane g: group g's
    int above = 0;
    for (int o = 0; o < p.n_group; ++o) {
      const uint64_t other = readlane64(mine, o);
      above += other > mine || (other == mine && o < lane);
    }
    return __ballot(lane < p.n_group && above < p.topk_group);
  }

  // The k best of n <= 64 candidates in LDS, which are overwritten: lane r returns the r-th (-1: there
  // are fewer).
  __device__ __forceinline__ int ranked(int* cand, int n) const {
    const int e = lane < n ? cand[lane] : 0;
    const uint64_t key = lane < n ? wide_key(c(load1(row + e), bias[e])) : 0;
    int rank = 0;
    for (int i = 0; i < n; ++i) {
      const uint64_t other = readlane64(key, i);
      rank += other > key || (other == key && readlane(e, i) < e);
    }
    lds_wave_sync();
    if (lane < n && rank < p.k) cand[rank] = e;
    lds_wave_sync();
    return lane < min(n, p.k) ? cand[lane] : -1;
  }
  // The same of all experts whose fp32 sum is above `edge` in the groups of `stay`, however many they
  // are: round by round, the best after the last taken.  Every token of a peaked softmax comes here where
  // the bias is as small as the other scores (one score near 1, the others some 2e-9 and a bias of 1e-7:
  // all sums lie within 2^-17 of each other): 4096 tokens of 1024 experts 127 us, 16384 of 256 145, 64 of
  // 256 23; with a bias of 1e-3 10 to 16.
  __device__ __forceinline__ int rounds(uint64_t stay, float edge, float rden) const {
    const int S = p.E / p.n_group;
    uint64_t last = ~0ull;
    int last_e = -1, mine = -1;
    for (int r = 0; r < p.k; ++r) {
      uint64_t best = 0;
      int at = -1;
      each(lane, kWave, p.E, [&](int e, float l, float b) {
        const bool in = l != -INFINITY && !(fast_score(l, softmax, float(top), rden) + b <= edge) &&
                        (stay >> (e / S & 63) & 1);
        const uint64_t key = in ? wide_key(c(l, b)) : 0;
        if ((key < last || (key == last && e > last_e)) && key > best) {
          best = key;
          at = e;
        }
      });
      for (int i = 1; i < kWave; i <<= 1) {
        const uint64_t o = shfl64(best, lane ^ i);
        const int oe = __shfl(at, lane ^ i);
        if (o > best || (o == best && oe < at)) {
          best = o;
          at = oe;
        }
      }
      last = best;
      last_e = at;
      if (lane == r) mine = at;
    }
    return mine;
  }
};

// where a lane's experts are
struct Lanes {
  int g, first, n;            // the lane's group, its first expert, its experts
};
// the shape's layout on the token's lanes, made by the host
struct RouteLayout {
  int G, S, C;                // groups (1 without a group step), experts per group and per lane
  int shift;                  // log2 of the lanes per group
  int whole;                  // every lane with experts has NS of them, aligned for wide loads
  __device__ __forceinline__ Lanes lanes(int sub) const {
    Lanes ln;
    ln.g = sub >> shift;
    const int at = (sub & ((1 << shift) - 1)) * C;
    ln.first = ln.g * S + at;
    ln.n = ln.g < G ? min(max(S - at, 0), C) : 0;
    if (ln.n == 0) ln.first = 0;
    return ln;
  }
};

// NS values of consecutive experts; `whole`: NS of them, 4-element aligned (bf16: 8 bytes)
template <int NS>
__device__ __forceinline__ void load_slots(const float* p, int n, bool whole, float (&v)[NS]) {
  if (NS >= 4 && whole) {
#pragma unroll
    for (int j = 0; j < NS / 4; ++j) {
      const float4 f = reinterpret_cast<const float4*>(p)[j];
      v[4 * j] = f.x; v[4 * j + 1 < NS ? 4 * j + 1 : 0] = f.y;
      v[4 * j + 2 < NS ? 4 * j + 2 : 0] = f.z; v[4 * j + 3 < NS ? 4 * j + 3 : 0] = f.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) v[j] = p[min(j, max(n - 1, 0))];
}
template <int NS>
__device__ __forceinline__ void load_slots(const uint16_t* p, int n, bool whole, float (&v)[NS]) {
  if (NS >= 4 && whole) {
#pragma unroll
    for (int j = 0; j < NS / 4; ++j) {
      const uint2 u = reinterpret_cast<const uint2*>(p)[j];
      v[4 * j] = u2f(u.x << 16); v[4 * j + 1 < NS ? 4 * j + 1 : 0] = u2f(u.x & 0xFFFF0000u);
      v[4 * j + 2 < NS ? 4 * j + 2 : 0] = u2f(u.y << 16);
      v[4 * j + 3 < NS ? 4 * j + 3 : 0] = u2f(u.y & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) v[j] = bf16_to_f32(p[min(j, max(n - 1, 0))]);
}

// (b1, b2), b1 >= b2, of two lanes joined
__device__ __forceinline__ void join2(uint32_t& b1, uint32_t& b2, uint32_t o1, uint32_t o2) {
  b2 = umax(umin(b1, o1), umax(b2, o2));
  b1 = umax(b1, o1);
}
template <int CTRL>
__device__ __forceinline__ void join2_dpp(uint32_t& b1, uint32_t& b2) {
  join2(b1, b2, uint32_t(dpp<CTRL>(0, int(b1))), uint32_t(dpp<CTRL>(0, int(b2))));
}

// The W lanes of a token, W = 64 (a wave per token) or 16 (a DPP row).
template <int W>
struct Token {
  static_assert(W == 64 || W == 16, "a wave or a row");
  template <typename T, typename Op>
  static __device__ __forceinline__ T reduce(T v, Op op, T ident) {
    if constexpr (W == 64) {
      return wave_reduce(v, op, ident);
    } else {
      v = op(v, dpp<kDppQuadSwap1>(ident, v));
      v = op(v, dpp<kDppQuadSwap2>(ident, v));
      v = op(v, dpp<kDppRowHalfMirror>(ident, v));
      return op(v, dpp<kDppRowMirror>(ident, v));
    }
  }
  static __device__ __forceinline__ float max(float v) {
    return reduce(v, [](float a, float b) { return fmaxf(a, b); }, -INFINITY);
  }
  static __device__ __forceinline__ float sum(float v) {
    return reduce(v, [](float a, float b) { return a + b; }, 0.0f);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t v) {
    return uint32_t(reduce(int(v), [](int a, int b) { return int(umax(uint32_t(a), uint32_t(b))); }, 0));
  }
  // bit i: the condition of the token's lane i
  static __device__ __forceinline__ uint64_t ballot(bool v, int lane) {
    const uint64_t b = __ballot(v);
    return W == 64 ? b : b >> (lane & 48) & 0xFFFFu;
  }
  // the value of the token's lane i (the same i in every lane)
  template <typename T>
  static __device__ __forceinline__ T from(T v, int i, int lane) {
    if constexpr (W == 64) return readlane(v, i);
    else return __shfl(v, (lane & 48) + i);
  }
};

// A lane's experts as sorted lists of up to four (best first, the lower slot among equals), so that a
// round of the selection looks at the heads only and taking one is a shift.  `order` holds a list's
// slots, a byte each.
template <int NS>
struct SortedSlots {
  static constexpr int kLen = NS < 4 ? NS : 4, kLists = NS / kLen;
  uint32_t key[kLists][kLen], order[kLists];
  __device__ __forceinline__ void sort(const uint32_t (&k)[NS]) {
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
#pragma unroll
      for (int j = 0; j < kLen; ++j) key[i][j] = k[kLen * i + j];
      order[i] = 0x03020100u;
      // neighbours exchanged only where the later is larger: equal keys keep their order
#pragma unroll
      for (int end = 1; end < kLen; ++end)
#pragma unroll
        for (int j = end; j > 0; --j) exchange(i, j - 1);
    }
  }
  // bytes j and j + 1 of `order` change places with the keys
  __device__ __forceinline__ void exchange(int i, int j) {
    const bool swap = key[i][j + 1] > key[i][j];
    const uint32_t a = key[i][j], b = key[i][j + 1];
    key[i][j] = swap ? b : a;
    key[i][j + 1] = swap ? a : b;
    const uint32_t sel = j == 0 ? 0x03020001u : j == 1 ? 0x03010200u : 0x02030100u;
    const uint32_t moved = __builtin_amdgcn_perm(0u, order[i], sel);
    order[i] = swap ? moved : order[i];
  }
  // the best left: its key, and its slot in `slot`
  __device__ __forceinline__ uint32_t best(int& slot, int& list) const {
    uint32_t k = key[0][0], o = order[0];
    list = 0;
#pragma unroll
    for (int i = 1; i < kLists; ++i) {
      const bool more = key[i][0] > k;
      k = more ? key[i][0] : k;
      o = more ? order[i] : o;
      list = more ? i : list;
    }
    slot = kLen * list + int(o & 255u);
    return k;
  }
  // takes the head of the lane's own `list`
  __device__ __forceinline__ void take_own(int list) {
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
      const bool it = i == list;
#pragma unroll
      for (int j = 0; j + 1 < kLen; ++j) key[i][j] = it ? key[i][j + 1] : key[i][j];
      key[i][kLen - 1] = it ? 0u : key[i][kLen - 1];
      order[i] = it ? order[i] >> 8 : order[i];
    }
  }
  // takes the head of `list` (wave-uniform)
  __device__ __forceinline__ void take(int list) {
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
      if (i != list) continue;
#pragma unroll
      for (int j = 0; j + 1 < kLen; ++j) key[i][j] = key[i][j + 1];
      key[i][kLen - 1] = 0u;
      order[i] >>= 8;
    }
  }
};

// W = 64: tokens are few or their experts many.  W = 16: four tokens share a wave's instructions, but
// a lane's lists are four times as many.
template <typename LT, int W, int NS>
__global__ void __launch_bounds__(64 * kRouteWaves)
route_experts_kernel(const LT* __restrict__ logits, const float* __restrict__ bias, RouteShape p,
                     RouteLayout lay, int32_t* __restrict__ ids, float* __restrict__ w) {
  using Tok = Token<W>;
  constexpr int kTokens = kWave / W;                         // of a wave
  __shared__ int s_cand[kRouteWaves][kWave];
  const int lane = threadIdx.x & 63, sub = lane & (W - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = (blockIdx.x * kRouteWaves + wave) * kTokens;
  if (t0 >= p.T) return;                                     // whole wave exits together
  const int t = W == 64 ? t0 : min(t0 + lane / W, p.T - 1);  // (past the end the last token again)
  const bool grouped = p.topk_group < p.n_group;
  const bool softmax = p.scoring == MOEQ_SCORE_SOFTMAX;
  const Lanes ln = lay.lanes(sub);
  const LT* row = logits + int64_t(t) * p.ld;

  float l[NS], c[NS];
  load_slots<NS>(row + ln.first, ln.n, lay.whole, l);
  if (bias) load_slots<NS>(bias + ln.first, ln.n, lay.whole, c);
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (j >= ln.n) l[j] = -INFINITY;

  // softmax: largest logit and denominator over all experts
  float top = 0.0f, den = 1.0f;
  if (softmax) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NS; ++j) m = fmaxf(m, l[j]);
    top = Tok::max(m);
    if (top == -INFINITY) top = 0.0f;                        // every expert masked
    if (bias || !p.renormalize || (grouped && p.group_best == 2)) {
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) part += exp_fast(l[j] - top);
      den = Tok::sum(part);
    }
  }

  // keys that order experts: c, or without a bias the logits (the fp32 scores are then needed for
  // sums of two in groups only)
  const bool by_logit = bias == nullptr;
  const bool scores = !by_logit || (grouped && p.group_best == 2);
  const float rden = softmax ? 1.0f / den : 1.0f;
  const float smax = softmax ? rden : 0.125f;
  const uint32_t none = score_key(-INFINITY);
  uint32_t key[NS];
  if (scores) {
    if (by_logit) {
#pragma unroll
      for (int j = 0; j < NS; ++j) c[j] = 0.0f;
    }
    if (softmax) {
#pragma unroll
      for (int j = 0; j < NS; ++j) c[j] = l[j] == -INFINITY ? -INFINITY : fast_score(l[j], true, top, rden) + c[j];
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) c[j] = l[j] == -INFINITY ? -INFINITY : fast_score(l[j], false, top, rden) + c[j];
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) key[j] = j < ln.n ? slot_key(c[j]) : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) key[j] = j < ln.n ? slot_key(l[j]) : 0u;
  }

  bool stays = true;
  if (grouped) {
    uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      b2 = umax(b2, umin(b1, key[j]));
      b1 = umax(b1, key[j]);
    }
    if (lay.shift > 0) join2_dpp<kDppQuadSwap1>(b1, b2);
    if (lay.shift > 1) join2_dpp<kDppQuadSwap2>(b1, b2);
    if (lay.shift > 2) join2_dpp<kDppRowHalfMirror>(b1, b2);
    if (W == 64 && lay.shift > 3) join2_dpp<kDppRowMirror>(b1, b2);
    if (W == 64 && lay.shift > 4)
      join2(b1, b2, uint32_t(__shfl_xor(int(b1), 16)), uint32_t(__shfl_xor(int(b2), 16)));
    if (ln.g >= lay.G) b1 = b2 = 0u;
    const bool live = b1 > none;
    const bool two = p.group_best == 2 && b2 > none;
    const float f1 = key_score(b1), f2 = two ? key_score(b2) : 0.0f;
    // (of sums half their value: that of two biases at either end of fp32 passes it)
    const float mid = scores ? 0.5f * f1 + 0.5f * f2 : f1;
    const float half = scores ? 0x1p-18f * smax + 0x1p-23f * fabsf(f1) + 0x1p-23f * fabsf(f2) : 0.0f;
    const float lo = mid - half;
    const float hi = live ? mid + half : -INFINITY;
    // A group stays for sure if at most topk_group - 1 others may be above it.  If as many stay for
    // sure as are to stay, the choice is made.  (The best of the logits are exact: equal ones count
    // if their group is lower.)
    int maybe = 0;                                           // groups, itself among them
    if constexpr (W == 64) {
      for (int g = 0; g < lay.G; ++g) {
        const float other = readlane(hi, g << lay.shift);
        maybe += other > lo || (other == lo && (scores || g <= ln.g)) ? 1 : 0;
      }
    } else {                                                 // a lane of each group, by rotation of the row
      const auto count = [&](auto n) {
        const float other = dpp<kDppRowRor + decltype(n)::value>(0.0f, hi);
        const int og = ((sub - decltype(n)::value) & 15) >> lay.shift;
        maybe += other > lo || (other == lo && (scores || og <= ln.g)) ? 1 : 0;
      };
      maybe += hi >= lo ? 1 : 0;
      count(SlotsTag<8>{});
      if (lay.shift <= 2) {
        count(SlotsTag<4>{}); count(SlotsTag<12>{});
      }
      if (lay.shift <= 1) {
        count(SlotsTag<2>{}); count(SlotsTag<6>{}); count(SlotsTag<10>{}); count(SlotsTag<14>{});
      }
      if (lay.shift == 0) {
        count(SlotsTag<1>{}); count(SlotsTag<3>{}); count(SlotsTag<5>{}); count(SlotsTag<7>{});
        count(SlotsTag<9>{}); count(SlotsTag<11>{}); count(SlotsTag<13>{}); count(SlotsTag<15>{});
      }
    }
    const bool lead = ln.g < lay.G && sub == ln.g << lay.shift;
    const int n_live = __popcll(Tok::ballot(live && lead, lane));
    // empty groups: after all the others, the lower first
    const uint64_t empty = Tok::ballot(!live && lead, lane);
    stays = live ? maybe <= p.topk_group
                 : n_live + __popcll(empty & ((uint64_t(1) << (ln.g << lay.shift & 63)) - 1)) < p.topk_group;
    const bool open = __popcll(Tok::ballot(stays && live && lead, lane)) < min(p.topk_group, n_live);
    for (uint64_t tokens = __ballot(open && sub == 0); tokens; tokens &= tokens - 1) {
      const int at = __ffsll(static_cast<unsigned long long>(tokens)) - 1;     // the token's first lane
      const WideChoice<LT> wide(logits + int64_t(min(t0 + at / W, p.T - 1)) * p.ld, bias, p, lane,
                                __shfl(top, at));
      const uint64_t stay = wide.groups(lay.shift + (W == 64 ? 0 : 2));
      if (lane / W == at / W) stays = stay >> (ln.g & 63) & 1;
    }
    if (scores && by_logit) {
#pragma unroll
      for (int j = 0; j < NS; ++j) key[j] = j < ln.n ? slot_key(l[j]) : 0u;
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) key[j] = stays ? key[j] : umin(key[j], none);
  }

  // k rounds of an argmax over the heads
  SortedSlots<NS> left;
  left.sort(key);
  int e = 0, ekey = 0;                                       // lane r: the r-th pick and its key
  for (int r = 0; r < p.k; ++r) {
    int slot, list;
    const uint32_t mine = left.best(slot, list);
    const uint32_t kmax = Tok::max(mine);
    if constexpr (W == 64) {
      const int from = __ffsll(static_cast<unsigned long long>(__ballot(mine == kmax))) - 1;
      const int be = readlane(ln.first + slot, from);
      const int from_list = SortedSlots<NS>::kLists > 1 ? readlane(list, from) : 0;
      if (lane == from) left.take(from_list);
      e = lane == r ? be : e;
      ekey = lane == r ? int(kmax) : ekey;
    } else {
      // the row's lowest lane at the maximum takes its head and leaves the expert in LDS
      const uint64_t tied = Tok::ballot(mine == kmax, lane);
      if ((tied & ((2u << sub) - 1u)) == (1u << sub)) {
        s_cand[wave][(lane & 48) + r] = ln.first + slot;
        left.take_own(list);
      }
      ekey = sub == r ? int(kmax) : ekey;
    }
  }
  if constexpr (W == 16) {
    lds_wave_sync();
    e = sub < p.k ? s_cand[wave][lane] : 0;
    lds_wave_sync();
  }
  const bool pick = sub < p.k;
  float el = load1(row + e);
  bool live = pick && uint32_t(ekey) > none;

  if (!by_logit) {
    // does the fp32 order stand?
    const float ec = key_score(uint32_t(ekey)), eb = bias[e];
    const float tol = 0x1p-17f * smax + 0x1p-22f * fabsf(ec);
    const float nc = dpp<kDppRowShl1>(0.0f, ec), nl = dpp<kDppRowShl1>(0.0f, el), nb = dpp<kDppRowShl1>(0.0f, eb);
    const bool nlive = dpp<kDppRowShl1>(0, int(live)) != 0;
    bool open = live && nlive && sub + 1 < p.k && ec - nc < tol && !(nl == el && nb == eb);
    const int last = p.k - 1;
    const bool last_live = Tok::from(int(live), last, lane) != 0;
    const float edge = last_live ? Tok::from(ec - tol, last, lane) : -INFINITY;
    const uint32_t edge_key = last_live ? umax(score_key(edge), none) : 0xFFFFFFFFu;
    bool near = false;
#pragma unroll
    for (int i = 0; i < SortedSlots<NS>::kLists; ++i) near |= left.key[i][0] > edge_key;
    if (__ballot(near)) {                                    // equal to the last pick in both parts?
      const float ll = Tok::from(el, last, lane), lb = Tok::from(eb, last, lane);
#pragma unroll
      for (int i = 0; i < SortedSlots<NS>::kLists; ++i)
#pragma unroll
        for (int j = 0; j < SortedSlots<NS>::kLen; ++j)
          if (left.key[i][j] > edge_key) {
            const int at = ln.first + SortedSlots<NS>::kLen * i + int(left.order[i] >> (8 * j) & 255u);
            open |= !(load1(row + at) == ll && bias[at] == lb);
          }
    }
    if (__ballot(open)) {
      // candidates: the picks that have a score and the experts within tol of the last one or above it,
      // W at most in LDS
      int n = 0;
      const auto add = [&](bool take, int expert) {
        const uint64_t takers = Tok::ballot(take, lane);
        const int to = n + __popcll(takers & ((uint64_t(1) << sub) - 1));
        if (take && to < W) s_cand[wave][(lane & ~(W - 1)) + to] = expert;
        n += __popcll(takers);
      };
      add(live, e);
      if (__ballot(near)) {
#pragma unroll
        for (int i = 0; i < SortedSlots<NS>::kLists; ++i)
#pragma unroll
          for (int j = 0; j < SortedSlots<NS>::kLen; ++j)
            add(left.key[i][j] > edge_key,
                ln.first + SortedSlots<NS>::kLen * i + int(left.order[i] >> (8 * j) & 255u));
      }
      lds_wave_sync();
      // tokens in turn, each by the whole wave
      for (int i = 0; i < kTokens; ++i) {
        const uint64_t mine = W == 64 ? ~0ull : uint64_t(0xFFFFu) << (16 * i);
        if ((__ballot(open) & mine) == 0) continue;
        const WideChoice<LT> wide(logits + int64_t(min(t0 + i, p.T - 1)) * p.ld, bias, p, lane,
                                  readlane(top, W * i));
        const int m = readlane(n, W * i);
        int got;
        if (m <= W) {
          got = wide.ranked(s_cand[wave] + W * i, m);
        } else {
          uint64_t stay = ~0ull;                             // groups of the public numbering
          if (grouped) {
            const uint64_t lanes = __ballot(stays) >> (W * i & 63);
            stay = 0;
            for (int g = 0; g < lay.G; ++g) stay |= (lanes >> (g << lay.shift) & 1) << g;
          }
          got = wide.rounds(stay, readlane(edge, W * i), readlane(rden, W * i));
        }
        // (as many as have a score: with a NaN among the values not always, and then the fp32 picks,
        // which are distinct, stay)
        const bool all = __popcll(__ballot(got >= 0)) == __popcll(__ballot(live) & mine);
        got = __shfl(got, lane & (W - 1));
        if (lane / W == i && pick && got >= 0 && all) {
          e = got;
          el = load1(row + e);
        }
      }
    }
  }

  // weights, lane r the r-th expert's: sigmoid scores 1 / (1 + exp(-l)); where only their ratios
  // count and all are below 1/2 the common factor exp(max l) is left out, so that none
  // underflows.  Softmax scores relative to the largest chosen, or to the largest of all.
  const float lmax = Tok::max(live ? el : -INFINITY);
  float s = 0.0f;
  if (live) {
    if (softmax)
      s = expf(el - (p.renormalize ? lmax : top));
    else if (p.renormalize && lmax < 0.0f)
      s = expf(el - lmax) / (1.0f + expf(el));
    else
      s = 1.0f / (1.0f + expf(-el));
  }
  const float sum = p.renormalize ? Tok::sum(s) : den;
  if (pick && (W == 64 || t0 + lane / W < p.T)) {
    ids[int64_t(t) * p.k + sub] = e;
    w[int64_t(t) * p.k + sub] = live ? s / sum * p.scale : 0.0f;
  }
}

// the layout on W lanes (W not enough for the groups: C = 0)
RouteLayout route_layout(const RouteShape& s, int W) {
  RouteLayout at;
  at.G = s.topk_group < s.n_group ? s.n_group : 1;
  at.S = s.E / at.G;
  at.shift = 0;
  while ((W >> at.shift) > 1 && at.G <= (W >> (at.shift + 1))) ++at.shift;
  at.C = at.G <= W ? (at.S + (1 << at.shift) - 1) >> at.shift : 0;
  at.whole = 0;
  return at;
}

template <typename LT, int W, int NS>
hipError_t launch_slots(const LT* logits, const float* bias, const RouteShape& s, RouteLayout at,
                        int32_t* ids, float* w, hipStream_t stream) {
  at.whole = at.C == NS && at.S % NS == 0 && s.ld % 4 == 0 &&
             reinterpret_cast<uintptr_t>(logits) % (4 * sizeof(LT)) == 0 &&
             reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  constexpr int kPerBlock = kRouteWaves * (kWave / W);
  hipLaunchKernelGGL((route_experts_kernel<LT, W, NS>), dim3(unsigned((s.T + kPerBlock - 1) / kPerBlock)),
                     dim3(64 * kRouteWaves), 0, stream, logits, bias, s, at, ids, w);
  return hipGetLastError();
}

// Four tokens a wave from this many tokens on for each expert of a lane: before that there are fewer
// waves than SIMDs want, and one takes longer.  us at 1024 / 2048 / 4096 / 8192 / 16384 tokens, four
// against one: 64 experts 3.5 / 3.5 / 3.5 / 3.7 / 5.0 against 3.4 / 3.6 / 4.4 / 6.2 / 10.3; 128 with a
// bias 5.0 / 5.4 / 6.0 / 7.3 / 9.6 against 4.3 / 4.7 / 5.8 / 8.5 / 13.7; 256 in 8 groups 6.8 / 7.5 / 8.3 /
// 10.5 / 13.9 against 5.2 / 5.8 / 7.5 / 11.7 / 18.5.
constexpr int kShareTokens = 512;

template <typename LT>
hipError_t launch_typed(const LT* logits, const float* bias, const RouteShape& s, int32_t* ids,
                        float* w, hipStream_t stream) {
  RouteLayout at = route_layout(s, 16);
  if (at.C >= 1 && at.C <= 16 && s.T >= kShareTokens * std::max(at.C, 4)) {
    if (at.C <= 4) return launch_slots<LT, 16, 4>(logits, bias, s, at, ids, w, stream);
    if (at.C <= 8) return launch_slots<LT, 16, 8>(logits, bias, s, at, ids, w, stream);
    return launch_slots<LT, 16, 16>(logits, bias, s, at, ids, w, stream);
  }
  at = route_layout(s, 64);
  if (at.C <= 1) return launch_slots<LT, 64, 1>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 2) return launch_slots<LT, 64, 2>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 4) return launch_slots<LT, 64, 4>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 8) return launch_slots<LT, 64, 8>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 16) return launch_slots<LT, 64, 16>(logits, bias, s, at, ids, w, stream);
  return launch_slots<LT, 64, 32>(logits, bias, s, at, ids, w, stream);   // C <= 31: E <= 1024
}

}  // namespace

hipError_t launch_route_experts(const void* logits, int logits_dtype, const float* bias,
                                const RouteShape& shape, int32_t* ids, float* w,
                                hipStream_t stream) {
  if (shape.T == 0) return hipSuccess;
  if (logits_dtype == MOEQ_BF16)
    return launch_typed(static_cast<const uint16_t*>(logits), bias, shape, ids, w, stream);
  return launch_typed(static_cast<const float*>(logits), bias, shape, ids, w, stream);
}

}  // namespace moeq
