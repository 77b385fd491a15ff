// moe_route_experts: one wave64 per token.
//
// Layout.  A group of experts lies on whole lanes, a power of two of them: with Gp the
// groups rounded up to a power of two, lane l holds experts sub C .. sub C + C - 1 of
// group l / (64 / Gp), sub = l % (64 / Gp), C = the group's experts per lane.  Lanes
// ascend with the expert index, so the lowest tied lane (then the lowest slot of it)
// is the lowest tied expert.  Without a group step (all groups stay) there is one group.
//
// Choice.  The order wanted is that of the real numbers c = s + bias.
//  * No bias: s grows with the logit, so experts are ordered by their logits, exactly.
//  * Bias: c is formed in fp32 within an error of tol / 2 (below).  The fp32 order of the k
//    picks stands if neighbours among them, and the last pick and every expert left, are
//    at least tol apart or are the same number (equal logit and equal bias, hence a tie
//    that the index decides).  Otherwise, and likewise for groups, the wave computes the
//    token's c in 64 bits into LDS and picks there.
//
// tol: with u = 2^-24, exp by the hardware's 2^x is within (1.5 |x| + 2) u of its value
// (the product with log2 e, its rounding, 1 ulp).  Sigmoid: s (1 - s) |l| < 0.23, so
// |ds| <= (0.9 + 1 + 2) u with the sum and the reciprocal.  Softmax: p |l - max| <= 0.37
// pmax, pmax the largest score; its denominator's relative error is the p-weighted mean of
// (2.5 |x| + 2) u, |x| <= 7 on average for 1024 experts, plus NS + 6 roundings: |dp| <=
// 60 u pmax.  The sum with the bias: u |c|.  Twice that, and some: 2^-17 smax + 2^-22 |c|
// with smax = pmax, or 1/8 for sigmoid.
#include "front.hpp"
#include "serve_kernels.hpp"

namespace moeq {

namespace {

constexpr int kRouteWaves = 4;                 // tokens per workgroup

// natural exponential by the hardware's 2^x
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }

// order-preserving key of a double (as score_key), at least 1 so that 0 marks "no candidate"
__device__ __forceinline__ uint64_t wide_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t k = b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
  return k ? k : 1ull;
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
  const int lo = __shfl_xor(int(uint32_t(v)), m), hi = __shfl_xor(int(uint32_t(v >> 32)), m);
  return uint64_t(uint32_t(lo)) | (uint64_t(uint32_t(hi)) << 32);
}
__device__ __forceinline__ double shfl_xor64(double v, int m) {
  return __builtin_bit_cast(double, shfl_xor64(__builtin_bit_cast(uint64_t, v), m));
}

// where a lane's experts are
struct Lanes {
  int G, S, C;                // groups (1 without a group step), experts per group and per lane
  int width;                  // lanes per group
  int g, first, n;            // this lane's group, its first expert, its experts
  __device__ __forceinline__ Lanes(const RouteShape& s, bool grouped, int c, int w, int lane)
      : G(grouped ? s.n_group : 1), S(s.E / G), C(c), width(w) {
    g = lane / width;
    const int at = (lane - g * width) * C;
    first = g * S + at;
    n = g < G ? min(max(S - at, 0), C) : 0;
    if (n == 0) first = 0;
  }
};

// The token's choice in 64 bits, for the lanes' experts: keys in LDS at [slot][lane].
template <typename LT>
struct WideChoice {
  uint64_t* keys;
  const Lanes& ln;
  int lane;

  // c of every expert, and the lane's two best unmasked (-inf: none)
  __device__ __forceinline__ void fill(const LT* row, const float* bias, int scoring, double& b1,
                                       double& b2) {
    double top = 0.0, den = 1.0;
    if (scoring == MOEQ_SCORE_SOFTMAX) {
      top = -INFINITY;
#pragma unroll 1
      for (int j = 0; j < ln.n; ++j) top = fmax(top, double(load1(row + ln.first + j)));
      for (int m = 1; m < kWave; m <<= 1) top = fmax(top, shfl_xor64(top, m));
      double part = 0.0;
#pragma unroll 1
      for (int j = 0; j < ln.n; ++j) part += exp(double(load1(row + ln.first + j)) - top);
      for (int m = 1; m < kWave; m <<= 1) part += shfl_xor64(part, m);
      den = part;
    }
    b1 = b2 = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < ln.n; ++j) {
      const float l = load1(row + ln.first + j);
      const double s = scoring == MOEQ_SCORE_SOFTMAX ? exp(double(l) - top) / den
                                                     : 1.0 / (1.0 + exp(-double(l)));
      double c = bias ? s + double(bias[ln.first + j]) : s;
      if (l == -INFINITY) c = -INFINITY;
      keys[j * kWave + lane] = wide_key(c);
      if (c > b1) { b2 = b1; b1 = c; }
      else if (c > b2) b2 = c;
    }
  }

  // whether the lane's group stays
  __device__ __forceinline__ bool group_stays(double b1, double b2, int best, int topk_group) const {
    for (int m = 1; m < ln.width; m <<= 1) {
      const double o1 = shfl_xor64(b1, m), o2 = shfl_xor64(b2, m);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const double v = best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    const uint64_t key = wide_key(v);
    int above = 0;
    for (int g = 0; g < ln.G; ++g) {
      const uint32_t lo = uint32_t(readlane(int(uint32_t(key)), g * ln.width));
      const uint32_t hi = uint32_t(readlane(int(uint32_t(key >> 32)), g * ln.width));
      const uint64_t other = uint64_t(lo) | (uint64_t(hi) << 32);
      above += other > key || (other == key && g < ln.g);
    }
    return above < topk_group;
  }

  // the k best; lane r returns the r-th
  __device__ __forceinline__ int pick(bool stays, int k, bool* live) {
    const uint64_t none = wide_key(-INFINITY);
    int mine = 0;
    *live = false;
    for (int r = 0; r < k; ++r) {
      uint64_t best = 0;
      int at = 0;
#pragma unroll 1
      for (int j = 0; j < ln.n; ++j) {
        uint64_t key = keys[j * kWave + lane];
        if (!stays && key != 0) key = none;
        if (key > best) { best = key; at = j; }
      }
      uint64_t top = best;
      for (int m = 1; m < kWave; m <<= 1) {
        const uint64_t o = shfl_xor64(top, m);
        top = o > top ? o : top;
      }
      const int from = __ffsll(static_cast<unsigned long long>(__ballot(best == top))) - 1;
      const int e = readlane(ln.first + at, from);
      if (lane == from) keys[at * kWave + lane] = 0;
      if (lane == r) {
        mine = e;
        *live = top > none;
      }
    }
    return mine;
  }
};

template <typename LT, int NS>
__global__ void __launch_bounds__(64 * kRouteWaves)
route_experts_kernel(const LT* __restrict__ logits, const float* __restrict__ bias, RouteShape p,
                     int C, int width, int32_t* __restrict__ ids, float* __restrict__ w) {
  extern __shared__ __align__(16) uint64_t wide_keys[];      // [waves][NS][64] where needed
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;                                      // whole wave exits together
  const bool grouped = p.topk_group < p.n_group;
  const bool softmax = p.scoring == MOEQ_SCORE_SOFTMAX;
  const Lanes ln(p, grouped, C, width, lane);
  const LT* row = logits + int64_t(t) * p.ld;

  // every load issued before the first use, clamped instead of branched around
  float l[NS], c[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) l[j] = load1(row + ln.first + min(j, max(ln.n - 1, 0)));
#pragma unroll
  for (int j = 0; j < NS; ++j) c[j] = bias ? bias[ln.first + min(j, max(ln.n - 1, 0))] : 0.0f;
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (j >= ln.n) l[j] = -INFINITY;

  // softmax: largest logit and denominator over all experts
  float top = 0.0f, den = 1.0f;
  if (softmax) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NS; ++j) m = fmaxf(m, l[j]);
    top = wave_reduce(m, [](float a, float b) { return fmaxf(a, b); }, -INFINITY);
    if (top == -INFINITY) top = 0.0f;                        // every expert masked
    if (bias || !p.renormalize || (grouped && p.group_best == 2)) {
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) part += exp_fast(l[j] - top);
      den = wave_sum(part);
    }
  }

  // what orders experts (without a bias the logits) and groups
  const bool by_logit = bias == nullptr;
  const bool scores = !by_logit || (grouped && p.group_best == 2);
  const float rden = softmax ? 1.0f / den : 1.0f;
  const float smax = softmax ? rden : 0.125f;
  if (scores) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float s = softmax ? exp_fast(l[j] - top) * rden
                              : __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[j]));
      c[j] = l[j] == -INFINITY ? -INFINITY : s + c[j];
    }
  }

  WideChoice<LT> wide{wide_keys + size_t(wave) * NS * kWave, ln, lane};
  bool filled = false;
  double w1 = 0.0, w2 = 0.0;
  bool stays = true;
  if (grouped) {
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float v = j < ln.n ? (scores ? c[j] : l[j]) : -INFINITY;
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
    }
    for (int m = 1; m < width; m <<= 1) {
      const float o1 = __shfl_xor(b1, m), o2 = __shfl_xor(b2, m);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    }
    if (!scores) {                                           // best of the logits: exact
      const uint32_t key = max(score_key(b1), 1u);
      int above = 0;
      for (int g = 0; g < ln.G; ++g) {
        const uint32_t other = uint32_t(readlane(int(key), g * width));
        above += other > key || (other == key && g < ln.g);
      }
      stays = above < p.topk_group;
    } else {
      const bool two = p.group_best == 2 && b2 > -INFINITY;
      const float v = two ? b1 + b2 : b1;
      const float half = 0x1p-17f * smax + 0x1p-22f * (fabsf(b1) + (two ? fabsf(b2) : 0.0f));
      const bool live = b1 > -INFINITY;
      const float lo = live ? v - half : -INFINITY, hi = live ? v + half : -INFINITY;
      int sure = 0, maybe = 0, empty_below = 0, n_live = 0;
      for (int g = 0; g < ln.G; ++g) {
        const float olo = readlane(lo, g * width), ohi = readlane(hi, g * width);
        const bool olive = ohi > -INFINITY;
        sure += olo > hi;
        maybe += ohi >= lo && g != ln.g;
        n_live += olive;
        empty_below += !olive && g < ln.g;
      }
      stays = live ? maybe < p.topk_group : n_live + empty_below < p.topk_group;
      const bool open = live && !stays && sure < p.topk_group && ln.g < ln.G;
      if (__ballot(open)) {
        wide.fill(row, bias, p.scoring, w1, w2);
        filled = true;
        stays = wide.group_stays(w1, w2, p.group_best, p.topk_group);
      }
    }
  }

  // k rounds of a wave-wide argmax
  uint32_t key[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const float v = stays ? (by_logit ? l[j] : c[j]) : -INFINITY;
    key[j] = j < ln.n ? max(score_key(v), 1u) : 0u;
  }
  int e = 0;
  uint32_t ekey = 0;
  for (int r = 0; r < p.k; ++r) {
    uint32_t ck = 0;
    int cj = 0;
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (key[j] > ck) { ck = key[j]; cj = j; }
    const uint32_t kmax = uint32_t(wave_reduce(
        int(ck), [](int a, int b) { return int(max(uint32_t(a), uint32_t(b))); }, 0));
    const int from = __ffsll(static_cast<unsigned long long>(__ballot(ck == kmax))) - 1;
    const int be = readlane(ln.first + cj, from);
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
        if (j == cj) key[j] = 0u;                            // taken
    }
    if (lane == r) { e = be; ekey = kmax; }
  }
  const uint32_t none = score_key(-INFINITY);
  const bool pick = lane < p.k;
  float el = load1(row + e);
  bool live = pick && ekey > none;

  if (!by_logit) {
    // does the fp32 order stand?
    const float ec = key_score(ekey), eb = bias[e];
    const float tol = 0x1p-17f * smax + 0x1p-22f * fabsf(ec);
    const float nc = __shfl_down(ec, 1), nl = __shfl_down(el, 1), nb = __shfl_down(eb, 1);
    const bool nlive = __shfl_down(int(live), 1) != 0;
    bool open = live && nlive && lane + 1 < p.k && ec - nc < tol && !(nl == el && nb == eb);
    const int last = p.k - 1;
    if (__ballot(live && lane == last)) {
      const float lc = readlane(ec, last), ll = readlane(el, last), lb = readlane(eb, last);
      const float edge = lc - readlane(tol, last);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        if (key[j] > none && key_score(key[j]) > edge)
          open |= !(l[j] == ll && bias[ln.first + j] == lb);
    }
    if (__ballot(open)) {
      if (!filled) wide.fill(row, bias, p.scoring, w1, w2);
      e = wide.pick(stays, p.k, &live);
      live = live && pick;
      el = load1(row + e);
    }
  }

  // weights, lane r the r-th expert's: sigmoid scores 1 / (1 + exp(-l)); where only their ratios
  // count and all are below 1/2 the common factor exp(max l) is left out, so that none
  // underflows.  Softmax scores relative to the largest chosen, or to the largest of all.
  const float lmax = wave_reduce(live ? el : -INFINITY,
                                 [](float a, float b) { return fmaxf(a, b); }, -INFINITY);
  float s = 0.0f;
  if (live) {
    if (softmax)
      s = expf(el - (p.renormalize ? lmax : top));
    else if (p.renormalize && lmax < 0.0f)
      s = expf(el - lmax) / (1.0f + expf(el));
    else
      s = 1.0f / (1.0f + expf(-el));
  }
  const float sum = p.renormalize ? wave_sum(s) : den;
  if (pick) {
    ids[int64_t(t) * p.k + lane] = e;
    w[int64_t(t) * p.k + lane] = live ? s / sum * p.scale : 0.0f;
  }
}

// lanes per group and experts per lane
struct RouteLayout {
  int width, C;
};
RouteLayout route_layout(const RouteShape& s) {
  const int G = s.topk_group < s.n_group ? s.n_group : 1;
  int gp = 1;
  while (gp < G) gp *= 2;
  const int width = kWave / gp;
  return {width, (s.E / G + width - 1) / width};
}

template <typename LT, int NS>
hipError_t launch_slots(const LT* logits, const float* bias, const RouteShape& s, RouteLayout at,
                        int32_t* ids, float* w, hipStream_t stream) {
  // the 64-bit choice may be needed where fp32 scores decide
  const bool scores = bias || (s.topk_group < s.n_group && s.group_best == 2);
  const size_t lds = scores ? size_t(kRouteWaves) * NS * kWave * sizeof(uint64_t) : 0;
  hipLaunchKernelGGL((route_experts_kernel<LT, NS>), dim3(unsigned((s.T + kRouteWaves - 1) / kRouteWaves)),
                     dim3(64 * kRouteWaves), lds, stream, logits, bias, s, at.C, at.width, ids, w);
  return hipGetLastError();
}

template <typename LT>
hipError_t launch_typed(const LT* logits, const float* bias, const RouteShape& s, int32_t* ids,
                        float* w, hipStream_t stream) {
  const RouteLayout at = route_layout(s);
  if (at.C <= 1) return launch_slots<LT, 1>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 2) return launch_slots<LT, 2>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 4) return launch_slots<LT, 4>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 8) return launch_slots<LT, 8>(logits, bias, s, at, ids, w, stream);
  if (at.C <= 16) return launch_slots<LT, 16>(logits, bias, s, at, ids, w, stream);
  return launch_slots<LT, 32>(logits, bias, s, at, ids, w, stream);   // C <= 31: E <= 1024
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
