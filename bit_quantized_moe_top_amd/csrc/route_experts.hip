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

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  return uint32_t(wave_reduce(int(v), [](int a, int b) { return int(umax(uint32_t(a), uint32_t(b))); }, 0));
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

template <typename LT, int NS>
__global__ void __launch_bounds__(64 * kRouteWaves)
route_experts_kernel(const LT* __restrict__ logits, const float* __restrict__ bias, RouteShape p,
                     int C, int width, int whole, int32_t* __restrict__ ids, float* __restrict__ w) {
  extern __shared__ __align__(16) uint64_t wide_keys[];      // [waves][NS][64] where needed
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;                                      // whole wave exits together
  const bool grouped = p.topk_group < p.n_group;
  const bool softmax = p.scoring == MOEQ_SCORE_SOFTMAX;
  const Lanes ln(p, grouped, C, width, lane);
  const LT* row = logits + int64_t(t) * p.ld;

  float l[NS], c[NS];
  load_slots<NS>(row + ln.first, ln.n, whole, l);
  if (bias) load_slots<NS>(bias + ln.first, ln.n, whole, c);
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

  // keys that order experts: c, or without a bias the logits (the fp32 scores are then needed for
  // sums of two in groups only)
  const bool by_logit = bias == nullptr;
  const bool scores = !by_logit || (grouped && p.group_best == 2);
  const float rden = softmax ? 1.0f / den : 1.0f;
  const float smax = softmax ? rden : 0.125f;
  const uint32_t none = score_key(-INFINITY);
  uint32_t key[NS];
  if (scores) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float s = softmax ? exp_fast(l[j] - top) * rden
                              : __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[j]));
      c[j] = l[j] == -INFINITY ? -INFINITY : by_logit ? s : s + c[j];
    }
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    key[j] = umax(score_key(scores ? c[j] : l[j]), 1u);      // (one NaN has key 0)
    if (j >= ln.n) key[j] = 0u;
  }

  WideChoice<LT> wide{wide_keys + size_t(wave) * NS * kWave, ln, lane};
  bool filled = false;
  double w1 = 0.0, w2 = 0.0;
  bool stays = true;
  if (grouped) {
    uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      b2 = umax(b2, umin(b1, key[j]));
      b1 = umax(b1, key[j]);
    }
    if (width > 1) join2_dpp<kDppQuadSwap1>(b1, b2);
    if (width > 2) join2_dpp<kDppQuadSwap2>(b1, b2);
    if (width > 4) join2_dpp<kDppRowHalfMirror>(b1, b2);
    if (width > 8) join2_dpp<kDppRowMirror>(b1, b2);
    if (width > 16) join2(b1, b2, uint32_t(__shfl_xor(int(b1), 16)), uint32_t(__shfl_xor(int(b2), 16)));
    const bool live = b1 > none;
    if (!scores) {                                           // best of the logits: exact
      int above = 0;
      for (int g = 0; g < ln.G; ++g) {
        const uint32_t other = uint32_t(readlane(int(b1), g * width));
        above += other > b1 || (other == b1 && g < ln.g);
      }
      stays = above < p.topk_group;
    } else {
      // A group stays for sure if at most topk_group - 1 others may be above it.  If as many stay
      // for sure as are to stay, the choice is made.
      const bool two = p.group_best == 2 && b2 > none;
      const float f1 = key_score(b1), f2 = two ? key_score(b2) : 0.0f;
      const float half = 0x1p-17f * smax + 0x1p-22f * (fabsf(f1) + fabsf(f2));
      const float lo = f1 + f2 - half;
      const float hi = live ? f1 + f2 + half : -INFINITY;
      int maybe = 0;
      for (int g = 0; g < ln.G; ++g) maybe += readlane(hi, g * width) >= lo ? 1 : 0;   // and itself
      const uint64_t leads = __ballot(live && ln.g < ln.G && lane == ln.g * width);
      const int n_live = __popcll(leads);
      stays = live ? maybe <= p.topk_group
                   // empty groups: after all the others, the lower first
                   : n_live + __popcll(__ballot(!live && ln.g < ln.G && lane == ln.g * width) &
                                       ((uint64_t(1) << (ln.g * width & 63)) - 1)) < p.topk_group;
      const int sure = __popcll(__ballot(stays) & leads);
      if (sure < min(p.topk_group, n_live)) {
        wide.fill(row, bias, p.scoring, w1, w2);
        filled = true;
        stays = wide.group_stays(w1, w2, p.group_best, p.topk_group);
      }
    }
  }
  if (scores && by_logit) {
#pragma unroll
    for (int j = 0; j < NS; ++j) key[j] = j < ln.n ? umax(score_key(l[j]), 1u) : 0u;
  }
  if (grouped) {
#pragma unroll
    for (int j = 0; j < NS; ++j) key[j] = stays ? key[j] : umin(key[j], none);
  }

  // k rounds of a wave-wide argmax over the heads
  SortedSlots<NS> left;
  left.sort(key);
  int e = 0, ekey = 0;
  for (int r = 0; r < p.k; ++r) {
    int slot, list;
    const uint32_t mine = left.best(slot, list);
    const uint32_t kmax = wave_umax(mine);
    const int from = __ffsll(static_cast<unsigned long long>(__ballot(mine == kmax))) - 1;
    const int be = readlane(ln.first + slot, from);
    const int from_list = SortedSlots<NS>::kLists > 1 ? readlane(list, from) : 0;
    if (lane == from) left.take(from_list);
    e = lane == r ? be : e;
    ekey = lane == r ? int(kmax) : ekey;
  }
  const bool pick = lane < p.k;
  float el = load1(row + e);
  bool live = pick && uint32_t(ekey) > none;

  if (!by_logit) {
    // does the fp32 order stand?
    const float ec = key_score(uint32_t(ekey)), eb = bias[e];
    const float tol = 0x1p-17f * smax + 0x1p-22f * fabsf(ec);
    const float nc = __shfl_down(ec, 1), nl = __shfl_down(el, 1), nb = __shfl_down(eb, 1);
    const bool nlive = __shfl_down(int(live), 1) != 0;
    bool open = live && nlive && lane + 1 < p.k && ec - nc < tol && !(nl == el && nb == eb);
    const int last = p.k - 1;
    if (uint32_t(readlane(ekey, last)) > none) {
      const uint32_t edge = umax(score_key(readlane(ec - tol, last)), none);
      bool near = false;
#pragma unroll
      for (int i = 0; i < SortedSlots<NS>::kLists; ++i) near |= left.key[i][0] > edge;
      if (__ballot(near)) {                                  // equal to the last pick in both parts?
        const float ll = readlane(el, last), lb = readlane(eb, last);
#pragma unroll
        for (int i = 0; i < SortedSlots<NS>::kLists; ++i)
#pragma unroll
          for (int j = 0; j < SortedSlots<NS>::kLen; ++j)
            if (left.key[i][j] > edge) {
              const int at = ln.first + SortedSlots<NS>::kLen * i + int(left.order[i] >> (8 * j) & 255u);
              open |= !(load1(row + at) == ll && bias[at] == lb);
            }
      }
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
  // every lane with experts has NS of them, on the alignment of the wide loads
  const int S = s.E / (s.topk_group < s.n_group ? s.n_group : 1);
  const int whole = at.C == NS && S % NS == 0 && s.ld % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(logits) % (4 * sizeof(LT)) == 0 &&
                    reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  hipLaunchKernelGGL((route_experts_kernel<LT, NS>), dim3(unsigned((s.T + kRouteWaves - 1) / kRouteWaves)),
                     dim3(64 * kRouteWaves), lds, stream, logits, bias, s, at.C, at.width, whole, ids, w);
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
