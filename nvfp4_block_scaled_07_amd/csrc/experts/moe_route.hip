// Routing: the experts of each token and their weights, from router logits.
//
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e));  v_e = s_e + bias_e
//   group value = sum of the group_top largest v of a group; the top_groups
//   best groups stay;  ids = the top_k largest v among them, largest first
//   w_j = s of id_j, over their sum if renormalised, times scale
// All ties go to the lowest index; NaN ranks below everything.
//
// One wave a token, lane l holding experts VPL l .. VPL l + VPL - 1, so that
// the first lane of a ballot is the lowest index.  Values are compared as
// integers (the order-preserving map of the floats' bits, 1 for NaN, 0 for "not
// there"), whose maximum over a wave is six DPP and lane-swap steps.
//
// Exact choice.  Whole numbers come out, so two values that differ by less than
// the fp32 rounding of s must not trade places.  Where v increases with x (no
// bias, and no group sums) the logits themselves are ranked, which is exact.
// Else values are formed in fp32 and every comparison that decides (each
// chosen value with the next, the last chosen group with the best left out) is
// checked against a bound on that rounding; a token with a closer one is done
// again with fp64 values, by the same code.
#include "experts.h"
#include "mx_block.h"

namespace nvfp4 {

// ------------------------------------------------------------ ordered keys

template <typename F>
struct Key;
template <>
struct Key<float> {
  typedef uint32_t type;
  static __device__ __forceinline__ uint32_t of(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);  // one zero
    return f == f ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : 1u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((uint32_t)(~(int32_t)k >> 31) | 0x80000000u));
  }
};
template <>
struct Key<double> {
  typedef uint64_t type;
  static __device__ __forceinline__ uint64_t of(double f) {
    const uint64_t u = __builtin_bit_cast(uint64_t, f + 0.0);
    return f == f ? u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull) : 1ull;
  }
  static __device__ __forceinline__ double value(uint64_t k) {
    return __builtin_bit_cast(double, k ^ ((uint64_t)(~(int64_t)k >> 63) | 0x8000000000000000ull));
  }
};

// DPP moves that the compiler folds into the instruction that uses them: lanes
// without a source would read 0
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t kmax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t kmax(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  return (uint64_t)moved<CTRL>((uint32_t)(v >> 32)) << 32 | moved<CTRL>((uint32_t)v);
}
__device__ __forceinline__ uint32_t swap16(uint32_t v, int half) {
  return __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane16_swap(v, v, false, false))[half];
}
__device__ __forceinline__ uint32_t swap32(uint32_t v, int half) {
  return __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(v, v, false, false))[half];
}

// Maximum over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = kmax(v, moved<kDppXor1>(v));
  v = kmax(v, moved<kDppXor2>(v));
  v = kmax(v, moved<kDppHalfMirror>(v));
  v = kmax(v, moved<kDppMirror>(v));
  v = kmax(swap16(v, 0), swap16(v, 1));
  v = kmax(swap32(v, 0), swap32(v, 1));
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = kmax(v, dpp64<kDppXor1>(v));
  v = kmax(v, dpp64<kDppXor2>(v));
  v = kmax(v, dpp64<kDppHalfMirror>(v));
  v = kmax(v, dpp64<kDppMirror>(v));
#pragma unroll
  for (int o = 16; o <= 32; o *= 2) v = kmax(v, (uint64_t)__shfl_xor((unsigned long long)v, o));
  return v;
}

template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __uint_as_float(moved<CTRL>(__float_as_uint(v)));
}
// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dppf<kDppXor1>(v);
  v += dppf<kDppXor2>(v);
  v += dppf<kDppHalfMirror>(v);
  v += dppf<kDppMirror>(v);
  const uint32_t u = __float_as_uint(v);
  v = __uint_as_float(swap16(u, 0)) + __uint_as_float(swap16(u, 1));
  const uint32_t w = __float_as_uint(v);
  return __uint_as_float(swap32(w, 0)) + __uint_as_float(swap32(w, 1));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

// exp(x): in fp32 the hardware exp2 of the rounded x log2 e, relative error
// below (1.23 |x| + 2) 2^-24 (the product's rounding and the constant's, which is
// 0.23 of one; one unit of the exponential)
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// exp(hi + lo) with the rounding of hi log2 e made up for: within 3 x 2^-24
// where the result is a normal number.
__device__ __forceinline__ float exp_fine(float hi, float lo) {
  const float t = hi * 1.44269504f;
  const float r = __builtin_fmaf(lo, 1.44269504f, __builtin_fmaf(hi, 1.92596303e-8f, __builtin_fmaf(hi, 1.44269504f, -t)));
  return __builtin_amdgcn_exp2f(t) * (fabsf(hi) < 200.0f ? __builtin_fmaf(r, 0.69314718f, 1.0f) : 1.0f);
}

// ----------------------------------------------------------------- scores

// What turns a token's logits into scores: softmax's maximum and the inverse
// of its sum (a token whose logits are all -infinity has scores 0).
template <typename F>
struct Scorer {
  F top, inv;
  bool softmax;
  __device__ __forceinline__ F operator()(float x) const {
    return softmax ? exp_of((F)x - top) * inv : inverse((F)1 + exp_of(-(F)x));
  }
  // for a weight: far logits as exactly as near ones
  __device__ __forceinline__ float fine(float x) const {
    if (!softmax) return inverse(1.0f + exp_fine(-x, 0.0f));
    const float d = x - top, b = d - x;  // x - top = d + its rounding
    return exp_fine(d, (x - (d - b)) - (top + b)) * inv;
  }
};

template <int VPL, typename F>
__device__ __forceinline__ Scorer<F> scorer(const float (&x)[VPL], int have, bool softmax) {
  Scorer<F> s{(F)0, (F)1, softmax};
  if (!softmax) return s;
  uint32_t k = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) k = kmax(k, i < have ? Key<float>::of(x[i]) : 0u);
  const float top = Key<float>::value(wave_max(k));
  s.top = top == -__builtin_inff() ? (F)0 : (F)top;
  F sum = (F)0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum += i < have ? exp_of((F)x[i] - s.top) : (F)0;
  sum = wave_sum(sum);
  s.inv = sum == (F)0 ? (F)0 : inverse(sum);
  return s;
}

// ----------------------------------------------------------------- choice

// The choice among a wave's keys (key[i]: expert VPL lane + i).  mine: lane j's
// chosen expert.  Returns whether every decision was clear: values further
// apart than slack(value) allows.  Which lane and which of its keys hold the
// maximum is found in scalar registers, from ballots.
template <int VPL, typename F, class S>
__device__ __forceinline__ bool choose(const RouteLaunch& p, typename Key<F>::type (&key)[VPL], const S& slack,
                                       int& mine) {
  typedef typename Key<F>::type K;
  const int lane = threadIdx.x & 63;
  K taken = 0, top;  // lane j: the key of choice j; lane top_k: the best one left, which is also the last top
  for (int j = 0;; ++j) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = kmax(best, key[i]);
    top = wave_max(best);
    taken = lane == j ? top : taken;
    if (j == p.top_k) break;
    const int from = __builtin_ctzll(__ballot(best == top));
    int at = VPL - 1;
#pragma unroll
    for (int i = VPL - 2; i >= 0; --i) at = __ballot(key[i] == top) >> from & 1 ? i : at;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane == from && i == at ? (K)0 : key[i];
    mine = lane == j ? from * VPL + at : mine;
  }
  // the pairs (choice j, choice j + 1), and the last choice with the best one left
  // (64 choices leave no lane for it)
  const K next = __shfl_down(taken, 1), after = lane == 63 ? top : next;
  const F a = Key<F>::value(taken), b = Key<F>::value(after);
  const bool there = after != 0 && lane < p.top_k;
  return __ballot(there && !(a - b > slack(a, b))) == 0;
}

// Two largest of (a, b) and of the pair of another lane, a >= b; c >= d.
template <typename K>
__device__ __forceinline__ void top_two(K& a, K& b, K c, K d) {
  const K low = a < c ? a : c;
  a = kmax(a, c);
  b = kmax(low, kmax(b, d));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dppk(uint32_t v) { return moved<CTRL>(v); }
template <int CTRL>
__device__ __forceinline__ uint64_t dppk(uint64_t v) { return dpp64<CTRL>(v); }

__device__ __forceinline__ uint32_t key_of_lane(uint32_t k, int lane) { return __builtin_amdgcn_readlane(k, lane); }
__device__ __forceinline__ uint64_t key_of_lane(uint64_t k, int lane) {
  return (uint64_t)key_of_lane((uint32_t)(k >> 32), lane) << 32 | key_of_lane((uint32_t)k, lane);
}

// Keys of experts outside the best groups become 0.  cell: this wave's LDS.
template <int VPL, typename F, class S>
__device__ __forceinline__ bool keep_groups(const RouteLaunch& p, typename Key<F>::type (&key)[VPL], int have,
                                            typename Key<F>::type* cell, const S& slack) {
  typedef typename Key<F>::type K;
  const int lane = threadIdx.x & 63, size = p.E / p.groups;
  int per;  // lanes of a group, a power of two; all of them end with the group's value
  K a = 0, b = 0;  // two largest
  const int whole = size / VPL;
  // each group is the experts of 1, 2, 4, 8 or 16 lanes
  const bool lanes = whole * VPL == size && (whole & (whole - 1)) == 0 && whole <= 16;
  if (lanes) {
    per = whole;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top_two(a, b, key[i], (K)0);
    if (per > 1) top_two(a, b, dppk<kDppXor1>(a), dppk<kDppXor1>(b));
    if (per > 2) top_two(a, b, dppk<kDppXor2>(a), dppk<kDppXor2>(b));
    if (per > 4) top_two(a, b, dppk<kDppHalfMirror>(a), dppk<kDppHalfMirror>(b));
    if (per > 8) top_two(a, b, dppk<kDppMirror>(a), dppk<kDppMirror>(b));
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < have) cell[lane * VPL + i] = key[i];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    per = 1;
    while (2 * per * p.groups <= 64 && per < size) per *= 2;
    if (lane / per < p.groups)
      for (int i = lane & (per - 1); i < size; i += per) top_two(a, b, cell[lane / per * size + i], (K)0);
    for (int o = 1; o < per; o *= 2) top_two(a, b, (K)__shfl_xor(a, o), (K)__shfl_xor(b, o));
    __builtin_amdgcn_wave_barrier();
  }
  const bool in = lane / per < p.groups;
  const F sum = p.group_top == 2 ? Key<F>::value(a) + Key<F>::value(b) : Key<F>::value(a);
  const K k = in ? Key<F>::of(sum) : (K)0;
  // rank of a group: groups with a larger value, or the same and a lower index
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const K other = key_of_lane(k, g * per);
    rank += other > k || (other == k && g < lane / per);
  }
  const uint64_t kept = __ballot(in && rank < p.top_groups);
  const int last = __builtin_ctzll(__ballot(in && rank == p.top_groups - 1));
  const int left = __builtin_ctzll(__ballot(in && rank == p.top_groups));
  const F c = Key<F>::value(key_of_lane(k, last)), d = Key<F>::value(key_of_lane(k, left));
  const bool mine = kept >> lane & 1;
  if (lanes) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = mine ? key[i] : (K)0;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < have && !(kept >> ((lane * VPL + i) / size * per) & 1)) key[i] = 0;
  }
  return c - d > slack(c, d);
}

// Values in F, the choice among them; returns whether it was clear.
template <int VPL, typename F, class S, class G>
__device__ __forceinline__ bool route(const RouteLaunch& p, const float (&x)[VPL], const float (&bias)[VPL], int have,
                                      typename Key<F>::type* cell, bool by_logit, const Scorer<F>& score, const S& slack, const G& gslack,
                                      int& mine) {
  typename Key<F>::type key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const F v = by_logit ? (F)x[i] : score(x[i]) + (F)bias[i];
    key[i] = i < have ? Key<F>::of(v) : (typename Key<F>::type)0;
  }
  bool clear = true;
  if (p.groups > 1 && p.top_groups < p.groups) clear = keep_groups<VPL, F>(p, key, have, cell, gslack);
  return choose<VPL, F>(p, key, slack, mine) && clear;
}

__device__ __forceinline__ float logit_at(const RouteLaunch& p, int64_t at) {
  return p.bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p.logits)[at] << 16) : ((const float*)p.logits)[at];
}

// This lane's logits: one or a few wide loads where the lanes' experts are
// whole runs, of any alignment that the type has.
template <int VPL>
__device__ __forceinline__ void load_logits(const RouteLaunch& p, int64_t t, int lane, int have, float (&x)[VPL]) {
  typedef uint32_t words_t __attribute__((ext_vector_type(VPL >= 8 ? 4 : VPL >= 4 ? 2 : 1), aligned(2)));
  typedef float floats_t __attribute__((ext_vector_type(VPL >= 4 ? 4 : VPL), aligned(4)));
  const int64_t at = t * p.ldl + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = 0.0f;
  if (VPL == 1 || p.E % VPL != 0) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < have) x[i] = logit_at(p, at + i);
  } else if (have > 0) {
    if (p.bf16) {
      constexpr int W = sizeof(words_t) / 4;
#pragma unroll
      for (int c = 0; c < VPL / (2 * W); ++c) {
        const words_t w = ((const words_t*)((const uint16_t*)p.logits + at))[c];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          x[(2 * W * c + 2 * i) % VPL] = __uint_as_float(w[i] << 16);
          x[(2 * W * c + 2 * i + 1) % VPL] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    } else {
      constexpr int W = sizeof(floats_t) / 4;
#pragma unroll
      for (int c = 0; c < VPL / W; ++c) {
        const floats_t w = ((const floats_t*)((const float*)p.logits + at))[c];
#pragma unroll
        for (int i = 0; i < W; ++i) x[W * c + i] = w[i];
      }
    }
  }
}

constexpr int kRouteWaves = 4;

// Waves a SIMD: a token is a long chain, so more of them hide each other's, up to
// where registers spill in earnest (four at 256 experts like this, nine with one
// wave more).  16384 tokens on 256 experts by the compiler's choice (4 waves) 28.0
// us, 5 waves 25.2, 6 24.9, 7 25.7; 128 experts, 6 / 7 / 8: 15.4 / 16.1 / 16.2; 512
// experts, 3 / 4 / 5: 38 / 36 / 32; 1024, 2 / 3: 79 / 64.
constexpr int route_occupancy(int vpl) { return vpl <= 2 ? 7 : vpl == 4 ? 6 : vpl == 8 ? 4 : 2; }

template <int VPL>
__global__ __launch_bounds__(64 * kRouteWaves) __attribute__((amdgpu_waves_per_eu(route_occupancy(VPL)))) void k_moe_route(
    RouteLaunch p) {
  __shared__ uint64_t cells[kRouteWaves][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int have = min(max(p.E - lane * VPL, 0), VPL);  // this lane's experts
  float bias[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) bias[i] = p.bias && i < have ? p.bias[lane * VPL + i] : 0.0f;
  const bool softmax = p.score == 0;
  // scores increase with the logits: without a bias or group sums they rank the same
  const bool grouped = p.groups > 1 && p.top_groups < p.groups;
  const bool by_logit = !p.bias && !(grouped && p.group_top == 2);
  const int64_t step = (int64_t)gridDim.x * kRouteWaves;
  int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  float next[VPL];
  if (t < p.T) load_logits<VPL>(p, t, lane, have, next);
  float lift = 0.0f;  // largest positive bias
  if (grouped && p.group_top == 2) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) lift = fmaxf(lift, bias[i]);
    lift = Key<float>::value(wave_max(Key<float>::of(lift)));
  }
  for (; t < p.T; t += step) {
    float x[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = next[i];
    if (t + step < p.T) load_logits<VPL>(p, t + step, lane, have, next);
    const Scorer<float> score = scorer<VPL, float>(x, have, softmax);
    // Twice the error of a value, in units u = 2^-24.  Sigmoid: the exponential's
    // error reaches s by s (1 - s), an addition and the reciprocal (two) add 3 s: at
    // most 3.2 u.  Softmax, of inv: its own exponential, whose argument x - top is
    // rounded as well, e^-d (2.23 d + 2) <= 2.1, a product 1, and in inv the sum's
    // exponentials 12 (1023 others at d = 5), its additions 21, the reciprocal 2: 38 u,
    // and s <= inv.  2^-20 is 16 u, 2^-17 128.  The sum with the bias is rounded once.
    const float es = softmax ? 0x1p-17f * score.inv : 0x1p-20f;
    const auto slack = [=](float a, float b) { return es + 0x1p-22f * (fabsf(a) + fabsf(b)); };
    // a group's sum also has the rounding of its two values, which a bias can make
    // far larger than their sum: |a| + |b| <= |a + b| + 2 max(a, 0), a <= score + lift
    const auto gslack = [=](float a, float b) { return 2.0f * es + 0x1p-21f * (fabsf(a) + fabsf(b) + lift); };
    const auto none = [](auto, auto) { return -__builtin_inff(); };
    int mine = 0;
    const bool clear = route<VPL, float>(p, x, bias, have, (uint32_t*)cells[wave], by_logit, score, slack, gslack, mine);
    if (!clear && !by_logit) {  // uniform
      const Scorer<double> exact = scorer<VPL, double>(x, have, softmax);
      route<VPL, double>(p, x, bias, have, cells[wave], false, exact, none, none, mine);
    }
    const float chosen = lane < p.top_k ? logit_at(p, t * p.ldl + mine) : 0.0f;
    float w = lane < p.top_k ? score.fine(chosen) : 0.0f;
    if (p.renormalize) {
      const float sum = wave_sum(w);
      // A score below 2^-126 counts, in the sum or on its own (over a small sum, or
      // times a large scale): uniform, and rare, as the logit is then 87 below the
      // largest (sigmoid: below 0).
      const bool far = lane < p.top_k && w < 0x1p-126f && chosen != -__builtin_inff();
      if (sum < 0x1p-90f || __ballot(far) != 0) {
        const Scorer<double> exact = scorer<VPL, double>(x, have, softmax);
        const double v = lane < p.top_k ? exact(chosen) : 0.0, all = wave_sum(v);
        w = all == 0.0 ? 0.0f : (float)(v / all * p.scale);
      } else {
        w = w * inverse(sum) * p.scale;
      }
    } else {
      w *= p.scale;
    }
    if (lane < p.top_k) {
      p.ids[t * p.top_k + lane] = mine;
      p.weights[t * p.top_k + lane] = w;
    }
  }
}

template <int VPL>
static void launch_route(const RouteLaunch& p, hipStream_t stream) {
  int64_t blocks = (p.T + kRouteWaves - 1) / kRouteWaves;
  if (blocks > 8 * kCUs) blocks = 8 * kCUs;
  hipLaunchKernelGGL(k_moe_route<VPL>, dim3((unsigned)blocks), dim3(64 * kRouteWaves), 0, stream, p);
}

hipError_t launch_moe_route(const RouteLaunch& p, hipStream_t stream) {
  if (p.E <= 64) launch_route<1>(p, stream);
  else if (p.E <= 128) launch_route<2>(p, stream);
  else if (p.E <= 256) launch_route<4>(p, stream);
  else if (p.E <= 512) launch_route<8>(p, stream);
  else launch_route<16>(p, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
