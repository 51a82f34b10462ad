// Routing: the experts of each token and their weights, from router logits.
//
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e));  v_e = s_e + bias_e
//   group value = sum of the group_top largest v of a group; the top_groups
//   best groups stay;  ids = the top_k largest v among them, largest first
//   w_j = s of id_j, over their sum if renormalised, times scale
// All ties go to the lowest index; NaN ranks as -infinity.
//
// One wave a token, lane l holding experts VPL l .. VPL l + VPL - 1, so that
// the first lane of a ballot is the lowest index.  Values are compared as
// integers (the order-preserving map of the floats' bits, 0 for "not there"),
// whose maximum over a wave is six DPP and lane-swap steps.
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
    const uint32_t u = __float_as_uint(f == f ? f + 0.0f : -__builtin_inff());  // + 0: one zero
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((uint32_t)(~(int32_t)k >> 31) | 0x80000000u));
  }
};
template <>
struct Key<double> {
  typedef uint64_t type;
  static __device__ __forceinline__ uint64_t of(double f) {
    const uint64_t u = __builtin_bit_cast(uint64_t, f == f ? f + 0.0 : -(double)__builtin_inff());
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  }
  static __device__ __forceinline__ double value(uint64_t k) {
    return __builtin_bit_cast(double, k ^ ((uint64_t)(~(int64_t)k >> 63) | 0x8000000000000000ull));
  }
};

__device__ __forceinline__ uint32_t kmax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t kmax(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  return (uint64_t)dpp<CTRL>((uint32_t)(v >> 32)) << 32 | dpp<CTRL>((uint32_t)v);
}
__device__ __forceinline__ uint32_t swap16(uint32_t v, int half) {
  return __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane16_swap(v, v, false, false))[half];
}
__device__ __forceinline__ uint32_t swap32(uint32_t v, int half) {
  return __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(v, v, false, false))[half];
}

// Maximum over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = kmax(v, dpp<kDppXor1>(v));
  v = kmax(v, dpp<kDppXor2>(v));
  v = kmax(v, dpp<kDppHalfMirror>(v));
  v = kmax(v, dpp<kDppMirror>(v));
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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// ----------------------------------------------------------------- scores

// What turns a token's logits into scores: softmax's maximum and the inverse
// of its sum (a token whose logits are all -infinity has scores 0).
template <typename F>
struct Scorer {
  F top, inv;
  bool softmax;
  __device__ __forceinline__ F operator()(float x) const {
    return softmax ? exp_of((F)x - top) * inv : (F)1 / ((F)1 + exp_of(-(F)x));
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
  s.inv = sum == (F)0 ? (F)0 : (F)1 / sum;
  return s;
}

// ----------------------------------------------------------------- choice

// The choice among a wave's keys (key[i]: expert VPL lane + i).  mine: lane j's
// chosen expert.  Returns whether every decision was clear: values further
// apart than slack(value) allows.
template <int VPL, typename F, class S>
__device__ __forceinline__ bool choose(const RouteLaunch& p, typename Key<F>::type (&key)[VPL], const S& slack,
                                       int& mine) {
  typedef typename Key<F>::type K;
  const int lane = threadIdx.x & 63;
  bool clear = true;
  K last = 0;
  for (int j = 0; j <= p.top_k; ++j) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = kmax(best, key[i]);
    const K top = wave_max(best);
    if (j > 0 && top != 0) {
      const F a = Key<F>::value(last), b = Key<F>::value(top);
      clear = clear && a - b > slack(a, b);
    }
    if (j == p.top_k) break;
    last = top;
    const int from = __builtin_ctzll(__ballot(best == top));
    int at = VPL - 1;
#pragma unroll
    for (int i = VPL - 2; i >= 0; --i) at = key[i] == top ? i : at;
    at = __builtin_amdgcn_readlane(at, from);
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane == from && i == at ? (K)0 : key[i];
    if (lane == j) mine = from * VPL + at;
  }
  return clear;
}

// Keys of experts outside the best groups become 0.  cell: this wave's LDS.
template <int VPL, typename F, class S>
__device__ __forceinline__ bool keep_groups(const RouteLaunch& p, const F (&v)[VPL], typename Key<F>::type (&key)[VPL],
                                            int have, F* cell, const S& slack) {
  typedef typename Key<F>::type K;
  const int lane = threadIdx.x & 63, size = p.E / p.groups;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (i < have) cell[lane * VPL + i] = v[i];
  __builtin_amdgcn_wave_barrier();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  // lanes per group: a power of two, groups <= 64
  int per = 1;
  while (2 * per * p.groups <= 64 && per < size) per *= 2;
  const int g = lane / per, part = lane & (per - 1);
  const bool in = g < p.groups;
  const F low = -(F)__builtin_inff();
  F a = low, b = low;  // two largest
  if (in)
    for (int i = part; i < size; i += per) {
      const F f = cell[g * size + i];
      const F c = f == f ? f : low;
      b = c > a ? a : c > b ? c : b;
      a = c > a ? c : a;
    }
  for (int o = 1; o < per; o *= 2) {
    const F c = __shfl_xor(a, o), d = __shfl_xor(b, o);
    const F m = c > a ? a : c, n = d > b ? d : b;
    a = c > a ? c : a;
    b = m > n ? m : n;
  }
  const F sum = p.group_top == 2 ? a + b : a;
  K k = in ? Key<F>::of(sum) : (K)0;
  K left = part == 0 ? k : (K)0;
  uint64_t kept = 0;
  bool clear = true;
  K last = 0;
  for (int j = 0; j <= p.top_groups; ++j) {
    const K top = wave_max(left);
    if (j == p.top_groups) {
      if (top != 0) {
        const F c = Key<F>::value(last), d = Key<F>::value(top);
        clear = c - d > slack(c, d);
      }
      break;
    }
    last = top;
    const int from = __builtin_ctzll(__ballot(left == top && part == 0 && in));
    kept |= 1ull << from;
    if (lane == from) left = 0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if (i < have && !(kept >> ((e / size) * per) & 1)) key[i] = 0;
  }
  __builtin_amdgcn_wave_barrier();
  return clear;
}

// Values in F, the choice among them; returns whether it was clear.
template <int VPL, typename F, class S, class G>
__device__ __forceinline__ bool route(const RouteLaunch& p, const float (&x)[VPL], const float (&bias)[VPL], int have,
                                      F* cell, bool by_logit, const Scorer<F>& score, const S& slack, const G& gslack,
                                      int& mine) {
  F v[VPL];
  typename Key<F>::type key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    v[i] = by_logit ? (F)x[i] : score(x[i]) + (F)bias[i];
    key[i] = i < have ? Key<F>::of(v[i]) : (typename Key<F>::type)0;
  }
  bool clear = true;
  if (p.groups > 1 && p.top_groups < p.groups) clear = keep_groups<VPL, F>(p, v, key, have, cell, gslack);
  return choose<VPL, F>(p, key, slack, mine) && clear;
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteLaunch& p, int64_t t, int lane, int have, float (&x)[VPL]) {
  const int64_t at = t * p.ldl + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    x[i] = i >= have ? 0.0f
           : p.bf16  ? __uint_as_float((uint32_t)((const uint16_t*)p.logits)[at + i] << 16)
                     : ((const float*)p.logits)[at + i];
}

constexpr int kRouteWaves = 4;

template <int VPL>
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(RouteLaunch p) {
  __shared__ double cells[kRouteWaves][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int have = min(max(p.E - lane * VPL, 0), VPL);  // this lane's experts
  float bias[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) bias[i] = p.bias && i < have ? p.bias[lane * VPL + i] : 0.0f;
  const bool softmax = p.score == 0;
  // scores increase with the logits: without a bias or group sums they rank the same
  const bool grouped = p.groups > 1 && p.top_groups < p.groups;
  const bool by_logit = !p.bias && !(grouped && p.group_top == 2);
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < p.T; t += (int64_t)gridDim.x * kRouteWaves) {
    float x[VPL];
    load_logits<VPL>(p, t, lane, have, x);
    const Scorer<float> score = scorer<VPL, float>(x, have, softmax);
    // Twice the error of a value: s has relative error below 2^-21.4 (sigmoid)
    // or 2^-18.5 (softmax, s <= inv); its sum with the bias one rounding.
    const float es = softmax ? 0x1p-17f * score.inv : 0x1p-20f;
    const auto slack = [=](float a, float b) { return es + 0x1p-22f * (fabsf(a) + fabsf(b)); };
    const auto gslack = [=](float a, float b) { return 2.0f * es + 0x1p-21f * (fabsf(a) + fabsf(b)); };
    const auto none = [](auto, auto) { return -__builtin_inff(); };
    int mine = 0;
    bool clear;
    if (by_logit) {
      route<VPL, float>(p, x, bias, have, (float*)cells[wave], true, score, none, none, mine);
      clear = true;
    } else {
      clear = route<VPL, float>(p, x, bias, have, (float*)cells[wave], false, score, slack, gslack, mine);
    }
    if (!clear) {  // uniform
      const Scorer<double> exact = scorer<VPL, double>(x, have, softmax);
      route<VPL, double>(p, x, bias, have, cells[wave], false, exact, none, none, mine);
    }
    float w = 0.0f;
    if (lane < p.top_k) {
      const int64_t at = t * p.ldl + mine;
      w = score(p.bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p.logits)[at] << 16) : ((const float*)p.logits)[at]);
    }
    if (p.renormalize) {
      const float sum = wave_sum(w);
      w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (lane < p.top_k) {
      p.ids[t * p.top_k + lane] = mine;
      p.weights[t * p.top_k + lane] = w * p.scale;
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
