// Epilogues of the block GEMMs: what happens to a tile's fp32 sums between
// the last MFMA and the one rounding to the output.
//
// The MFMA layouts give a lane one column and rows four apart.  The unsplit
// large tiles of the plain epilogue work on that layout (finish_direct: 64
// bytes of a row per half wave; stores and the next block's residual loads in
// flight while a block is computed).  Where a sum passes through LDS anyway
// (K-groups, split K), or a result needs its neighbours (a gate column its up
// column, an NVFP4 block its 16 columns), the tile is read back from LDS with
// consecutive columns per lane.
//
// Arithmetic is fp32, in the order of the formulas, one rounding per step and
// one rounding to bf16 (or to e4m3 and e2m1) at the end.  The sums and the
// hidden layer are never rounded to bf16 in between.
#pragma once

#include "../kreg_tile.h"
#include "block.h"
#include "quantize_block.h"
#include "vec8.h"

namespace nvfp4 {

// Activations (u = 2^-24).  Each is the argument times a factor in (0, 1) built
// from the hardware exp2 and reciprocal (1 ulp each); the exponent's rounding
// gives the value a relative error of the exponent's size times u, large only
// where the value itself vanishes, and far below the bf16 step (2^-8) and the
// e2m1 step that the result is rounded to.  exp2 overflowing to infinity or
// underflowing to 0 gives the limits.  NaN stays NaN.

// x / (1 + exp2(e)): x sigmoid(-e ln 2)
__device__ __forceinline__ float over_one_plus_exp2(float x, float e) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(e));
}

// x Phi(x) = max(x, 0) - |x| / 2 erfc(|x| / sqrt 2), which has no cancellation
// for x < 0.  With z = |x| / sqrt 2 and t = 1 / (1 + z / 2), erfc(z) = t exp2(p(t)
// - z^2 log2 e), the form of Press, Teukolsky, Vetterling and Flannery, Numerical
// Recipes, section 6.2, with a fit of its own: p is a degree-8 Chebyshev fit of
// log2(erfc(z) exp(z^2) / t) over |x| <= 20 (relative error 6.5 u; erfc is 0 in
// fp32 beyond).  About 18 VALU instructions and the two transcendental ones.
__device__ __forceinline__ float gelu_erf(float x) {
  const float a = fminf(fabsf(x), 20.0f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35355339f, 1.0f));
  float e = 0.0656675398f;
  e = __builtin_fmaf(e, t, -0.571985662f);
  e = __builtin_fmaf(e, t, 1.66417825f);
  e = __builtin_fmaf(e, t, -2.05382848f);
  e = __builtin_fmaf(e, t, 0.885032177f);
  e = __builtin_fmaf(e, t, -0.200422123f);
  e = __builtin_fmaf(e, t, 0.599930644f);
  e = __builtin_fmaf(e, t, 1.43694723f);
  e = __builtin_fmaf(e, t, -1.82552004f);
  e = __builtin_fmaf(a * a, -0.72134752f, e);
  return (x < 0.0f ? 0.0f : x) - 0.5f * a * t * __builtin_amdgcn_exp2f(e);
}

template <int W>
__device__ __forceinline__ void activate(float (&v)[W], int act) {
  if (act == 4) {  // uniform branches, once per chunk
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = over_one_plus_exp2(v[i], v[i] * -1.44269504f);
  } else if (act == 3) {
    // x (1 + tanh(z)) / 2 = x sigmoid(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x = v[i];
      v[i] = over_one_plus_exp2(x, x * __builtin_fmaf(x * x, -0.102943240f, -2.30220820f));
    }
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = gelu_erf(v[i]);
  } else if (act == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
  }
}

// 8 bf16 values at p, packed; columns [col, cols) are valid, the others 0.
__device__ __forceinline__ u4_t load_bf16x8(const uint16_t* p, int64_t col, int64_t cols) {
  return col + 8 <= cols ? load8(p) : load_tail8(p, (int)(cols & 7));
}

// v[i] += the W bf16 values at p (a bias vector)
template <int W>
__device__ __forceinline__ void add_bf16(float (&v)[W], const uint16_t* p, int64_t col, int64_t cols) {
#pragma unroll
  for (int c = 0; c < W / 8; ++c) {
    const u4_t w = load_bf16x8(p + 8 * c, col + 8 * c, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * c + i] += bf16_at(w, i);
  }
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float (&v)[8], int64_t col, int64_t cols) {
  if (col + 8 <= cols) store8(p, to_bf16x8(v));
  else store_tail8(p, to_bf16x8(v), (int)(cols & 7));
}

// Columns a lane takes at once: one 16-byte bf16 vector, or one NVFP4 block.
template <bool QUANT>
constexpr int kChunk = QUANT ? 16 : 8;

// The residual of columns [col, col + 8) of one row (plain epilogues).
__device__ __forceinline__ u4_t load_residual(const EpilogueLaunch& p, int64_t row, int64_t col) {
  return load_bf16x8(p.res + row * p.ldr + col, col, p.cols);
}

// The epilogue of columns [col, col + W) of one row, from the sums s (gate or
// only) and u (up) of those columns and their residual (if p.res).
template <bool GATED, bool QUANT>
__device__ __forceinline__ void finish(const EpilogueLaunch& p, float a0, float a1, int64_t row, int64_t col,
                                       const float (&s)[kChunk<QUANT>], const float (&u)[kChunk<QUANT>], u4_t res) {
  constexpr int W = kChunk<QUANT>;
  float v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = a0 * s[i];
  if (p.bias) add_bf16<W>(v, p.bias + col, col, p.cols);
  activate<W>(v, p.act);
  if constexpr (GATED) {
    float t[W];
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = a1 * u[i];
    if (p.bias) add_bf16<W>(t, p.bias + p.cols + col, col, p.cols);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= t[i];
  } else if (p.res) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += p.beta * bf16_at(res, i);
  }
  if constexpr (QUANT) {
    // cols % 16 == 0: the block is whole
    f4_t x[4];
#pragma unroll
    for (int i = 0; i < W; ++i) x[i / 4][i % 4] = v[i];
    uint32_t w[2];
    const uint32_t code = quantize_lane16(x, p.gs ? *p.gs : 1.0f, w);
    *(u2_t*)(p.q + row * (p.cols / 2) + col / 2) = u2_t{w[0], w[1]};
    p.sf[row * (p.cols / 16) + col / 16] = (uint8_t)code;
  } else {
    store_bf16x8(p.g.d + row * p.ldd + col, v, col, p.cols);
  }
}

template <int W>
__device__ __forceinline__ void lds_chunk(float (&v)[W], const float* src) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const f4_t x = *(const f4_t*)(src + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * i + e] = x[e];
  }
}

// One output from its sum (gate or only) s and up sum u, its residual and its
// bias values: the epilogue of the small tiles, where a thread has an output
// or two and everything but the sums was loaded before the main loop.
struct Scalars {
  float a0, a1, bias, bias_up, res;
};

template <bool GATED>
__device__ __forceinline__ float finish_one(const EpilogueLaunch& p, const Scalars& c, float s, float u) {
  float v[1] = {c.a0 * s};
  if (p.bias) v[0] += c.bias;
  activate<1>(v, p.act);
  if constexpr (GATED) {
    float t = c.a1 * u;
    if (p.bias) t += c.bias_up;
    return v[0] * t;
  }
  if (p.res) v[0] += p.beta * c.res;
  return v[0];
}

template <bool GATED>
__device__ __forceinline__ Scalars load_scalars(const EpilogueLaunch& p, float a0, float a1, int64_t row, int64_t col,
                                                bool valid) {
  Scalars c = {a0, a1, 0.0f, 0.0f, 0.0f};
  auto at = [&](const uint16_t* q, int64_t i) { return __uint_as_float((uint32_t)q[i] << 16); };
  if (valid && p.bias) c.bias = at(p.bias, col);
  if constexpr (GATED) {
    if (valid && p.bias) c.bias_up = at(p.bias, p.cols + col);
  } else {
    if (valid && p.res) c.res = at(p.res, row * p.ldr + col);
  }
  return c;
}

// Epilogue of a tile whose sums lie in LDS, row-major with stride LD (gated:
// gate columns, then up columns from UP on), by NT threads, 8 or 16 columns
// at a time.
template <bool GATED, bool QUANT, int ROWS, int COLS, int LD, int UP, int NT>
__device__ __forceinline__ void finish_tile(const EpilogueLaunch& p, const float* tile, float a0, float a1, int64_t m0,
                                            int64_t n0, int rows_valid, int cols_valid) {
  constexpr int W = kChunk<QUANT>, kPerRow = COLS / W;
  static_assert(COLS % W == 0 && LD % 4 == 0 && UP % 4 == 0, "chunks of a row");
  for (int c = threadIdx.x; c < ROWS * kPerRow; c += NT) {
    const int row = c / kPerRow, col = c % kPerRow * W;
    if (row >= rows_valid || col >= cols_valid) continue;
    float s[W], u[W];
    lds_chunk<W>(s, tile + row * LD + col);
    if constexpr (GATED) lds_chunk<W>(u, tile + row * LD + UP + col);
    u4_t res = {0u, 0u, 0u, 0u};
    if (!GATED && p.res) res = load_residual(p, m0 + row, n0 + col);
    finish<GATED, QUANT>(p, a0, a1, m0 + row, n0 + col, s, u, res);
  }
}

}  // namespace nvfp4
