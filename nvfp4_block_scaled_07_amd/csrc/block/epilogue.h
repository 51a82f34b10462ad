// Epilogues of the block GEMMs: what happens to a tile's fp32 sums between
// the last MFMA and the one rounding to the output.
//
// The MFMA layouts give a lane one column and rows four apart, so its own
// accumulators touch 2 bytes of a row.  Every epilogue therefore passes the
// sums through LDS (free by then: the main loop's stages are done) and reads
// them back with 8 or 16 consecutive columns of one row per lane: bias,
// residual and output move as 16-byte vectors, a gate column meets its up
// column in one lane, and a 16-element NVFP4 block belongs to one lane, which
// quantises it with no cross-lane step.
//
// Arithmetic is fp32, in the order of the formulas, one rounding per step and
// one rounding to bf16 (or to e4m3 and e2m1) at the end.  The sums and the
// hidden layer are never rounded to bf16 in between.
#pragma once

#include "../kreg_tile.h"
#include "block.h"

namespace nvfp4 {

// 1 / (1 + exp(-x)) from the hardware exp2 and reciprocal (1 ulp each).  The
// argument's rounding adds |x| 2^-24 relative error where the value is small;
// both stay far below half a bf16 step (2^-9).  exp2 overflows to infinity and
// the reciprocal gives 0, the limit; NaN stays NaN.
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {  // uniform
    case 1: return x < 0.0f ? 0.0f : x;  // NaN stays NaN
    case 2: return 0.5f * x * erfcf(x * -0.70710678f);
    // 0.5 x (1 + tanh(z)) = x sigmoid(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3)
    case 3: return x * sigmoid_f32(1.59576912f * (x + 0.044715f * x * x * x));
    case 4: return x * sigmoid_f32(x);
    default: return x;
  }
}

// W (a multiple of 8) bf16 values at p, columns [col, cols) valid, as fp32;
// the others are 0.  vec: p is 16-byte aligned when col is a multiple of 8.
template <int W>
__device__ __forceinline__ void load_bf16(float (&v)[W], const uint16_t* p, int64_t col, int64_t cols, bool vec) {
  if (vec && col + W <= cols) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      f4_t lo, hi;
      bf16x8_to_f32(*(const u4_t*)(p + 8 * i), lo, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * i + e] = lo[e];
        v[8 * i + 4 + e] = hi[e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = col + i < cols ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f;
  }
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float (&v)[8], int64_t col, int64_t cols, bool vec) {
  if (vec && col + 8 <= cols) {
    *(u4_t*)p = u4_t{f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]),
                     f32x2_to_bf16x2_bits(v[4], v[5]), f32x2_to_bf16x2_bits(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) p[i] = f32_to_bf16_bits(v[i]);
  }
}

// Columns a lane takes at once: one 16-byte bf16 vector, or one NVFP4 block.
template <bool QUANT>
constexpr int kChunk = QUANT ? 16 : 8;

// The epilogue of columns [col, col + W) of one row, from the sums s (gate or
// only) and u (up) of those columns.
template <bool GATED, bool QUANT>
__device__ __forceinline__ void finish(const EpilogueLaunch& p, float a0, float a1, int64_t row, int64_t col,
                                       const float (&s)[kChunk<QUANT>], const float (&u)[kChunk<QUANT>]) {
  constexpr int W = kChunk<QUANT>;
  float v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = a0 * s[i];
  if (p.bias) {
    float b[W];
    load_bf16<W>(b, p.bias + col, col, p.cols, p.vec);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += b[i];
  }
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = activate(v[i], p.act);
  if constexpr (GATED) {
    float t[W];
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = a1 * u[i];
    if (p.bias) {
      float b[W];
      load_bf16<W>(b, p.bias + p.cols + col, col, p.cols, p.vec);
#pragma unroll
      for (int i = 0; i < W; ++i) t[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= t[i];
  } else if (p.res) {
    float r[W];
    load_bf16<W>(r, p.res + row * p.ldr + col, col, p.cols, p.vec);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += p.beta * r[i];
  }
  if constexpr (QUANT) {
    // cols % 16 == 0: the block is whole
    f4_t x[4];
#pragma unroll
    for (int i = 0; i < W; ++i) x[i / 4][i % 4] = v[i];
    uint32_t w[2];
    const uint32_t code = quantize_block16(x, p.gs ? *p.gs : 1.0f, w);
    *(u2_t*)(p.q + row * (p.cols / 2) + col / 2) = u2_t{w[0], w[1]};
    p.sf[row * (p.cols / 16) + col / 16] = (uint8_t)code;
  } else {
    store_bf16x8(p.g.d + row * p.ldd + col, v, col, p.cols, p.vec);
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

// Epilogue of a tile whose sums lie in LDS, row-major with stride LD (gated:
// gate columns, then up columns from UP on), by NT threads.
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
    finish<GATED, QUANT>(p, a0, a1, m0 + row, n0 + col, s, u);
  }
}

}  // namespace nvfp4
