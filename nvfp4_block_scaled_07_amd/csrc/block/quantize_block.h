// NVFP4 quantisation in the block operators: the steps of nvfp4_quantize
// (quantize_block16 in device.h, the same codes and scales for finite blocks),
// and one rule for NaN, which that function leaves open: a block that holds a
// NaN gets scale byte 0x7F (the e4m3 NaN) and codes 0, however its elements
// are spread over lanes, so that every product with it is NaN.  The rows that a
// norm makes NaN as a whole, and the tokens behind them, would otherwise turn
// into zeros or into saturated values.  Infinities saturate: scale 448, code 6.
//
// The block's largest magnitude is taken over the bits (non-negative floats
// order like them, and NaN lies above infinity), which costs what the
// maximum of the values does.
#pragma once
#include "../device.h"

namespace nvfp4 {

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t magnitude(f4_t x) {
  return umax(umax(magnitude(x[0]), magnitude(x[1])), umax(magnitude(x[2]), magnitude(x[3])));
}

// The scale code of a block from its largest magnitude, the factor r of its
// elements and a mask for their code words.
struct BlockScale {
  uint32_t code, keep;
  float r;
};

__device__ __forceinline__ BlockScale block_scale(uint32_t peak, float gs) {
  const bool nan = peak > 0x7F800000u;
  const uint32_t code = e4m3_encode_pos((__uint_as_float(peak) / 6.0f) * gs);
  const float sv = e4m3_value_pos(code);
  return BlockScale{nan ? 0x7Fu : code, nan ? 0u : ~0u, sv == 0.0f ? 0.0f : gs / sv};
}

// A block whose 16 elements one lane holds: returns the scale code; w[0] the
// codes of elements 0..7, w[1] of 8..15.
__device__ __forceinline__ uint32_t quantize_lane16(const f4_t (&v)[4], float gs, uint32_t (&w)[2]) {
  const BlockScale s =
      block_scale(umax(umax(magnitude(v[0]), magnitude(v[1])), umax(magnitude(v[2]), magnitude(v[3]))), gs);
  w[0] = e2m1x8(v[0], v[1], s.r) & s.keep;
  w[1] = e2m1x8(v[2], v[3], s.r) & s.keep;
  return s.code;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
// within a quad: lane ^ 1, lane ^ 2; within a row of 16: mirrors of 8 and 16
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// A block that the lanes l and l ^ 1 hold, 8 elements each: w, those of this lane.
__device__ __forceinline__ uint32_t quantize_pair16(f4_t lo, f4_t hi, float gs, uint32_t& w) {
  const uint32_t a = umax(magnitude(lo), magnitude(hi));
  const BlockScale s = block_scale(umax(a, dpp<kDppXor1>(a)), gs);
  w = e2m1x8(lo, hi, s.r) & s.keep;
  return s.code;
}

// A block that the 16 lanes of a DPP row hold, one element each; every lane of
// the row must be active.  codes: those of the lane's 8 elements (its half of
// the row).
__device__ __forceinline__ uint32_t quantize_row16(float x, float gs, uint32_t& codes) {
  uint32_t a = magnitude(x);
  a = umax(a, dpp<kDppXor1>(a));
  a = umax(a, dpp<kDppXor2>(a));
  a = umax(a, dpp<kDppHalfMirror>(a));
  a = umax(a, dpp<kDppMirror>(a));
  const BlockScale s = block_scale(a, gs);
  const float v = x * s.r;
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, v, 1.0f, 0) & 15u & s.keep;
  w <<= 4 * (threadIdx.x & 7);
  w |= dpp<kDppXor1>(w);
  w |= dpp<kDppXor2>(w);
  codes = w | dpp<kDppHalfMirror>(w);
  return s.code;
}

}  // namespace nvfp4
