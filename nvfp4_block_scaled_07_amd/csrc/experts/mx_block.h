// MXFP4 quantisation of one block of 32 elements, shared by the quantise
// kernels and the grouped product that writes MXFP4 rows.
//
// With p the block's largest magnitude and e its scale's exponent (byte e +
// 127), the codes are e2m1_rne(x 2^-e), saturating, sign kept.  e is
//   rule 0: floor(log2 p) - 2, the OCP Microscaling v1.0 conversion: p 2^-e
//           lies in [4, 8), what lies above 6 saturates;
//   rule 1: the least e with p <= 6 2^e, so that nothing up to 6 2^125 saturates;
// limited to bytes 0 .. 252 (252: the largest scale whose codes are all finite
// fp32 values).  2^-e is a power of two, so x 2^-e is exact (bytes 0 .. 252
// give 2^127 .. 2^-125; a product that underflows is far below the rounding to
// 0) and the only roundings are those of the codes.
//
// A block that holds a NaN gets scale byte 0xFF (the E8M0 NaN) and codes 0, so
// that what reads it is NaN; infinities saturate.  The magnitudes are compared
// as bits (non-negative floats order like them, NaN above infinity).
#pragma once
#include "../block/quantize_block.h"

namespace nvfp4 {

struct MxScale {
  uint32_t byte, keep;  // scale byte, mask of the code words
  float r;              // 2^-e
};

__device__ __forceinline__ MxScale mx_scale(uint32_t peak, int rule) {
  int b = (int)(peak >> 23) - 2;
  if (rule == 1 && (peak & 0x7FFFFFu) > 0x400000u) ++b;
  b = b < 0 ? 0 : b > 252 ? 252 : b;
  const bool nan = peak > 0x7F800000u;
  // 2^(127 - b): exponent field 254 - b, never below 2
  return MxScale{nan ? 0xFFu : (uint32_t)b, nan ? 0u : ~0u, __uint_as_float((uint32_t)(254 - b) << 23)};
}

// A block that a DPP quad holds, 8 elements a lane: w, those of this lane.
__device__ __forceinline__ uint32_t mx_quantize_quad(f4_t lo, f4_t hi, int rule, uint32_t& w) {
  uint32_t a = umax(magnitude(lo), magnitude(hi));
  a = umax(a, dpp<kDppXor1>(a));
  a = umax(a, dpp<kDppXor2>(a));
  const MxScale s = mx_scale(a, rule);
  w = e2m1x8(lo, hi, s.r) & s.keep;
  return s.byte;
}

}  // namespace nvfp4
