// Eight consecutive bf16 values as one 16-byte access at any 2-byte alignment
// (global accesses of a wave need no more; a misaligned 1 KB run touches one
// line more), and the shorter last group of a row whose length is no multiple
// of 8: 4, 2 and 1 values by the bits of their number, which is uniform, so a
// row's tail costs at most three accesses.
#pragma once
#include "../device.h"

namespace nvfp4 {

typedef u4_t u4_any_t __attribute__((aligned(2)));
typedef u2_t u2_any_t __attribute__((aligned(2)));
typedef uint32_t u1_any_t __attribute__((aligned(2)));

__device__ __forceinline__ u4_t load8(const uint16_t* p) { return *(const u4_any_t*)p; }
__device__ __forceinline__ void store8(uint16_t* p, u4_t w) { *(u4_any_t*)p = w; }

// The first n (< 8, uniform) of 8 values, the others 0.
__device__ __forceinline__ u4_t load_tail8(const uint16_t* p, int n) {
  u4_t w = {0u, 0u, 0u, 0u};
  if (n & 4) {
    const u2_t v = *(const u2_any_t*)p;
    w[0] = v[0];
    w[1] = v[1];
  }
  if (n & 2) {
    const uint32_t v = *(const u1_any_t*)(p + (n & 4));
    if (n & 4) w[2] = v;
    else w[0] = v;
  }
  if (n & 1) {
    const uint32_t v = p[n & 6];
    if ((n & 6) == 6) w[3] = v;
    else if (n & 4) w[2] = v;
    else if (n & 2) w[1] = v;
    else w[0] = v;
  }
  return w;
}

__device__ __forceinline__ void store_tail8(uint16_t* p, u4_t w, int n) {
  if (n & 4) *(u2_any_t*)p = u2_t{w[0], w[1]};
  if (n & 2) *(u1_any_t*)(p + (n & 4)) = n & 4 ? w[2] : w[0];
  if (n & 1) p[n & 6] = (uint16_t)((n & 6) == 6 ? w[3] : n & 4 ? w[2] : n & 2 ? w[1] : w[0]);
}

__device__ __forceinline__ float bf16_at(u4_t w, int e) {
  return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}

__device__ __forceinline__ u4_t to_bf16x8(const float (&v)[8]) {
  return u4_t{f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]), f32x2_to_bf16x2_bits(v[4], v[5]),
              f32x2_to_bf16x2_bits(v[6], v[7])};
}

}  // namespace nvfp4
