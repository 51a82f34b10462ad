// MXFP4 quantisation of fp32 arrays and of (gathered) bf16 rows.
//
// Four lanes share a block of 32: a lane takes 8 consecutive elements (16
// bytes of bf16, 32 of fp32), the block's peak is two DPP steps away, every
// lane stores its 4 code bytes and one of the four the scale byte, so loads and
// code stores of a wave are whole consecutive lines.  Bound by HBM.
#include "experts.h"
#include "mx_block.h"

namespace nvfp4 {

// Chunks of 8 elements a thread has in flight, a grid's width apart.
constexpr int kMxChunks = 4;

template <bool BF16>
struct Chunk8;
template <>
struct Chunk8<false> {
  f4_t v[2];
  __device__ __forceinline__ void load(const void* x, int64_t c) {
    v[0] = ((const f4_t*)x)[2 * c];
    v[1] = ((const f4_t*)x)[2 * c + 1];
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = f4_t{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void values(f4_t& lo, f4_t& hi) const {
    lo = v[0];
    hi = v[1];
  }
};
template <>
struct Chunk8<true> {
  u4_t v;
  __device__ __forceinline__ void load(const void* x, int64_t c) { v = ((const u4_t*)x)[c]; }
  __device__ __forceinline__ void zero() { v = u4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void values(f4_t& lo, f4_t& hi) const { bf16x8_to_f32(v, lo, hi); }
};

// nc chunks in order (a multiple of 4, so a quad is inside or outside as a whole).
template <bool BF16>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ x, int64_t nc, int rule,
                                                     uint32_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t c0 = (int64_t)blockIdx.x * 256 + threadIdx.x; c0 < nc; c0 += kMxChunks * stride) {
    Chunk8<BF16> v[kMxChunks];
#pragma unroll
    for (int j = 0; j < kMxChunks; ++j) {
      const int64_t c = c0 + j * stride;
      if (c < nc) v[j].load(x, c);
      else v[j].zero();
    }
#pragma unroll
    for (int j = 0; j < kMxChunks; ++j) {
      const int64_t c = c0 + j * stride;
      f4_t lo, hi;
      v[j].values(lo, hi);
      uint32_t w;
      const uint32_t byte = mx_quantize_quad(lo, hi, rule, w);
      if (c < nc) {
        q[c] = w;
        if ((threadIdx.x & 3) == 0) sf[c >> 2] = (uint8_t)byte;
      }
    }
  }
}

// Gathered rows: a row's chunks lie a work-group's or a part of one's threads
// apart, so that no chunk index is divided.  Tokens outside [0, T) give zero rows.
__global__ __launch_bounds__(256) void k_mx_quantize_rows(const u4_t* __restrict__ x, const int32_t* __restrict__ tok,
                                                          int64_t rows, int64_t T, int kc, int tpr, int rule,
                                                          uint32_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const int lane = threadIdx.x & (tpr - 1), per = 256 / tpr;
  for (int64_t i = (int64_t)blockIdx.x * per + threadIdx.x / tpr; i < rows; i += (int64_t)gridDim.x * per) {
    const int64_t t = tok[i];
    const bool in = t >= 0 && t < T;
    const u4_t* src = x + (in ? t : 0) * kc;
    for (int c0 = lane; c0 < kc; c0 += kMxChunks * tpr) {
      Chunk8<true> v[kMxChunks];
#pragma unroll
      for (int j = 0; j < kMxChunks; ++j) {
        const int c = c0 + j * tpr;
        if (in && c < kc) v[j].load(src, c);
        else v[j].zero();
      }
#pragma unroll
      for (int j = 0; j < kMxChunks; ++j) {
        const int c = c0 + j * tpr;
        f4_t lo, hi;
        v[j].values(lo, hi);
        uint32_t w;
        const uint32_t byte = mx_quantize_quad(lo, hi, rule, w);
        if (c < kc) {
          q[i * kc + c] = w;
          if ((c & 3) == 0) sf[i * (kc >> 2) + (c >> 2)] = (uint8_t)byte;
        }
      }
    }
  }
}

// about 8 work-groups (32 waves) per CU
static unsigned quantize_grid(int64_t nc) {
  const int64_t blocks = (nc + 256 * kMxChunks - 1) / (256 * kMxChunks);
  return (unsigned)(blocks > 2048 ? 2048 : blocks);
}

hipError_t launch_mx_quantize(const float* x, int64_t n, int rule, uint8_t* q, uint8_t* sf, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(k_mx_quantize<false>, dim3(quantize_grid(n / 8)), dim3(256), 0, stream, x, n / 8, rule,
                     (uint32_t*)q, sf);
  return hipGetLastError();
}

hipError_t launch_mx_quantize_rows(const uint16_t* x, const int32_t* row_token, int64_t rows, int64_t T, int64_t K,
                                   int rule, uint8_t* q, uint8_t* sf, hipStream_t stream) {
  if (rows == 0 || K == 0) return hipSuccess;
  if (!row_token) {
    const int64_t nc = rows * (K / 8);
    hipLaunchKernelGGL(k_mx_quantize<true>, dim3(quantize_grid(nc)), dim3(256), 0, stream, x, nc, rule, (uint32_t*)q, sf);
    return hipGetLastError();
  }
  // threads of a row: the smallest power of two that holds its chunks, 4 to 256
  const int kc = (int)(K / 8);
  int tpr = 4;
  while (tpr < 256 && tpr < kc) tpr *= 2;
  int64_t blocks = (rows + 256 / tpr - 1) / (256 / tpr);
  if (blocks > 1 << 20) blocks = 1 << 20;
  hipLaunchKernelGGL(k_mx_quantize_rows, dim3((unsigned)blocks), dim3(256), 0, stream, (const u4_t*)x, row_token, rows,
                     T, kc, tpr, rule, (uint32_t*)q, sf);
  return hipGetLastError();
}

}  // namespace nvfp4
