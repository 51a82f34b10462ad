// The norms before and after a block, fused with its gate and residual:
//
//   u = post(x)                      post(x) = norm of x with post_w, post_b; or x
//   r = beta res + gate u            gate: one row for all, or one per gate_group rows; or 1
//   y = norm(r) with w, b            to bf16 and / or NVFP4
//
//   norm(v) = (v - m) rstd w + b,  rstd = 1 / sqrt(mean((v - m)^2) + eps),
//   m = mean(v) (layer norm) or 0 (RMS norm)
//
// One pass over memory: a row's chunks of 8 columns stay in the registers of
// the threads that own them from the first load to the last store, so x and
// res are read once and r, y written once; every load (the vectors too) is
// issued before the first sum.  Bound by HBM for long inputs and by one
// memory round trip plus the launch for a few rows.
//
// Arithmetic: the sums of a row (mean, mean square) and rstd are in fp64 and
// rstd is rounded once to fp32, which makes it independent of the order of
// the sum to within one rounding in 2^29; everything else is fp32, one
// rounding per step in the formulas' order (r is not rounded to bf16 before
// the second norm).  Built without fp contraction, so a plain evaluation of
// the same steps gives the same bits, the NVFP4 codes and scales among them.
// The fp64 sums cost two instructions an element, far below the memory time.
#include "../device.h"
#include "block.h"

namespace nvfp4 {

// The 8 columns of chunk c of a row as packed bf16; columns past H are 0.
template <bool VEC>
__device__ __forceinline__ u4_t load_chunk(const uint16_t* row, int64_t c, int64_t H) {
  if constexpr (VEC) return c * 8 < H ? ((const u4_t*)row)[c] : u4_t{0u, 0u, 0u, 0u};
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = c * 8 + e < H ? row[c * 8 + e] : 0u;
  return u4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

template <bool VEC>
__device__ __forceinline__ void store_chunk(uint16_t* row, int64_t c, int64_t H, const float (&v)[8]) {
  const u4_t w = {f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]),
                  f32x2_to_bf16x2_bits(v[4], v[5]), f32x2_to_bf16x2_bits(v[6], v[7])};
  if constexpr (VEC) {
    if (c * 8 < H) ((u4_t*)row)[c] = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c * 8 + e < H) row[c * 8 + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

__device__ __forceinline__ float bf16_at(u4_t w, int e) {
  return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}

// Sum over the TPR threads of a row, in a fixed order, to all of them.
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* cell) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    __syncthreads();  // the cells' last readers are done
    if ((threadIdx.x & 63) == 0) cell[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += cell[w];
  }
  return v;
}

// mean (0 for RMS) and rstd of one row from its sums
struct Stats {
  double mean;
  float rstd;
};

__device__ __forceinline__ float rstd_of(double sq, int64_t H, float eps) {
  return (float)(1.0 / sqrt(sq / (double)H + (double)eps));
}

__device__ __forceinline__ float normed(float v, const Stats& s, bool layer, float w, bool has_w, float b, bool has_b) {
  float y = (layer ? (float)((double)v - s.mean) : v) * s.rstd;
  if (has_w) y = y * w;
  if (has_b) y = y + b;
  return y;
}

// Statistics of a row held as V chunks of 8 per thread.
template <int TPR, int V, bool VEC>
__device__ __forceinline__ Stats row_stats(const float (&v)[V][8], int tid, const NormLaunch& p, double* cell) {
  Stats s{0.0, 0.0f};
  if (p.layer) {
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) a += (double)v[i][e];  // columns past H are 0
    s.mean = row_sum<TPR>(a, cell) / (double)p.H;
  }
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = (int64_t)i * TPR + tid;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = (double)v[i][e] - s.mean;
      if (VEC ? c * 8 < p.H : c * 8 + e < p.H) q = __builtin_fma(d, d, q);
    }
  }
  s.rstd = rstd_of(row_sum<TPR>(q, cell), p.H, p.eps);
  return s;
}

template <int TPR, int V, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_residual_norm(NormLaunch p) {
  constexpr int WG = TPR < 256 ? 256 : TPR;
  __shared__ double cell[WG / 64];
  const int64_t t = (int64_t)blockIdx.x * (WG / TPR) + threadIdx.x / TPR;
  if (t >= p.T) return;  // whole waves: a row has 64 threads, or the work-group
  const int tid = threadIdx.x % TPR;
  const int64_t H = p.H;
  const int64_t gt = p.gate_group > 0 ? t / p.gate_group : 0;
  u4_t x[V], res[V], pw[V], pb[V], g[V], w[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = (int64_t)i * TPR + tid;
    x[i] = load_chunk<VEC>(p.x + t * p.ldx, c, H);
    if (p.res) res[i] = load_chunk<VEC>(p.res + t * p.ldres, c, H);
    if (p.post_w) pw[i] = load_chunk<VEC>(p.post_w, c, H);
    if (p.post_b) pb[i] = load_chunk<VEC>(p.post_b, c, H);
    if (p.gate) g[i] = load_chunk<VEC>(p.gate + gt * H, c, H);
    if (p.w) w[i] = load_chunk<VEC>(p.w, c, H);
    if (p.b) b[i] = load_chunk<VEC>(p.b, c, H);
  }
  float v[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = bf16_at(x[i], e);
  if (p.post_w) {
    const Stats s = row_stats<TPR, V, VEC>(v, tid, p, cell);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = (int64_t)i * TPR + tid;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = normed(v[i][e], s, p.layer, bf16_at(pw[i], e), true, p.post_b ? bf16_at(pb[i], e) : 0.0f, p.post_b);
        v[i][e] = (VEC ? c * 8 < H : c * 8 + e < H) ? u : 0.0f;  // columns past H stay out of the sums
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.gate) v[i][e] = bf16_at(g[i], e) * v[i][e];
      if (p.res) v[i][e] = p.beta * bf16_at(res[i], e) + v[i][e];
    }
  if (p.r) {
#pragma unroll
    for (int i = 0; i < V; ++i) store_chunk<VEC>(p.r + t * p.ldr, (int64_t)i * TPR + tid, H, v[i]);
  }
  if (!p.y && !p.q) return;
  const Stats s = row_stats<TPR, V, VEC>(v, tid, p, cell);
  const float gs = p.q && p.gs ? *p.gs : 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = (int64_t)i * TPR + tid;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[i][e] = normed(v[i][e], s, p.layer, p.w ? bf16_at(w[i], e) : 1.0f, p.w, p.b ? bf16_at(b[i], e) : 0.0f, p.b);
    if (p.y) store_chunk<VEC>(p.y + t * p.ldy, c, H, v[i]);
    if (p.q && c * 8 < H) {
      // H % 16 == 0: the lanes of a pair hold the two halves of a block
      uint32_t codes;
      const uint32_t sf = quantize_half_block16(f4_t{v[i][0], v[i][1], v[i][2], v[i][3]},
                                                f4_t{v[i][4], v[i][5], v[i][6], v[i][7]}, gs, codes);
      ((uint32_t*)(p.q + t * (H / 2)))[c] = codes;
      if ((c & 1) == 0) p.sf[t * (H / 16) + c / 2] = (uint8_t)sf;
    }
  }
}

// Rows too long for the registers: the same steps with the row read again for
// each sum, one work-group per row.  A thread stores only columns it reads,
// after its last read of them, so r may be x or res here too.
template <bool VEC>
__global__ __launch_bounds__(1024) void k_residual_norm_long(NormLaunch p) {
  constexpr int TPR = 1024;
  __shared__ double cell[TPR / 64];
  const int64_t t = blockIdx.x, H = p.H;
  const int64_t gt = p.gate_group > 0 ? t / p.gate_group : 0;
  const int tid = threadIdx.x;
  const int64_t n8 = (H + 7) / 8;
  Stats sx{0.0, 0.0f};
  if (p.post_w) {
    if (p.layer) {
      double a = 0.0;
      for (int64_t c = tid; c < n8; c += TPR) {
        const u4_t x = load_chunk<VEC>(p.x + t * p.ldx, c, H);
        for (int e = 0; e < 8; ++e) a += (double)bf16_at(x, e);
      }
      sx.mean = row_sum<TPR>(a, cell) / (double)H;
    }
    double q = 0.0;
    for (int64_t c = tid; c < n8; c += TPR) {
      const u4_t x = load_chunk<VEC>(p.x + t * p.ldx, c, H);
      for (int e = 0; e < 8; ++e) {
        const double d = (double)bf16_at(x, e) - sx.mean;
        if (c * 8 + e < H) q = __builtin_fma(d, d, q);
      }
    }
    sx.rstd = rstd_of(row_sum<TPR>(q, cell), H, p.eps);
  }
  auto r_chunk = [&](int64_t c, float (&v)[8]) {
    const u4_t none = {0u, 0u, 0u, 0u};
    const u4_t x = load_chunk<VEC>(p.x + t * p.ldx, c, H);
    const u4_t res = p.res ? load_chunk<VEC>(p.res + t * p.ldres, c, H) : none;
    const u4_t pw = p.post_w ? load_chunk<VEC>(p.post_w, c, H) : none, pb = p.post_b ? load_chunk<VEC>(p.post_b, c, H) : none;
    const u4_t g = p.gate ? load_chunk<VEC>(p.gate + gt * H, c, H) : none;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = bf16_at(x, e);
      if (p.post_w) v[e] = normed(v[e], sx, p.layer, bf16_at(pw, e), true, bf16_at(pb, e), p.post_b);
      if (p.gate) v[e] = bf16_at(g, e) * v[e];
      if (p.res) v[e] = p.beta * bf16_at(res, e) + v[e];
    }
  };
  Stats s{0.0, 0.0f};
  const bool norm = p.y || p.q;
  if (norm && p.layer) {
    double a = 0.0;
    for (int64_t c = tid; c < n8; c += TPR) {
      float v[8];
      r_chunk(c, v);
      for (int e = 0; e < 8; ++e)
        if (c * 8 + e < H) a += (double)v[e];
    }
    s.mean = row_sum<TPR>(a, cell) / (double)H;
  }
  if (norm) {
    double q = 0.0;
    for (int64_t c = tid; c < n8; c += TPR) {
      float v[8];
      r_chunk(c, v);
      for (int e = 0; e < 8; ++e) {
        const double d = (double)v[e] - s.mean;
        if (c * 8 + e < H) q = __builtin_fma(d, d, q);
      }
    }
    s.rstd = rstd_of(row_sum<TPR>(q, cell), H, p.eps);
  }
  const float gs = p.q && p.gs ? *p.gs : 1.0f;
  for (int64_t c = tid; c < n8; c += TPR) {
    float v[8];
    r_chunk(c, v);
    if (p.r) store_chunk<VEC>(p.r + t * p.ldr, c, H, v);
    if (!norm) continue;
    const u4_t none = {0u, 0u, 0u, 0u};
    const u4_t w = p.w ? load_chunk<VEC>(p.w, c, H) : none, b = p.b ? load_chunk<VEC>(p.b, c, H) : none;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = normed(v[e], s, p.layer, bf16_at(w, e), p.w, bf16_at(b, e), p.b);
    if (p.y) store_chunk<VEC>(p.y + t * p.ldy, c, H, v);
    if (p.q) {
      uint32_t codes;
      const uint32_t sf = quantize_half_block16(f4_t{v[0], v[1], v[2], v[3]}, f4_t{v[4], v[5], v[6], v[7]}, gs, codes);
      ((uint32_t*)(p.q + t * (H / 2)))[c] = codes;
      if ((c & 1) == 0) p.sf[t * (H / 16) + c / 2] = (uint8_t)sf;
    }
  }
}

template <int TPR, int V>
static void launch_norm(const NormLaunch& p, hipStream_t stream) {
  constexpr int WG = TPR < 256 ? 256 : TPR, kRows = WG / TPR;
  const unsigned grid = (unsigned)((p.T + kRows - 1) / kRows);
  if (p.vec) hipLaunchKernelGGL((k_residual_norm<TPR, V, true>), dim3(grid), dim3(WG), 0, stream, p);
  else hipLaunchKernelGGL((k_residual_norm<TPR, V, false>), dim3(grid), dim3(WG), 0, stream, p);
}

hipError_t launch_residual_norm(const NormLaunch& p, hipStream_t stream) {
  const int64_t n8 = (p.H + 7) / 8;
  if (n8 <= 64) launch_norm<64, 1>(p, stream);
  else if (n8 <= 128) launch_norm<64, 2>(p, stream);
  else if (n8 <= 256) launch_norm<256, 1>(p, stream);
  else if (n8 <= 512) launch_norm<256, 2>(p, stream);
  else if (n8 <= 768) launch_norm<256, 3>(p, stream);
  else if (n8 <= 1024) launch_norm<512, 2>(p, stream);
  else if (n8 <= 2048) launch_norm<1024, 2>(p, stream);
  else if (p.vec) hipLaunchKernelGGL((k_residual_norm_long<true>), dim3((unsigned)p.T), dim3(1024), 0, stream, p);
  else hipLaunchKernelGGL((k_residual_norm_long<false>), dim3((unsigned)p.T), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
