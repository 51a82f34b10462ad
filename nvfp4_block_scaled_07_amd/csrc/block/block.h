// Internal interfaces of the block operators: the GEMMs with a fused epilogue
// (gemm_epilogue.hip, gemm_epilogue_large.hip) and the norms around a block
// (norm.hip), between their kernels and their C entry points (block_api.hip).
#pragma once
#include "../internal.h"

namespace nvfp4 {

// An NVFP4 GEMM and what its epilogue does with each fp32 sum s of A B^T
// before the one rounding to the output:
//   plain: d = act(alpha s + bias) + beta res
//   gated: h = act(alpha[0] s_gate + bias_gate) * (alpha[1] s_up + bias_up), B
//          being I gate rows, then I up rows (g.N = 2 I)
// to bf16 (g.d) or, gated only, to NVFP4 (q, sf with encode scale *gs).
struct EpilogueLaunch {
  GemmLaunch g;
  const uint16_t* bias;  // bf16 [g.N], or NULL
  const uint16_t* res;   // bf16 [M][cols], row stride ldr, or NULL
  int64_t ldr, ldd;      // row strides of res and of g.d, in elements
  int64_t cols;          // output columns: N, or I
  float beta;
  int act;
  const float* gs;
  uint8_t* q;
  uint8_t* sf;
};

GemmPlan choose_epilogue_plan(int64_t M, int64_t N, int64_t K);
GemmPlan choose_gated_plan(int64_t M, int64_t I, int64_t K, bool quantize);
hipError_t launch_gemm_epilogue(const GemmPlan& plan, EpilogueLaunch p, hipStream_t stream);
// quantize: NVFP4 output instead of bf16 (cols % 16 == 0)
hipError_t launch_gemm_gated(const GemmPlan& plan, EpilogueLaunch p, bool quantize, hipStream_t stream);
// The unsplit 256-row tiles, in gemm_epilogue_large.hip (their own instruction
// schedule): kind 14 or 16 of the plain epilogue, 14 of the gated one.
void launch_epilogue_large(int kind, const EpilogueLaunch& p, unsigned grid, hipStream_t stream);
void launch_gated_large(const EpilogueLaunch& p, bool quantize, unsigned grid, hipStream_t stream);

// r = beta res + gate post(x); y = norm(r)  (norm.hip)
struct NormLaunch {
  const uint16_t* x;
  const uint16_t* post_w;
  const uint16_t* post_b;
  const uint16_t* gate;
  const uint16_t* res;
  const uint16_t* w;
  const uint16_t* b;
  uint16_t* r;
  uint16_t* y;
  const float* gs;
  uint8_t* q;
  uint8_t* sf;
  int64_t t0, T, H;              // rows t0 .. T - 1 of a launch
  int64_t ldx, ldres, ldr, ldy;  // row strides in elements
  int64_t gate_group;            // rows that share a gate row; 0: all of them
  float beta, eps;
  double inv_h;                  // 1 / H
  int layer;                     // 0: RMS, 1: mean removed first
};
hipError_t launch_residual_norm(NormLaunch p, hipStream_t stream);

}  // namespace nvfp4
