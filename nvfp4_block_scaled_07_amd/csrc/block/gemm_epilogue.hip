// NVFP4 GEMMs with a fused epilogue: bias, activation and residual
// (nvfp4_gemm_epilogue), and the two projections of a gated feed-forward with
// their product (nvfp4_gemm_gated, nvfp4_gemm_gated_quantize).
//
//   d = bf16( act(alpha A B^T + bias) + beta res )
//   h = act(alpha0 A G^T + bias_g) * (alpha1 A U^T + bias_u)    to bf16 or NVFP4
//
// The main loops are the plain GEMM's; a fused call saves the passes over the
// fp32 or bf16 sums that separate kernels would make (2 to 6 bytes an element
// and one launch each).  A gated tile takes the same columns of G and U, so
// each product is formed where both factors are.
#include "epilogue_tile.h"

namespace nvfp4 {

typedef Cfg<64, 64, 1, 1, 32, 256, 2, 0, 4, 4> EpiTile64k4;
typedef Cfg<128, 128, 2, 2, 32, 256, 2, 0, 1, 2> EpiTile128;
typedef Cfg<64, 64, 1, 1, 32, 256, 2, 0, 4, 4, 16, 0, 0, 1> GatedTile64k4;  // 32 gate and 32 up columns
typedef Cfg<128, 128, 2, 2, 32, 256, 2, 0, 1, 2, 16, 0, 0, 1> GatedTile128;
typedef KCfg<16, 16, 4, 3, 4> EpiReg16x16;
typedef KCfg<32, 16, 4, 3, 4> EpiReg32x16;
typedef KCfg<32, 32, 4, 3, 2> EpiReg32x32;
typedef KCfg<16, 32, 4, 3, 2, 0, 1> GatedReg16x16;  // 16 gate and 16 up columns
typedef KCfg<32, 32, 4, 3, 2, 0, 1> GatedReg32x16;

// Register-streamed tile with a fused epilogue (small M): the K-groups'
// partial tiles are summed in wave order, and over the splits in split order,
// into one fp32 tile in LDS that the epilogue reads.
template <class C, bool QUANT>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_gemm_kreg_epilogue(
    EpilogueLaunch p) {
  __shared__ __attribute__((aligned(16))) float red[C::KS * C::kTileFloats];
  __shared__ __attribute__((aligned(16))) float tile_sum[C::kTileFloats];
  __shared__ int last_flag;
  constexpr int kCols = C::kBlkN * 16;  // output columns of the tile
  const int tiles_n = (int)p.g.tiles_n, S = p.g.splits;
  const int L = xcd_remap(blockIdx.x, (int)(p.g.tiles_m * p.g.tiles_n) * S);
  const int tile = L / S, z = L % S;
  const int64_t m0 = (int64_t)(tile / tiles_n) * C::BM, n0 = (int64_t)(tile % tiles_n) * kCols;
  const int rows_a = (int)min<int64_t>(C::BM, p.g.M - m0), rows_b = (int)min<int64_t>(kCols, p.cols - n0);
  Mfma<16>::Acc acc[C::TM][C::TN];
  kreg_accumulate<C, 0>(p.g, m0, n0, rows_a, rows_b, z, S, acc);
  const int lane = threadIdx.x & 63, wave = wave_id();
  float* mine = red + wave * C::kTileFloats;
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) *(f4_t*)(mine + ((tm * C::TN + tn) * 64 + lane) * 4) = acc[tm][tn];
  __syncthreads();
  const rsrc_t part = partial_rsrc(p.g.ws + kCounterBytes / 4 + (int64_t)tile * S * C::kTileFloats, S, C::kTileFloats);
  for (int x = threadIdx.x; x < C::kTileFloats; x += C::kThreads) {
    const int row = x / C::BN, col = x % C::BN;
    const int rr = row & 15, cc = col & 15;
    const int idx = (((row >> 4) * C::TN + (col >> 4)) * 64 + (rr >> 2) * 16 + cc) * 4 + (rr & 3);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < C::KS; ++w) sum += red[w * C::kTileFloats + idx];
    if (S > 1) store_coherent(part, (uint32_t)(z * C::kTileFloats + x) * 4, sum);
    else tile_sum[x] = sum;
  }
  if (S > 1) {
    // publish the partial, count arrivals, the last split sums all of them
    int* counter = (int*)p.g.ws + tile;
    __builtin_amdgcn_s_waitcnt(0);  // this wave's partial stores are complete
    __syncthreads();
    if (threadIdx.x == 0) last_flag = count_arrival(counter, S);
    __syncthreads();
    if (!last_flag) return;
    for (int x = threadIdx.x; x < C::kTileFloats; x += C::kThreads) {
      float sum = 0.f;
      for (int zz = 0; zz < S; ++zz) sum += load_coherent(part, (uint32_t)(zz * C::kTileFloats + x) * 4);
      tile_sum[x] = sum;
    }
    if (threadIdx.x == 0) reset_counter(counter);
  }
  __syncthreads();
  const float a0 = p.g.alpha ? p.g.alpha[0] : 1.0f;
  const float a1 = C::kGated && p.g.alpha ? p.g.alpha[1] : 1.0f;
  finish_tile<C::kGated, QUANT, C::BM, kCols, C::BN, kCols, C::kThreads>(p, tile_sum, a0, a1, m0, n0, rows_a, rows_b);
}

template <class C, bool QUANT>
static void launch_kreg_epilogue(const EpilogueLaunch& p, unsigned grid, hipStream_t stream) {
  hipLaunchKernelGGL((k_gemm_kreg_epilogue<C, QUANT>), dim3(grid), dim3(C::kThreads), 0, stream, p);
}

// The plain epilogue runs the plain GEMM's plans: the epilogue adds no
// operand traffic to the main loop.
GemmPlan choose_epilogue_plan(int64_t M, int64_t N, int64_t K) {
  GemmPlan pl = choose_plan(M, N, K, kAutoKinds);
  if (pl.kind == 15) {  // never split by the plan's own rule; a forced split is not supported here
    pl.splits = 1;
    pl.workspace = 0;
  }
  return pl;
}

// Gated plans, numbered like the plain GEMM's kinds of the same shape; bn is
// the output columns of a tile (its B has twice as many).
static const PlanKind kGated14 = {"gated256x128w8", 256, 128, 256, false, false, false};
static const PlanKind kGated15 = {"gated128x64", 128, 64, 256, false, false, false};
static const PlanKind kGated9 = {"gated64x32k4", 64, 32, 256, true, false, false, 4};
static const PlanKind kGated10 = {"gatedreg16x16", 16, 16, 256, true, true, false, GatedReg16x16::KS, GatedReg16x16::D};
static const PlanKind kGated12 = {"gatedreg32x16", 32, 16, 256, true, true, false, GatedReg32x16::KS, GatedReg32x16::D};

// The plain GEMM's rules on the tiles of both matrices: register tiles up to
// M = 128 while they need at most one work-group per CU, 256-row tiles once
// they fill the CUs twice, 128-row tiles three times, else split 64-row tiles.
GemmPlan choose_gated_plan(int64_t M, int64_t I, int64_t K) {
  auto tiles = [&](const PlanKind& k) { return ((M + k.bm - 1) / k.bm) * ((I + k.bn - 1) / k.bn); };
  int kind = 9;
  if (M <= 128 && tiles(kGated10) <= kCUs) kind = 10;
  else if (M <= 128 && tiles(kGated12) <= kCUs) kind = 12;
  else if (M <= 32 && tiles(kGated12) <= 4 * kCUs) kind = 12;
  else if (M > 64 && tiles(kGated14) >= 2 * kCUs) kind = 14;
  else if (M > 64 && tiles(kGated15) >= 3 * kCUs) kind = 15;
  int fk = -1, forced_splits = 0;
  if (forced_plan(kForceGemm, &fk, &forced_splits) && (fk == 9 || fk == 10 || fk == 12 || fk == 14 || fk == 15))
    kind = fk;
  else
    forced_splits = 0;
  const PlanKind& k = kind == 14 ? kGated14 : kind == 15 ? kGated15 : kind == 10 ? kGated10 : kind == 12 ? kGated12
                                                                                                   : kGated9;
  GemmPlan pl;
  pl.kind = kind;
  pl.name = k.name;
  pl.tiles_m = (M + k.bm - 1) / k.bm;
  pl.tiles_n = (I + k.bn - 1) / k.bn;
  pl.group_m = 8;
  if (!k.splitk || pl.tiles_m * pl.tiles_n > kCounterBytes / 4) forced_splits = 1;
  PlanKind both = k;  // partial tiles hold both matrices' sums
  both.bn *= 2;
  plan_splits(pl, both, K, forced_splits);
  return pl;
}

hipError_t launch_gemm_epilogue(const GemmPlan& pl, EpilogueLaunch p, hipStream_t stream) {
  p.g.tiles_m = pl.tiles_m;
  p.g.tiles_n = pl.tiles_n;
  p.g.splits = pl.splits;
  p.g.group_m = pl.group_m;
  const unsigned grid = (unsigned)(pl.tiles_m * pl.tiles_n * pl.splits);
  switch (pl.kind) {
    case 10: launch_kreg_epilogue<EpiReg16x16, false>(p, grid, stream); break;
    case 11: launch_kreg_epilogue<EpiReg32x16, false>(p, grid, stream); break;
    case 12: launch_kreg_epilogue<EpiReg32x32, false>(p, grid, stream); break;
    case 14:
    case 16: launch_epilogue_large(pl.kind, p, grid, stream); break;
    case 15: launch_epilogue_tile<EpiTile128, false>(p, grid, stream); break;
    default: launch_epilogue_tile<EpiTile64k4, false>(p, grid, stream); break;
  }
  return hipGetLastError();
}

template <bool QUANT>
static void launch_gated(const GemmPlan& pl, const EpilogueLaunch& p, unsigned grid, hipStream_t stream) {
  switch (pl.kind) {
    case 10: launch_kreg_epilogue<GatedReg16x16, QUANT>(p, grid, stream); break;
    case 12: launch_kreg_epilogue<GatedReg32x16, QUANT>(p, grid, stream); break;
    case 14: launch_gated_large(p, QUANT, grid, stream); break;
    case 15: launch_epilogue_tile<GatedTile128, QUANT>(p, grid, stream); break;
    default: launch_epilogue_tile<GatedTile64k4, QUANT>(p, grid, stream); break;
  }
}

hipError_t launch_gemm_gated(const GemmPlan& pl, EpilogueLaunch p, bool quantize, hipStream_t stream) {
  p.g.tiles_m = pl.tiles_m;
  p.g.tiles_n = pl.tiles_n;
  p.g.splits = pl.splits;
  p.g.group_m = pl.group_m;
  const unsigned grid = (unsigned)(pl.tiles_m * pl.tiles_n * pl.splits);
  if (quantize) launch_gated<true>(pl, p, grid, stream);
  else launch_gated<false>(pl, p, grid, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
