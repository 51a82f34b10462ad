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
typedef KCfg<16, 32, 4, 3, 3> EpiReg16x32;
typedef KCfg<16, 32, 8, 2, 2> EpiReg16x32k8;
typedef KCfg<16, 32, 4, 3, 2, 0, 1> GatedReg16x16;  // 16 gate and 16 up columns
typedef KCfg<16, 64, 4, 2, 2, 0, 1> GatedReg16x32;
typedef KCfg<32, 32, 4, 3, 2, 0, 1> GatedReg32x16;

// Register-streamed tile with a fused epilogue (small M).  What the epilogue
// reads besides the sums (alpha, bias, residual) is loaded before the main
// loop, so that after the K-groups' sum (in wave order, and over the splits
// in split order) only arithmetic and one store remain.  A thread owns single
// outputs, 16 consecutive lanes 16 columns of a row: one NVFP4 block.
//
// SKIP leaves the products of K units past the end of a wave's share out
// instead of adding zeros (one token 6144 x 2048: 5.7 us against 6.3, 61 x 777 x
// 1280: 4.4 against 5.0); where every slot is filled its branches only cut the
// instruction schedule (1 x 4096 x 6144: 7.5 against 7.05), so the launcher
// picks by the shape.
template <class C, bool QUANT, bool SKIP>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_gemm_kreg_epilogue(
    EpilogueLaunch p) {
  __shared__ __attribute__((aligned(16))) float red[C::KS * C::kTileFloats];
  __shared__ int last_flag;
  constexpr bool kGated = C::kGated;
  constexpr int kCols = C::kBlkN * 16;  // output columns of the tile
  constexpr int kOut = C::BM * kCols, kPer = (kOut + C::kThreads - 1) / C::kThreads;
  static_assert(kCols % 16 == 0, "whole NVFP4 blocks in a row of lanes");
  const int tiles_n = (int)p.g.tiles_n, S = p.g.splits;
  const int L = xcd_remap(blockIdx.x, (int)(p.g.tiles_m * p.g.tiles_n) * S);
  // uniform shortcuts past the integer divisions (about 100 cycles each) for
  // unsplit calls and for one row of tiles
  const int tile = S == 1 ? L : L / S, z = L - tile * S;
  const int tm = p.g.tiles_m == 1 ? 0 : tile / tiles_n;
  const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)(tile - tm * tiles_n) * kCols;
  const int rows_a = (int)min<int64_t>(C::BM, p.g.M - m0), rows_b = (int)min<int64_t>(kCols, p.cols - n0);
  const float a0 = p.g.alpha ? p.g.alpha[0] : 1.0f;
  const float a1 = kGated && p.g.alpha ? p.g.alpha[1] : 1.0f;
  const float gs = QUANT && p.gs ? *p.gs : 1.0f;
  Scalars sc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int x = threadIdx.x + k * C::kThreads, row = x / kCols, col = x % kCols;
    sc[k] = load_scalars<kGated>(p, a0, a1, m0 + row, n0 + col, row < rows_a && col < rows_b);
  }
  Mfma<16>::Acc acc[C::TM][C::TN];
  kreg_accumulate<C, 0, SKIP>(p.g, m0, n0, rows_a, rows_b, z, S, acc);
  const int lane = threadIdx.x & 63, wave = wave_id();
  float* mine = red + wave * C::kTileFloats;
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) *(f4_t*)(mine + ((tm * C::TN + tn) * 64 + lane) * 4) = acc[tm][tn];
  __syncthreads();
  // the K-groups' sum of the tile's element (row, col), col < BN
  auto group_sum = [&](int row, int col) {
    const int idx = (((row >> 4) * C::TN + (col >> 4)) * 64 + ((row & 15) >> 2) * 16 + (col & 15)) * 4 + (row & 3);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < C::KS; ++w) sum += red[w * C::kTileFloats + idx];
    return sum;
  };
  const rsrc_t part = partial_rsrc(p.g.ws + kCounterBytes / 4 + (int64_t)tile * S * C::kTileFloats, S, C::kTileFloats);
  if (S > 1) {
    // publish the partial, count arrivals; the last split goes on
    for (int x = threadIdx.x; x < C::kTileFloats; x += C::kThreads)
      store_coherent(part, (uint32_t)(z * C::kTileFloats + x) * 4, group_sum(x / C::BN, x % C::BN));
    int* counter = (int*)p.g.ws + tile;
    __builtin_amdgcn_s_waitcnt(0);  // this wave's partial stores are complete
    __syncthreads();
    if (threadIdx.x == 0) last_flag = count_arrival(counter, S);
    __syncthreads();
    if (!last_flag) return;
    if (threadIdx.x == 0) reset_counter(counter);
  }
  // Over the splits, in split order; this split's own partial comes from LDS,
  // and the others' loads go out four at a time (one after the other they cost
  // a round trip each, 0.4 us; past the last split they read as zero).
  auto total = [&](int row, int col) {
    const float own = group_sum(row, col);
    if (S == 1) return own;
    float sum = 0.f;
    for (int z0 = 0; z0 < S; z0 += 4) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = load_coherent(part, (uint32_t)((z0 + i) * C::kTileFloats + row * C::BN + col) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += z0 + i == z ? own : v[i];
    }
    return sum;
  };
  // all of a thread's sums before the first use
  float s0[kPer], s1[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int x = threadIdx.x + k * C::kThreads, row = x / kCols, col = x % kCols;
    if (x >= kOut) break;
    s0[k] = total(row, col);
    s1[k] = kGated ? total(row, kCols + col) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int x = threadIdx.x + k * C::kThreads, row = x / kCols, col = x % kCols;
    if (x >= kOut) break;  // whole waves
    const float v = finish_one<kGated>(p, sc[k], s0[k], s1[k]);
    const bool valid = row < rows_a && col < rows_b;
    if constexpr (QUANT) {
      uint32_t codes;
      const uint32_t scale = quantize_row16(v, gs, codes);
      const int64_t r = m0 + row, c = n0 + col;
      if (valid && c % 8 == 0) *(uint32_t*)(p.q + r * (p.cols / 2) + c / 2) = codes;
      if (valid && c % 16 == 0) p.sf[r * (p.cols / 16) + c / 16] = (uint8_t)scale;
    } else if (valid) {
      p.g.d[(m0 + row) * p.ldd + n0 + col] = f32_to_bf16_bits(v);
    }
  }
}

template <class C, bool QUANT>
static void launch_kreg_epilogue(const EpilogueLaunch& p, unsigned grid, hipStream_t stream) {
  // K units of the longest split, and whether they fill every wave's slots
  const int64_t units = (p.g.K / C::kUnit + p.g.splits - 1) / p.g.splits;
  if (units % (C::KS * C::D) == 0)
    hipLaunchKernelGGL((k_gemm_kreg_epilogue<C, QUANT, false>), dim3(grid), dim3(C::kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((k_gemm_kreg_epilogue<C, QUANT, true>), dim3(grid), dim3(C::kThreads), 0, stream, p);
}

// Plan kinds that only the block GEMMs have, numbered past the plain GEMM's.
static constexpr int kReg16x32 = 32, kReg16x32k8 = 33;
static const PlanKind kEpi32 = {"kreg16x32", 16, 32, 256, true, true, false, EpiReg16x32::KS, EpiReg16x32::D};
static const PlanKind kEpi33 = {"kreg16x32k8", 16, 32, 256, true, true, false, EpiReg16x32k8::KS, EpiReg16x32k8::D};

static GemmPlan plan_of(const PlanKind& k, int kind, int64_t M, int64_t cols, int64_t K, int forced_splits, bool gated) {
  GemmPlan pl;
  pl.kind = kind;
  pl.name = k.name;
  pl.tiles_m = (M + k.bm - 1) / k.bm;
  pl.tiles_n = (cols + k.bn - 1) / k.bn;
  pl.group_m = 8;
  if (!k.splitk || pl.tiles_m * pl.tiles_n > kCounterBytes / 4) forced_splits = 1;
  PlanKind both = k;  // a gated tile's partials hold both matrices' sums
  if (gated) both.bn *= 2;
  plan_splits(pl, both, K, forced_splits);
  return pl;
}

// The plain epilogue runs the plain GEMM's plans (the epilogue adds no operand
// traffic to the main loop), except up to M = 16, where 16 x 32 tiles take the
// place of 32 x 32 ones, half of whose A rows would be empty: 8 waves with all
// of up to 16 K units in flight at once while a CU gets one work-group, else 4
// waves (16 x 6144 x 2048: 6.9 us against 8.1; 1 x 6144 x 2048: 6.4 against 7.4;
// 16 x 6144 x 16384: 20.6 against 24.6; 16 x 16384 x 6144: 18.1 against 20.4).
GemmPlan choose_epilogue_plan(int64_t M, int64_t N, int64_t K) {
  int fk = -1, fs = 0;
  const bool forced = forced_plan(kForceGemm, &fk, &fs);
  if (forced && fk == kReg16x32) return plan_of(kEpi32, fk, M, N, K, fs, false);
  if (forced && fk == kReg16x32k8) return plan_of(kEpi33, fk, M, N, K, fs, false);
  GemmPlan pl = choose_plan(M, N, K, kAutoKinds);
  if (M <= 16 && pl.kind == 12 && !(forced && fk == 12)) {
    if ((N + 31) / 32 <= kCUs) return plan_of(kEpi33, kReg16x32k8, M, N, K, 0, false);
    return plan_of(kEpi32, kReg16x32, M, N, K, 0, false);
  }
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
static const PlanKind kGated32 = {"gatedreg16x32", 16, 32, 256, true, true, false, GatedReg16x32::KS, GatedReg16x32::D};

// From sweeps of M = 32..4096, I = 1024..16384, K = 2048 and 6144.  Register
// tiles up to M = 128 while they need at most one work-group per CU; up to M =
// 16 wider matrices take 16 x 32 register tiles (16 x 6144 x 2048 outputs: 8.6 us
// against 11.9 for 32 x 16; 16 x 16384 x 6144: 30.6 against 38).  256-row tiles
// (one work-group per CU) where their last round is at least 85% full in the
// mean (2048 x 4096 x 6144, one full round: 163 us against 191 on 128-row
// tiles; 1024 x 4096, half a round: 133 against 100), 128-row tiles from one
// round of two work-groups per CU on (1024 x 4096 x 6144: 100 us against 108.5 on
// 64-row tiles; half a round: 59 against 57), else split 64-row tiles.
GemmPlan choose_gated_plan(int64_t M, int64_t I, int64_t K) {
  auto tiles = [&](const PlanKind& k) { return ((M + k.bm - 1) / k.bm) * ((I + k.bn - 1) / k.bn); };
  const int64_t t14 = tiles(kGated14), rounds14 = (t14 + kCUs - 1) / kCUs;
  int kind = 9;
  if (M <= 128 && tiles(kGated10) <= kCUs) kind = 10;
  else if (M <= 16 && tiles(kGated32) <= 4 * kCUs) kind = kReg16x32;
  else if (M <= 128 && tiles(kGated12) <= kCUs) kind = 12;
  else if (M > 64 && t14 * 100 >= rounds14 * kCUs * 85) kind = 14;
  else if (M > 64 && tiles(kGated15) >= 2 * kCUs) kind = 15;
  int fk = -1, fs = 0;
  auto has = [](int k) { return k == 9 || k == 10 || k == 12 || k == 14 || k == 15 || k == kReg16x32; };
  if (forced_plan(kForceGemm, &fk, &fs) && has(fk)) kind = fk;
  else fs = 0;
  switch (kind) {
    case 10: return plan_of(kGated10, kind, M, I, K, fs, true);
    case 12: return plan_of(kGated12, kind, M, I, K, fs, true);
    case 14: return plan_of(kGated14, kind, M, I, K, fs, true);
    case 15: return plan_of(kGated15, kind, M, I, K, fs, true);
    case kReg16x32: return plan_of(kGated32, kind, M, I, K, fs, true);
    default: return plan_of(kGated9, kind, M, I, K, fs, true);
  }
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
    case kReg16x32: launch_kreg_epilogue<EpiReg16x32, false>(p, grid, stream); break;
    case kReg16x32k8: launch_kreg_epilogue<EpiReg16x32k8, false>(p, grid, stream); break;
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
    case kReg16x32: launch_kreg_epilogue<GatedReg16x32, QUANT>(p, grid, stream); break;
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
