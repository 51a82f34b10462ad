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
#include <algorithm>

#include "epilogue_tile.h"

namespace nvfp4 {

typedef Cfg<64, 64, 1, 1, 32, 256, 2, 0, 4, 4> EpiTile64k4;
// the same tile with two waves a K-group, each half of the columns, for calls
// whose work-groups have a CU each: two waves per SIMD hide each other's LDS
// reads (333 x 2001 x 1536: 9.0 us against 9.8; 256 x 768 x 6144 in five splits 10.9
// against 11.9); with two work-groups per CU the doubled dequantisation of A
// costs more (1024 x 2048 x 6144: 33.7 against 31.4)
typedef Cfg<64, 64, 1, 2, 32, 256, 2, 0, 4, 4> EpiTile64k4w8;
typedef Cfg<128, 128, 2, 2, 32, 256, 2, 0, 1, 2> EpiTile128;
typedef Cfg<64, 64, 1, 1, 32, 256, 2, 0, 4, 4, 16, 0, 0, 1> GatedTile64k4;  // 32 gate and 32 up columns
typedef Cfg<128, 128, 2, 2, 32, 256, 2, 0, 1, 2, 16, 0, 0, 1> GatedTile128;
// Register tiles of 8 waves with one K unit each in flight: a CU that gets one
// work-group has two waves per SIMD, so one dequantises while the other waits
// for its unit.  4 waves of three units in flight, the plain GEMM's shape, keep
// as many bytes in flight in fewer waves (128 x 2048 x 2048: 8.6 us against 7.6;
// 64 x 2048 x 2048 6.9 against 5.8; 1 x 768 x 2048 4.2 against 3.6; 1 x 16384 x
// 2048 8.9 against 7.5), 8 waves of two or three units were no faster than 4
// (8.5 and 9.8 at the first of these), 16 waves of one between (1 x 768 x 2048
// 4.0).
typedef KCfg<16, 16, 8, 1, 4> EpiReg16x16;
typedef KCfg<16, 32, 8, 1, 4> EpiReg16x32;
typedef KCfg<32, 16, 8, 1, 4> EpiReg32x16;
typedef KCfg<32, 32, 8, 1, 4> EpiReg32x32;
typedef KCfg<16, 32, 8, 1, 4, 0, 1> GatedReg16x16;  // 16 gate and 16 up columns
typedef KCfg<16, 64, 8, 1, 4, 0, 1> GatedReg16x32;
typedef KCfg<16, 16, 8, 1, 4, 0, 2> GatedReg16x8;   // 8 and 8
typedef KCfg<32, 32, 8, 1, 4, 0, 1> GatedReg32x16;

// Register-streamed tile with a fused epilogue (small M).  What the epilogue
// reads besides the sums (alpha, bias, residual) is loaded before the main
// loop, so that after the K-groups' sum (in wave order, and over the splits
// in split order) only arithmetic and one store remain.  A thread owns single
// outputs, 16 consecutive lanes 16 columns of a row: one NVFP4 block.
//
// SKIP leaves the products of K units past the end of a wave's share out
// instead of adding zeros (1 x 6144 x 2304: 5.7 us against 6.1; 128 x 2048 x 2816:
// 8.2 against 9.0; gated 16 x 2048 x 6144, split in two: 8.8 against 9.4); where
// every slot is filled its branches only cut the instruction schedule (1 x 6144
// x 2048: 5.04 against 4.95), so the launcher picks by the shape.
template <class C, bool QUANT, bool SKIP>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_gemm_kreg_epilogue(
    EpilogueLaunch p) {
  __shared__ __attribute__((aligned(16))) float red[C::KS * C::kTileFloats];
  __shared__ int last_flag;
  constexpr bool kGated = C::kGated;
  constexpr int kCols = kGated ? C::BN / 2 : C::BN;  // output columns of the tile
  constexpr int kOut = C::BM * kCols, kPer = (kOut + C::kThreads - 1) / C::kThreads;
  static_assert(!QUANT || kCols % 16 == 0, "whole NVFP4 blocks in a row of lanes");
  // tile columns of output column c
  auto gate_col = [](int c) { return C::kHalves ? c / 8 * 16 + c % 8 : c; };
  auto up_col = [](int c) { return C::kHalves ? c / 8 * 16 + c % 8 + 8 : kCols + c; };
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
    s0[k] = total(row, gate_col(col));
    s1[k] = kGated ? total(row, up_col(col)) : 0.0f;
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

// Plan kinds, numbered like the plain GEMM's kinds of the same tile; bn is the
// output columns of a tile (a gated tile's B has twice as many).
static constexpr int kReg16x32 = 32, kReg16x8 = 33, kTile64w8 = 34;  // tiles that only the block GEMMs have
struct BlockKind {
  int kind;
  PlanKind k;
};
static const BlockKind kEpiKinds[] = {
    {9, {"tile64x64k4", 64, 64, 256, true, false, false, 4}},
    {kTile64w8, {"tile64x64k4w8", 64, 64, 256, true, false, false, 4}},
    {14, {"tile256x256w8k256_mfma32", 256, 256, 256, false, false, false}},
    {15, {"tile128x128k256_mfma32", 128, 128, 256, false, false, false}},
    {16, {"tile256x192w8k256_mfma32", 256, 192, 256, false, false, false}},
    {10, {"kreg16x16k8", 16, 16, 256, true, true, false, EpiReg16x16::KS, EpiReg16x16::D}},
    {11, {"kreg32x16k8", 32, 16, 256, true, true, false, EpiReg32x16::KS, EpiReg32x16::D}},
    {12, {"kreg32x32k8", 32, 32, 256, true, true, false, EpiReg32x32::KS, EpiReg32x32::D}},
    {kReg16x32, {"kreg16x32k8", 16, 32, 256, true, true, false, EpiReg16x32::KS, EpiReg16x32::D}}};
static const BlockKind kGatedKinds[] = {
    {9, {"gated64x32k4", 64, 32, 256, true, false, false, 4}},
    {10, {"gatedreg16x16k8", 16, 16, 256, true, true, false, GatedReg16x16::KS, GatedReg16x16::D}},
    {12, {"gatedreg32x16k8", 32, 16, 256, true, true, false, GatedReg32x16::KS, GatedReg32x16::D}},
    {14, {"gated256x128w8", 256, 128, 256, false, false, false}},
    {15, {"gated128x64", 128, 64, 256, false, false, false}},
    {kReg16x8, {"gatedreg16x8k8", 16, 8, 256, true, true, false, GatedReg16x8::KS, GatedReg16x8::D}},
    {kReg16x32, {"gatedreg16x32k8", 16, 32, 256, true, true, false, GatedReg16x32::KS, GatedReg16x32::D}}};

template <int N>
static const PlanKind* find_kind(const BlockKind (&kinds)[N], int kind) {
  for (const BlockKind& b : kinds)
    if (b.kind == kind) return &b.k;
  return nullptr;
}

static int64_t tiles_of(const PlanKind& k, int64_t M, int64_t cols) {
  return ((M + k.bm - 1) / k.bm) * ((cols + k.bn - 1) / k.bn);
}

// Splits of the 64-row K-group tiles: up to three work-groups per CU and five
// splits (as the plain GEMM), but each with about 5 stages at least, and the
// number that fills the rounds of 256 work-groups best.  An exchange costs about
// 2.5 us, four stages (333 x 2001 x 1536: 9.8 us unsplit, 12.7 in two; 1024 x 768 x
// 2048 10.5 and 12.1; 256 x 768 x 6144 11.9 in five, 13.0 in three).
static int tile_splits(int64_t tiles, int64_t K) {
  const int64_t stages = K / 256;
  int64_t most = std::min<int64_t>({3 * kCUs / tiles, 5, (stages + 1) / 5});
  if (tiles >= 2 * kCUs || most < 1) most = 1;
  int best = 1;
  double best_fill = 0.0;
  for (int s = 1; s <= most; ++s) {
    const int64_t wgs = tiles * s, rounds = (wgs + kCUs - 1) / kCUs;
    const double fill = (double)wgs / (double)(rounds * kCUs);
    if (fill > best_fill || (fill == best_fill && stages >= 6 * s)) {
      best = s;
      best_fill = fill;
    }
  }
  return best;
}

// Splits of the register tiles: the least estimated time, of the K units of a
// wave (proportional to the rows of A and B that a unit has: 1.3 us for 32 of
// them) and the exchange (1.5 us and a little more per split), while every
// work-group has a CU.  Cold, 16 x 256 x 6144 on 16 tiles of 16 x 16: 6.7, 6.3, 5.8,
// 5.8 us in 1 to 4 splits; 1 x 768 x 6144 on 48: 5.3, 5.6, 5.4, 5.6; 16 x 768 x 2304,
// one unit past a whole round: 4.4 unsplit, 5.2 in two; 32 x 32 tiles, 64 x 1024 x
// 6144: 12.6, 10.5, 9.7, 9.5.
static int register_splits(const PlanKind& k, int64_t M, int64_t tiles, int64_t b_rows, int64_t K) {
  const double units = (double)(K / 256) / k.ks;
  const double unit_us = 1.3 / 32 * (double)(std::min<int64_t>(M, k.bm) + b_rows);
  int best = 1;
  double least = units * unit_us;
  for (int s = 2; s <= 8 && tiles * s <= kCUs && s <= K / 256; ++s) {
    const double us = units / s * unit_us + 1.5 + 0.05 * s;
    if (us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

static GemmPlan plan_of(const PlanKind& k, int kind, int64_t M, int64_t cols, int64_t K, int forced_splits, bool gated) {
  GemmPlan pl;
  pl.kind = kind;
  pl.name = k.name;
  pl.tiles_m = (M + k.bm - 1) / k.bm;
  pl.tiles_n = (cols + k.bn - 1) / k.bn;
  pl.group_m = 8;
  PlanKind both = k;  // a gated tile's partials hold both matrices' sums
  if (gated) both.bn *= 2;
  const int64_t tiles = pl.tiles_m * pl.tiles_n;
  if (!k.splitk || tiles > kCounterBytes / 4) forced_splits = 1;
  else if (forced_splits <= 0) forced_splits = k.kreg ? register_splits(k, M, tiles, both.bn, K) : tile_splits(tiles, K);
  plan_splits(pl, both, K, forced_splits);
  return pl;
}

// The smallest register tile (fewest steps per wave) that needs at most one
// work-group per CU, where a long K counts as one work-group per 24 units (so
// that it is split over that many, or gets a larger tile: 64 x 768 x 16384, 14.9
// us on 16 x 16 tiles, 12.9 on 32 x 32; 128 x 768 x 16384 21.6 on 32 x 16, 16.5 on the
// 64-row tiles), per 20 for the largest where the 64-row tiles have full rows
// (256 x 768 x 6144 13.3 us against 11.8); up to M = 16 16 x 16 tiles are split
// less, and 16 x 32 tiles take over to four work-groups per CU (16 x 16384 x 6144:
// 16.6 us; 64-row tiles 21).  -1: none of them; their one wave per 16 or 32
// columns then dequantises A too often.
//
// The count of K holds for the 16 x 8 tiles too, which is not where the two
// cross: cold, gated calls of 2048 columns on 16 x 8 and on 16 x 16 tiles take 7.5
// and 8.6 us at K = 6144 (M = 1; 16 rows 8.2 and 9.3), 7.9 and 9.0 at 6400, 8.2 and
// 9.2 at 7168, 8.7 and 9.1 at 8192 (16 rows 9.5 and 10.2), the same within noise at
// 12288 (11 to 12), 14.5 and 13.3 at 16384, and the rule gives them 16 x 16 tiles
// from 6400 on; 768 and 1024 columns, where it does so above 12288, cross about
// there.
template <int N>
static int register_kind(const BlockKind (&kinds)[N], int64_t M, int64_t cols, int64_t K, bool halves) {
  const int64_t units = K / 256;
  for (int kind : {kReg16x8, 10, 11, 12}) {
    const PlanKind* k = find_kind(kinds, kind);
    if (!k || (kind == kReg16x8 && !halves) || (M <= 16 && k->bm > 16)) continue;
    const int64_t per = kind == 12 && M > 32 ? 20 : 24;
    const int64_t work_groups = M <= 16 && kind == 10 ? 1 : (units + per - 1) / per;
    if (tiles_of(*k, M, cols) * work_groups <= kCUs) return kind;
  }
  if (M <= 16 && tiles_of(*find_kind(kinds, kReg16x32), M, cols) <= 4 * kCUs) return kReg16x32;
  return -1;
}

// The LDS tile of the least estimated time.  Rounds of the unsplit tiles at K =
// 6144, measured: 163 us for 256 work-groups of 256 x 256 (one per CU), 127 for
// 256 of 256 x 192, 97 for 512 of 128 x 128 (two per CU); the 64-row tiles run
// four to a CU, and their last round costs what it holds: 10 us and 48 per 1024.
// The ratios are those of other K too (4096 x 4096 x 6144: 169, 236, 199, 200 us, x
// 1024: 43, 58, 45, 50; 1024 x 8192 x 6144: 142, 115, 103, 106; 2048 x 6144 x 2048:
// 63, 53, 61, 64).  Gated tiles do the same
// work (their columns are half of it).
template <int N>
static int tile_kind(const BlockKind (&kinds)[N], int64_t M, int64_t cols) {
  struct Round {
    int kind, work_groups;
    double us;
  };
  int best = 9;
  double least = 10.0 + 48.0 / 1024 * (double)tiles_of(*find_kind(kinds, 9), M, cols);
  for (const Round& r : {Round{14, kCUs, 163.0}, Round{16, kCUs, 127.0}, Round{15, 2 * kCUs, 97.0}}) {
    const PlanKind* k = find_kind(kinds, r.kind);
    if (!k) continue;
    const double us = r.us * (double)((tiles_of(*k, M, cols) + r.work_groups - 1) / r.work_groups);
    if (us < least) {
      best = r.kind;
      least = us;
    }
  }
  return best;
}

template <int N>
static GemmPlan choose_block_plan(const BlockKind (&kinds)[N], int64_t M, int64_t cols, int64_t K, bool gated, bool halves) {
  int fk = -1, fs = 0;
  if (!forced_plan(kForceGemm, &fk, &fs)) fk = -1;
  const bool forced = find_kind(kinds, fk) && (fk != kReg16x8 || halves);
  int kind = forced ? fk : register_kind(kinds, M, cols, K, halves);
  if (kind < 0) kind = tile_kind(kinds, M, cols);
  return plan_of(*find_kind(kinds, kind), kind, M, cols, K, forced ? fs : 0, gated);
}

GemmPlan choose_epilogue_plan(int64_t M, int64_t N, int64_t K) {
  GemmPlan pl = choose_block_plan(kEpiKinds, M, N, K, false, false);
  int fk = -1, fs = 0;
  if (pl.kind == 9 && !(forced_plan(kForceGemm, &fk, &fs) && fk == 9) && pl.tiles_m * pl.tiles_n * pl.splits <= kCUs) {
    pl.kind = kTile64w8;
    pl.name = find_kind(kEpiKinds, kTile64w8)->name;
  }
  return pl;
}

// 16 x 8 tiles, 8 gate and 8 up rows in one block of columns, have enough
// work-groups to leave K whole (one token, 2048 x 6144: 6.7 us against 8.2 on 16 x
// 16 tiles in two splits); an NVFP4 block has 16 columns, so they are for bf16.
GemmPlan choose_gated_plan(int64_t M, int64_t I, int64_t K, bool quantize) {
  const bool halves = !quantize && I * (K / 16) < (int64_t(1) << 30);
  return choose_block_plan(kGatedKinds, M, I, K, true, halves);
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
    case 14:
    case 16: launch_epilogue_large(pl.kind, p, grid, stream); break;
    case 15: launch_epilogue_tile<EpiTile128, false>(p, grid, stream); break;
    case kTile64w8: launch_epilogue_tile<EpiTile64k4w8, false>(p, grid, stream); break;
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
    case kReg16x8:
      if constexpr (!QUANT) launch_kreg_epilogue<GatedReg16x8, false>(p, grid, stream);
      break;
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
