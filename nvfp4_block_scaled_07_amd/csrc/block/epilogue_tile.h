// LDS-staged tile GEMM with a fused epilogue: the main loop, K-group sum and
// split-K exchange of gemm_tile.h around the epilogues of epilogue.h.
//
// Included by gemm_epilogue.hip and gemm_epilogue_large.hip; each kernel
// instantiation lives in exactly one of them.
#pragma once

#include "epilogue.h"

namespace nvfp4 {

// How a tile's sums pass through LDS.
//  * Direct (plain epilogue, KS == 1): not at all.
//  * Waves (gated, KS == 1): each wave sends the TN blocks of one of its row
//    blocks at a time through slices of its own, with no barrier between
//    waves.  Row stride 40 floats: a store of the MFMA layout (lanes 0-31 one
//    row, lanes 32-63 the row 4 below) covers all 64 banks once, and rows stay
//    16-byte aligned.
//  * Tile (K-groups, split K): the whole tile, stride BN + 4, then every
//    thread of the work-group takes part of it.
template <class C>
struct Staging {
  static constexpr bool kByWave = C::KS == 1;
  static constexpr bool kDirect = kByWave && !C::kGated;
  static constexpr int kSliceLd = 40;
  static constexpr int kSlice = 32 * kSliceLd;
  static constexpr int kTileLd = C::BN + 4;
  static constexpr int kFloats = kDirect ? 1 : kByWave ? C::kWaves * C::TN * kSlice : C::BM * kTileLd;
};

template <class C>
union SharedEpilogue {
  Smem<C> pipe;
  float red[GroupRed<C>::kFloats];
  float stage[Staging<C>::kFloats];
};

// acc block -> its 32 x 32 place at dst (row stride LD)
template <class C, int LD>
__device__ __forceinline__ void stage_block(float* dst, const typename C::Acc& a) {
  const int lane = threadIdx.x & 63, n_in = lane % C::MF, g = lane / C::MF;
#pragma unroll
  for (int j = 0; j < Mfma<C::MF>::kAcc; ++j) dst[Mfma<C::MF>::row(j, g) * LD + n_in] = a[j];
}

// LDS written by other lanes of this wave: the hardware keeps a wave's LDS
// accesses in order, the fence keeps the compiler's.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Plain epilogue on the accumulators themselves: lane l of a 32 x 32 block
// holds column l % 32 of rows 8 q + 4 (l / 32) + 0..3.  A block's 16 residual
// loads are issued one block ahead.  Against a pass through LDS with 16-byte
// accesses this is 2% faster (8192 x 6144 x 6144: 470 us against 480, with
// residual 490 against 501): no wait between a block's sums and its stores.
// FULL: the whole tile is inside the output.
template <class C, bool FULL>
__device__ __forceinline__ void finish_direct(const EpilogueLaunch& p, const typename C::Acc (&acc)[C::TM][C::TN],
                                              float a0, int64_t m0, int64_t n0, int rows_valid, int cols_valid) {
  constexpr int kAcc = Mfma<C::MF>::kAcc;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int row0 = wave / C::WN * C::kWM + 4 * (lane / 32), col0 = wave % C::WN * C::kWN + lane % 32;
  uint16_t* out = p.g.d + (m0 + row0) * p.ldd + n0 + col0;
  const uint16_t* res = p.res ? p.res + (m0 + row0) * p.ldr + n0 + col0 : nullptr;
  auto inside = [&](int row, int col) { return FULL || (row0 + row < rows_valid && col0 + col < cols_valid); };
  uint32_t next[kAcc];
  auto load = [&](auto block) {
    constexpr int tm = decltype(block)::value / C::TN, tn = decltype(block)::value % C::TN;
#pragma unroll
    for (int j = 0; j < kAcc; ++j) {
      const int row = tm * 32 + Mfma<C::MF>::row(j, 0);
      next[j] = inside(row, tn * 32) ? res[row * p.ldr + tn * 32] : 0u;
    }
  };
  if (res) load(std::integral_constant<int, 0>{});
  static_for<C::TM * C::TN>([&](auto block) {
    constexpr int tm = decltype(block)::value / C::TN, tn = decltype(block)::value % C::TN;
    uint32_t cur[kAcc];
#pragma unroll
    for (int j = 0; j < kAcc; ++j) cur[j] = next[j];
    if constexpr (tm * C::TN + tn + 1 < C::TM * C::TN) {
      if (res) load(std::integral_constant<int, tm * C::TN + tn + 1>{});
    }
    float v[kAcc];
#pragma unroll
    for (int j = 0; j < kAcc; ++j) v[j] = a0 * acc[tm][tn][j];
    if (p.bias) {
      const float b =
          FULL || col0 + tn * 32 < cols_valid ? __uint_as_float((uint32_t)p.bias[n0 + col0 + tn * 32] << 16) : 0.0f;
#pragma unroll
      for (int j = 0; j < kAcc; ++j) v[j] += b;
    }
    activate<kAcc>(v, p.act);
#pragma unroll
    for (int j = 0; j < kAcc; ++j) {
      const int row = tm * 32 + Mfma<C::MF>::row(j, 0);
      if (res) v[j] += p.beta * __uint_as_float(cur[j] << 16);
      if (inside(row, tn * 32)) out[row * p.ldd + tn * 32] = f32_to_bf16_bits(v[j]);
    }
    // block by block: mixing them would only lengthen the live ranges
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Each gated wave's blocks through its own slices (every wave is past its
// last read of the stage buffers).
template <class C, bool QUANT>
__device__ __forceinline__ void finish_by_wave(const EpilogueLaunch& p, float* stage,
                                               const typename C::Acc (&acc)[C::TM][C::TN], float a0, float a1,
                                               int64_t m0, int64_t n0, int rows_valid, int cols_valid) {
  typedef Staging<C> St;
  constexpr int W = kChunk<QUANT>, kPerRow = 32 / W, kRows = 64 / kPerRow;
  constexpr int kBlk = C::TN / 2, kPasses = 32 / kRows;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / C::WN, wn = wave % C::WN;
  float* slice = stage + wave * C::TN * St::kSlice;
  const int r_in = lane / kPerRow, c_in = lane % kPerRow * W;
  const float* src = slice + r_in * St::kSliceLd + c_in;
  static_for<C::TM>([&](auto tmc) {
    constexpr int tm = decltype(tmc)::value;
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) stage_block<C, St::kSliceLd>(slice + tn * St::kSlice, acc[tm][tn]);
    wave_sync();
    // a rolled loop: TM unrolled copies of a chunk's code are already long
#pragma unroll 1
    for (int c = 0; c < kBlk * kPasses; ++c) {
      const int row = wm * C::kWM + tm * 32 + c % kPasses * kRows + r_in;
      const int col = wn * C::kBWave + c / kPasses * 32 + c_in;
      const float* at = src + c / kPasses * St::kSlice + c % kPasses * kRows * St::kSliceLd;
      float s[W], u[W];
      lds_chunk<W>(s, at);
      lds_chunk<W>(u, at + kBlk * St::kSlice);
      if (row < rows_valid && col < cols_valid) finish<true, QUANT>(p, a0, a1, m0 + row, n0 + col, s, u, u4_t{});
    }
    wave_sync();
  });
}

// Split-K sums (S partial tiles in split order) into the tile in LDS.
template <class C, int S>
__device__ __forceinline__ void gather_partials_s(const rsrc_t& r, float* tile) {
  typedef PartLayout<C> P;
  constexpr int kLoads = C::OCC >= 4 ? 8 : 16;
  constexpr int PB = S >= kLoads ? 1 : kLoads / S;  // positions per batch
  for (int f0 = threadIdx.x; f0 < P::kQ; f0 += C::kThreads * PB) {
    f4_t v[PB][S];
#pragma unroll
    for (int b = 0; b < PB; ++b) {
      const int f = f0 + b * C::kThreads;
      if (f < P::kQ) {
#pragma unroll
        for (int z = 0; z < S; ++z) v[b][z] = load_coherent4(r, (uint32_t)(z * P::kQ + f) * 16);
      }
    }
#pragma unroll
    for (int b = 0; b < PB; ++b) {
      const int f = f0 + b * C::kThreads;
      if (f >= P::kQ) continue;
      f4_t sum = v[b][0];
#pragma unroll
      for (int z = 1; z < S; ++z) sum += v[b][z];
      const int lane = f & 63, i = (f >> 6) % P::kChunks, gw = (f >> 6) / P::kChunks;
      const int q = i % P::kAccQ, tn = (i / P::kAccQ) % C::TN, tm = (i / P::kAccQ) / C::TN;
      const int col = gw % C::WN * C::kWN + tn * C::MF + lane % C::MF;
      const int row = gw / C::WN * C::kWM + tm * C::MF;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        tile[(row + Mfma<C::MF>::row(4 * q + e, lane / C::MF)) * Staging<C>::kTileLd + col] = sum[e];
    }
  }
}

template <class C>
__device__ __forceinline__ void gather_partials(const rsrc_t& r, int S, float* tile) {
  switch (S) {
#define NVFP4_GATHER(n) \
  case n: gather_partials_s<C, n>(r, tile); break;
    NVFP4_GATHER(2) NVFP4_GATHER(3) NVFP4_GATHER(4) NVFP4_GATHER(5) NVFP4_GATHER(6) NVFP4_GATHER(7) NVFP4_GATHER(8)
    NVFP4_GATHER(9) NVFP4_GATHER(10) NVFP4_GATHER(11) NVFP4_GATHER(12) NVFP4_GATHER(13) NVFP4_GATHER(14)
    NVFP4_GATHER(15) NVFP4_GATHER(16)
#undef NVFP4_GATHER
    default: break;
  }
}

template <class C, bool QUANT>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_gemm_epilogue(
    EpilogueLaunch p) {
  typedef Staging<C> St;
  static_assert(C::MF == 32, "32 x 32 blocks");
  static_assert(St::kByWave || !C::kGated || C::kGroupWaves == 1, "gated K-group tiles hold one wave's columns in order");
  __shared__ __attribute__((aligned(16))) SharedEpilogue<C> shm;
  __shared__ int last_flag;
  const TileAt at = tile_at(p.g);
  const int S = p.g.splits;
  constexpr int kCols = C::kBRows;  // output columns of the tile
  const int64_t m0 = (int64_t)at.tm * C::BM, n0 = (int64_t)at.tn * kCols;
  const int64_t ld = p.g.K / 2, lds = p.g.K / 16;
  Operand A{p.g.a + m0 * ld, p.g.a_sf + m0 * lds, ld, lds, (int)min<int64_t>(C::BM, p.g.M - m0)};
  Operand B{p.g.b + n0 * ld, p.g.b_sf + n0 * lds, ld, lds, (int)min<int64_t>(kCols, p.cols - n0)};
  if constexpr (C::kGated) {
    B.data2 = B.data + p.cols * ld;
    B.sf2 = B.sf + p.cols * lds;
  }
  const int nk = (int)(p.g.K / C::BK);
  const int kt0 = (int)((int64_t)at.z * nk / S), kt1 = (int)((int64_t)(at.z + 1) * nk / S);
  typename C::Acc acc[C::TM][C::TN];
  if constexpr (St::kDirect) {
    // one load of every 128-byte line of the tile's residual under the last
    // stage's MFMAs: the epilogue's 2-byte loads then find it in L2 (8192 x
    // 6144 x 6144 with residual: 488 us against 496 on one box)
    constexpr int kLines = C::BM * C::BN / 64, kPer = (kLines + C::kThreads - 1) / C::kThreads;
    uint32_t line[kPer] = {};
    mainloop<C>(shm.pipe, A, B, kt0, kt1, C::TM, acc, [&](int left) {
      if (left != 1 || !p.res) return;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int l = threadIdx.x + i * C::kThreads, row = l / (C::BN / 64), col = l % (C::BN / 64) * 64;
        if (row < A.rows && col < B.rows) line[i] = p.res[(m0 + row) * p.ldr + n0 + col];
      }
    });
#pragma unroll
    for (int i = 0; i < kPer; ++i) asm volatile("" ::"v"(line[i]));  // the loads are not dead
  } else {
    mainloop<C>(shm.pipe, A, B, kt0, kt1, C::TM, acc);
  }
  const float a0 = p.g.alpha ? p.g.alpha[0] : 1.0f;
  const float a1 = C::kGated && p.g.alpha ? p.g.alpha[1] : 1.0f;
  if constexpr (St::kDirect) {
    if (A.rows >= C::BM && B.rows >= C::BN) finish_direct<C, true>(p, acc, a0, m0, n0, A.rows, B.rows);
    else finish_direct<C, false>(p, acc, a0, m0, n0, A.rows, B.rows);
  } else if constexpr (St::kByWave) {
    __syncthreads();  // every wave is past its last read of the stage buffers
    finish_by_wave<C, QUANT>(p, shm.stage, acc, a0, a1, m0, n0, A.rows, B.rows);
  } else {
    reduce_groups<C>(shm.red, acc);
    const bool lead = wave_id() < C::kGroupWaves;  // K-group 0 holds the sum
    if (S == 1) {
      if (lead) {
        float* dst = shm.stage + wave_id() / C::WN * C::kWM * St::kTileLd + wave_id() % C::WN * C::kWN;
#pragma unroll
        for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
          for (int tn = 0; tn < C::TN; ++tn)
            stage_block<C, St::kTileLd>(dst + tm * 32 * St::kTileLd + tn * 32, acc[tm][tn]);
      }
    } else {
      // publish this split's partial, count arrivals, the last one reduces
      constexpr int kTileFloats = C::BM * C::BN;
      int* counter = (int*)p.g.ws + at.tile;
      const rsrc_t part = partial_rsrc(p.g.ws + kCounterBytes / 4 + (int64_t)at.tile * S * kTileFloats, S, kTileFloats);
      if (lead) store_partial<C>(acc, part, at.z);
      __builtin_amdgcn_s_waitcnt(0);  // this wave's partial stores are complete
      __syncthreads();
      if (threadIdx.x == 0) last_flag = count_arrival(counter, S);
      __syncthreads();
      if (!last_flag) return;
      gather_partials<C>(part, S, shm.stage);
      if (threadIdx.x == 0) reset_counter(counter);
    }
    __syncthreads();
    finish_tile<C::kGated, QUANT, C::BM, kCols, St::kTileLd, kCols, C::kThreads>(p, shm.stage, a0, a1, m0, n0, A.rows,
                                                                                 B.rows);
  }
}

template <class C, bool QUANT>
inline void launch_epilogue_tile(const EpilogueLaunch& p, unsigned grid, hipStream_t stream) {
  hipLaunchKernelGGL((k_gemm_epilogue<C, QUANT>), dim3(grid), dim3(C::kThreads), 0, stream, p);
}

}  // namespace nvfp4
