// LDS-staged tile GEMM with a fused epilogue: the main loop, K-group sum and
// split-K exchange of gemm_tile.h around the epilogues of epilogue.h.
//
// Included by gemm_epilogue.hip and gemm_epilogue_large.hip; each kernel
// instantiation lives in exactly one of them.
#pragma once

#include "epilogue.h"

namespace nvfp4 {

// How a tile's sums pass through LDS.
//  * Waves (KS == 1): each wave sends its own 32 x 32 blocks through a slice
//    of its own, one at a time (a gated wave a gate block and its up block),
//    with no barrier between waves.  Row stride 40 floats: a store of the
//    MFMA layout (lanes 0-31 one row, lanes 32-63 the row 4 below) covers all
//    64 banks once, and rows stay 16-byte aligned.
//  * Tile (K-groups, split K): the whole tile, stride BN + 4, then every
//    thread of the work-group takes chunks of it.
template <class C>
struct Staging {
  static constexpr int kSliceLd = 40;
  static constexpr int kSlice = 32 * kSliceLd;
  static constexpr int kSlices = C::kGated ? 2 : 1;
  static constexpr bool kByWave = C::KS == 1;
  static constexpr int kTileLd = C::BN + 4;
  static constexpr int kFloats = kByWave ? C::kWaves * kSlices * kSlice : C::BM * kTileLd;
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

// Each wave's blocks through its own slice (every wave is past its last read
// of the stage buffers).
template <class C, bool QUANT>
__device__ __forceinline__ void finish_by_wave(const EpilogueLaunch& p, float* stage,
                                               const typename C::Acc (&acc)[C::TM][C::TN], float a0, float a1,
                                               int64_t m0, int64_t n0, int rows_valid, int cols_valid) {
  typedef Staging<C> St;
  constexpr int W = kChunk<QUANT>, kPerRow = 32 / W, kRows = 64 / kPerRow;
  constexpr int kBlk = C::kGated ? C::TN / 2 : C::TN;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / C::WN, wn = wave % C::WN;
  float* slice = stage + wave * St::kSlices * St::kSlice;
  const int r_in = lane / kPerRow, c_in = lane % kPerRow * W;
  const float* src = slice + r_in * St::kSliceLd + c_in;
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < kBlk; ++tn) {
      stage_block<C, St::kSliceLd>(slice, acc[tm][tn]);
      if constexpr (C::kGated) stage_block<C, St::kSliceLd>(slice + St::kSlice, acc[tm][tn + kBlk]);
      wave_sync();
      const int col = wn * C::kBWave + tn * 32 + c_in;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += kRows) {
        const int row = wm * C::kWM + tm * 32 + r0 + r_in;
        float s[W], u[W];
        lds_chunk<W>(s, src + r0 * St::kSliceLd);
        if constexpr (C::kGated) lds_chunk<W>(u, src + St::kSlice + r0 * St::kSliceLd);
        if (row < rows_valid && col < cols_valid) finish<C::kGated, QUANT>(p, a0, a1, m0 + row, n0 + col, s, u);
      }
      wave_sync();
    }
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
  static_assert(St::kByWave || C::kGroupWaves == 1, "K-group tiles hold one wave's columns in order");
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
  mainloop<C>(shm.pipe, A, B, kt0, kt1, C::TM, acc);
  const float a0 = p.g.alpha ? p.g.alpha[0] : 1.0f;
  const float a1 = C::kGated && p.g.alpha ? p.g.alpha[1] : 1.0f;
  if constexpr (St::kByWave) {
    __syncthreads();  // every wave is past its last read of the stage buffers
    finish_by_wave<C, QUANT>(p, shm.stage, acc, a0, a1, m0, n0, A.rows, B.rows);
  } else {
    reduce_groups<C>(shm.red, acc);
    const bool lead = wave_id() < C::kGroupWaves;  // K-group 0 holds the sum
    if (S == 1) {
      if (lead) {
#pragma unroll
        for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
          for (int tn = 0; tn < C::TN; ++tn)
            stage_block<C, St::kTileLd>(shm.stage + tm * 32 * St::kTileLd + tn * 32, acc[tm][tn]);
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
