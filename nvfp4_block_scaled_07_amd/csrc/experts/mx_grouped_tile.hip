// Grouped products of MXFP4 operands where experts have many rows: 256 rows x
// 256 weight rows a work-group, 8 waves of 128 x 64, both operands staged in
// LDS.  65536 rows on 32 experts of 2 x 2048 x 6144: 1012 to 1046 us over boxes,
// 3.2 PFLOP/s (the plain MX GEMM of 8192^3: 3.3 to 3.5).  Bound, like that GEMM,
// by a stage's loads into LDS, its LDS reads and its MFMAs, which overlap only in
// part (MFMA 35% busy), and with a short K by the stores of the outputs as well,
// which all work-groups issue at the same time (32768 rows of 6144 x 2048 on 64
// experts: 386 us, 325 without them).  A stage's scales in 6 reads of 8 bytes
// instead of 24 of a byte: the same gated, 2% slower plain.  See mx_grouped.hip for
// the formulas and for the kernel that serves few rows.
//
// A's rows are gathered on the way into LDS: the lanes of a load instruction
// that belong to one row add that row's own offset.  The weights are the MFMA's
// first operand, so a lane holds one row of the output and, of each 32 columns,
// 16: runs of 4, alternating with lane + 32.  One lane swap leaves 8 consecutive
// columns each, and an MXFP4 block in a pair of lanes.
//
// A gated tile holds 128 gate rows, then the same 128 up rows, and every wave 32
// of both.  The last tile of an expert is seldom full: a wave none of whose
// rows exist leaves out its products, and waves w and w + 4, which share a
// SIMD, have different rows, so that half a tile takes about half the time.
#include "../block/epilogue.h"
#include "expert_tile.h"
#include "mx_block.h"

namespace nvfp4 {

// The plain MX GEMM's 8-wave 256 x 256 tile; gated, its LDS rows of B are 128
// gate rows, then the same 128 up rows, and a wave's two column blocks are the
// same columns of each.
template <bool GATED>
struct CfgExperts : Cfg<256, 256, 2, 4, 32, 256, 2, 0, 1, 2, 32, 4> {
  static constexpr bool kGated = GATED;
  static constexpr int kBRows = GATED ? 128 : 256;        // tile rows of one matrix
  static constexpr int kBWave = GATED ? kWN / 2 : kWN;    // and of one wave in it
  static constexpr int b_row(int tn) { return GATED ? tn * kBRows : tn * MF; }
  static_assert(TN == 2, "gated: one column block of each matrix a wave");
  static_assert(BM == BN, "both operands' stage buffers are as far apart");
};

// LDS reads of sub-step SS of stage buffer BUF.
template <class C, int BUF, int SS>
__device__ __forceinline__ void tile_read(MxFrags<C>& f, const ReadAddr<C>& ra) {
  constexpr int kScale = SS * C::KG;  // one scale byte per chunk
  static_for<C::TM>([&](auto tmc) {
    constexpr int tm = decltype(tmc)::value;
    ds_read128_at<BUF * C::BM * C::RB + tm * 32 * C::RB>(f.ac[tm], ra.a[SS]);
    ds_read_u8_at<BUF * C::BM * C::SB + tm * 32 * C::SB + kScale>(f.asw[tm], ra.as);
  });
  static_for<C::TN>([&](auto tnc) {
    constexpr int tn = decltype(tnc)::value;
    ds_read128_at<BUF * C::BN * C::RB + C::b_row(tn) * C::RB>(f.bc[tn], ra.b[SS]);
    ds_read_u8_at<BUF * C::BN * C::SB + C::b_row(tn) * C::SB + kScale>(f.bsw[tn], ra.bs);
  });
}

// One stage: the next sub-step's reads are issued before this one's MFMAs.
template <class C, int BUF>
__device__ __forceinline__ void tile_stage(const ReadAddr<C>& ra, typename C::Acc (&acc)[C::TM][C::TN]) {
  typedef int v8i_t __attribute__((ext_vector_type(8)));
  MxFrags<C> f[2];
  tile_read<C, BUF, 0>(f[0], ra);
  static_for<C::kSub>([&](auto ssc) {
    constexpr int ss = decltype(ssc)::value;
    MxFrags<C>& cur = f[ss & 1];
    lgkm_wait();  // slot ss & 1 has landed (nothing else is in flight)
    v8i_t av[C::TM], bv[C::TN];
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm) {
      pin(cur.ac[tm]);
      pin(cur.asw[tm]);
      av[tm] = v8i_t{(int)cur.ac[tm][0], (int)cur.ac[tm][1], (int)cur.ac[tm][2], (int)cur.ac[tm][3], 0, 0, 0, 0};
    }
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) {
      pin(cur.bc[tn]);
      pin(cur.bsw[tn]);
      bv[tn] = v8i_t{(int)cur.bc[tn][0], (int)cur.bc[tn][1], (int)cur.bc[tn][2], (int)cur.bc[tn][3], 0, 0, 0, 0};
    }
    if constexpr (ss + 1 < C::kSub) tile_read<C, BUF, ss + 1>(f[(ss + 1) & 1], ra);
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn)
        acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bv[tn], av[tm], acc[tm][tn], 4, 4, 0,
                                                                       (int)cur.bsw[tn], 0, (int)cur.asw[tm]);
  });
  // computed here: not moved down to where the tile ends (no instruction reads it)
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) asm volatile("" : "+v"(acc[tm][tn]));
}

// Row offsets of this lane's pieces of A, in the order of issue_a.
template <class C>
struct GatherA {
  typedef DmaShape<C::BM, C::RB, 16> Codes;
  typedef DmaShape<C::BM, C::SB, 4> Scales;
  static constexpr int kCodes = Codes::kInst / C::kDmaWaves, kScales = Scales::kInst / C::kDmaWaves;
  static_assert(kCodes * C::kDmaWaves == Codes::kInst && kScales * C::kDmaWaves == Scales::kInst, "whole shares");
  uint32_t code[kCodes], scale[kScales];
};

// A 64-bit base whose halves are known to be the same in all lanes.
__device__ __forceinline__ rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return make_rsrc((const void*)(uintptr_t)(((uint64_t)hi << 32) | lo), __builtin_amdgcn_readfirstlane(bytes));
}

template <class C>
__device__ __forceinline__ void issue_tile(Smem<C>& sm, int buf, const GatherA<C>& ga, const rsrc_t& ra,
                                           const rsrc_t& ras, const Operand& B, int kt, int wave, int lane) {
  typedef GatherA<C> G;
  constexpr int W = C::kDmaWaves;
  if (wave >= W) return;
#pragma unroll
  for (int i = 0; i < G::kCodes; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(sm.a[buf] + (wave + i * W) * 1024), 16, ga.code[i],
                                             kt * C::RB, 0, 0);
#pragma unroll
  for (int i = 0; i < G::kScales; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ras, (lds_ptr_t)(sm.asf[buf] + (wave + i * W) * 256), 4, ga.scale[i],
                                             kt * C::SB, 0, 0);
  if constexpr (C::kGated) {
    constexpr int R = C::kBRows;
    dma_tile<R, C::RB, 16, C::MF, W, 0, true>(sm.b[buf], B.data, B.ld, B.rows, kt * C::RB, wave, lane);
    dma_tile<R, C::RB, 16, C::MF, W, 0, true>(sm.b[buf] + R * C::RB, B.data2, B.ld, B.rows, kt * C::RB, wave, lane);
    dma_tile<R, C::SB, 4, 0, W, 0, true>(sm.bsf[buf], B.sf, B.lds, B.rows, kt * C::SB, wave, lane);
    dma_tile<R, C::SB, 4, 0, W, 0, true>(sm.bsf[buf] + R * C::SB, B.sf2, B.lds, B.rows, kt * C::SB, wave, lane);
  } else {
    dma_tile<C::BN, C::RB, 16, C::MF, W, 0, true>(sm.b[buf], B.data, B.ld, B.rows, kt * C::RB, wave, lane);
    dma_tile<C::BN, C::SB, 4, 0, W, 0, true>(sm.bsf[buf], B.sf, B.lds, B.rows, kt * C::SB, wave, lane);
  }
}

// 16 columns of a row that this lane and lane ^ 32 hold in runs of 4 (v[0..3],
// v[4..7] here) -> this lane's 8 consecutive ones, as bf16.
__device__ __forceinline__ u4_t eight_columns(const float (&v)[8]) {
  uint32_t a[2] = {f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3])};
  uint32_t b[2] = {f32x2_to_bf16x2_bits(v[4], v[5]), f32x2_to_bf16x2_bits(v[6], v[7])};
  u4_t w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u2_t s = __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(a[i], b[i], false, false));
    w[i] = s[0];
    w[2 + i] = s[1];
  }
  return w;
}

// A tile's expert, rows and columns.
struct TileAtExpert {
  int e, rows_c, cols_c;  // expert (-1: no such tile), valid rows, valid columns
  int64_t mc, n0;         // first row, first column
};

// One tile, and where its operands are.
template <class C>
struct TileJob : TileAtExpert {
  Operand B;
  rsrc_t ra, ras;
  GatherA<C> ga;
};

// Logical tile L: the column tiles of a row tile are apart by the expert's row
// tiles, so that neighbours share the weights' tile.  limit: tiles that offsets
// which do not decrease may have.
template <class C>
__device__ __forceinline__ TileJob<C> tile_job(const MxGroupedLaunch& p, int L, int tiles_n, int limit) {
  typedef GatherA<C> G;
  TileJob<C> t;
  t.e = -1;
  if (L >= limit) return t;
  const ExpertTile at = find_tile<C::BM>(p, L / tiles_n);
  t.e = at.expert;
  if (t.e < 0) return t;
  const int64_t cols = C::kGated ? p.N / 2 : p.N, ld = p.K / 2, lds = p.K / 32;
  const int in = L - at.first * tiles_n, lane = threadIdx.x & 63, wave = wave_id();
  t.n0 = (int64_t)(in / at.tiles) * C::kBRows;
  t.mc = at.lo + (int64_t)(in % at.tiles) * C::BM;
  t.rows_c = (int)min<int64_t>(C::BM, at.hi - t.mc);
  t.cols_c = (int)min<int64_t>(C::kBRows, cols - t.n0);
  const int64_t row0 = (int64_t)t.e * p.N + t.n0, second = C::kGated ? p.N / 2 : 0;
  t.B = Operand{p.b + row0 * ld, p.b_sf + row0 * lds, ld, lds, t.cols_c, p.b + (row0 + second) * ld, p.b_sf + (row0 + second) * lds};
  const bool gather = p.row_token != nullptr;
  // never empty, so that no stage's scalar offset lies past the end (without
  // tokens every row's vector offset does)
  const int64_t most = gather ? max(p.T, (int64_t)1) : t.rows_c, skip = gather ? 0 : t.mc;
  t.ra = uniform_rsrc(p.a + skip * ld, (uint32_t)(most * ld));
  t.ras = uniform_rsrc(p.a_sf + skip * lds, (uint32_t)(most * lds));
  const auto source = [&](int r) -> int64_t {  // row r's row of a, or -1
    if (r >= t.rows_c) return -1;
    if (!gather) return r;
    const int64_t k = p.row_token[t.mc + r];
    return k >= 0 && k < p.T ? k : -1;
  };
#pragma unroll
  for (int i = 0; i < G::kCodes; ++i) {
    const int r = (wave % C::kDmaWaves + i * C::kDmaWaves) * G::Codes::kRowsPerInst + lane / C::CH;
    const int64_t k = source(r);
    t.ga.code[i] = k < 0 ? 0x80000000u : (uint32_t)(k * ld + (((lane % C::CH) ^ swz<C::CH, C::MF>(r)) << 4));
  }
#pragma unroll
  for (int i = 0; i < G::kScales; ++i) {
    const int r = (wave % C::kDmaWaves + i * C::kDmaWaves) * G::Scales::kRowsPerInst + lane / (C::SB / 4);
    const int64_t k = source(r);
    t.ga.scale[i] = k < 0 ? 0x80000000u : (uint32_t)(k * lds + (lane % (C::SB / 4)) * 4);
  }
  return t;
}

// Bytes of an output row in LDS: 64 columns and 16 more (other banks).
constexpr int kOutRow = 64 * 2 + 16;

template <class C>
__device__ __forceinline__ void finish_tile(const MxGroupedLaunch& p, const TileAtExpert& t,
                                            const typename C::Acc (&acc)[C::TM][C::TN], uint8_t* out) {
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN, wn = wave % C::WN;
  const int e = t.e, rows_c = t.rows_c;
  const int64_t mc = t.mc, n0 = t.n0;
  // lane: row lane % 32 of each row block; accumulator j is column
  // Mfma<32>::row(j, lane / 32) of each column block
  const int g = lane >> 5;
  if constexpr (C::kGated) {
    const float a0 = p.alpha ? p.alpha[2 * e] : 1.0f, a1 = p.alpha ? p.alpha[2 * e + 1] : 1.0f;
    const int64_t I = p.N / 2, col = n0 + 32 * wn;
    if (col >= I) return;  // blocks of 32 are whole
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm) {
      float h[16], u[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        h[j] = a0 * acc[tm][0][j];
        u[j] = a1 * acc[tm][1][j];
      }
      if (p.bias) {
        const uint16_t* bias = p.bias + (int64_t)e * p.N + col;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int c = Mfma<32>::row(j, g);
          h[j] += __uint_as_float((uint32_t)bias[c] << 16);
          u[j] += __uint_as_float((uint32_t)bias[I + c] << 16);
        }
      }
      activate<16>(h, p.act);
      uint32_t peak = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        h[j] *= u[j];
        peak = umax(peak, magnitude(h[j]));
      }
      const u2_t both = __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(peak, peak, false, false));
      const MxScale s = mx_scale(umax(both[0], both[1]), p.rule);
      uint32_t w[2];  // runs 0, 1 and 2, 3 of this lane, 16 bits each
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h[8 * c] * s.r, h[8 * c + 1] * s.r, 1.0f, 0);
        w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], h[8 * c + 2] * s.r, h[8 * c + 3] * s.r, 1.0f, 1);
        w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], h[8 * c + 4] * s.r, h[8 * c + 5] * s.r, 1.0f, 2);
        w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], h[8 * c + 6] * s.r, h[8 * c + 7] * s.r, 1.0f, 3);
        w[c] &= s.keep;
      }
      // lanes below 32: runs 0, 1 of both; the others runs 2, 3
      const u2_t x = __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false));
      const u2_t codes = {(x[0] & 0xFFFFu) | x[1] << 16, x[0] >> 16 | (x[1] & 0xFFFF0000u)};
      const int row = wm * C::kWM + tm * 32 + (lane & 31);
      if (row < rows_c) {
        const int64_t r = mc + row;
        *(u2_any_t*)(p.q + r * (I / 2) + col / 2 + 8 * g) = codes;
        if (g == 0) p.sf[r * (I / 32) + col / 32] = (uint8_t)s.byte;
      }
    }
  } else {
    // through LDS, 16 rows of this wave's 64 columns at a time, so that whole
    // 128-byte runs of a row are stored (65536 rows of 6144 x 2048 on 32 experts
    // 691 us against 782 with 32-byte runs from the accumulators; 641 non-temporal)
    const float alpha = p.alpha ? p.alpha[e] : 1.0f;
    const int col0 = wn * C::kWN;
    const uint16_t* bias = p.bias ? p.bias + (int64_t)e * p.N + n0 + col0 : nullptr;
    uint8_t* own = out + wave * 16 * kOutRow;
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm) {
      u4_t w[C::TN][2];
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn)
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // columns 16 c .. 16 c + 15 of the block
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = tn * 32 + Mfma<32>::row(8 * c + j, g);
            v[j] = alpha * acc[tm][tn][8 * c + j];
            if (bias && col0 + k < t.cols_c) v[j] += __uint_as_float((uint32_t)bias[k] << 16);
          }
          w[tn][c] = eight_columns(v);
        }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if ((lane >> 4 & 1) == half) {
#pragma unroll
          for (int tn = 0; tn < C::TN; ++tn)
#pragma unroll
            for (int c = 0; c < 2; ++c) *(u4_t*)(own + (lane & 15) * kOutRow + (tn * 32 + 16 * c + 8 * g) * 2) = w[tn][c];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * i + (lane >> 3), k = 8 * (lane & 7);
          const u4_t x = *(const u4_t*)(own + r * kOutRow + 2 * k);
          const int row = wm * C::kWM + tm * 32 + 16 * half + r, col = col0 + k;
          if (row < rows_c && col < t.cols_c) {
            uint16_t* to = p.d + (mc + row) * p.N + n0 + col;
            // non-temporal: the operands keep the caches (32768 rows of 6144 x 2048 on
            // 64 experts 407 -> 386 us, of 2048 x 768 84 -> 79)
            if (col + 8 <= t.cols_c) __builtin_nontemporal_store(x, (u4_any_t*)to);
            else
              for (int j = 0; j < t.cols_c - col; ++j) to[j] = (uint16_t)(x[j >> 1] >> (16 * (j & 1)));
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
}

// A work-group goes through the tiles that are gridDim.x apart.  The stage ring
// runs on over the ends of tiles: the next tile is looked up and its first stage
// loaded under the last products of the one before (8192 rows on 64 experts of
// 2 x 2048 x 6144 with a work-group a tile 309 us, like this 250; their down
// projections 187 and 165).
template <class C>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_mx_grouped_tile(MxGroupedLaunch p) {
  __shared__ __attribute__((aligned(16))) Smem<C> sm;
  __shared__ __attribute__((aligned(16))) uint8_t rows[C::kGated ? 16 : C::kWaves * 16 * kOutRow];
  const int64_t cols = C::kGated ? p.N / 2 : p.N;
  const int tiles_n = (int)((cols + C::kBRows - 1) / C::kBRows);
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN;
  const int n = (int)(p.K / C::BK);
  const int limit = (int)(most_tiles(p.rows, p.E, C::BM) * tiles_n);
  int L = xcd_remap(blockIdx.x, gridDim.x);
  TileJob<C> t = tile_job<C>(p, L, tiles_n, limit);
  if (t.e < 0) return;
  issue_tile<C>(sm, 0, t.ga, t.ra, t.ras, t.B, 0, wave, lane);
  wait_vm_barrier<0>();
  ReadAddr<C> rd = read_addr<C>(sm);
  int buf = 0;
#pragma unroll 1
  while (true) {
    typename C::Acc acc[C::TM][C::TN];
    zero_acc<C>(acc);
    const bool works = wm * C::kWM < t.rows_c;  // this wave has rows (uniform)
    const TileAtExpert out = t;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) {
        issue_tile<C>(sm, buf ^ 1, t.ga, t.ra, t.ras, t.B, i + 1, wave, lane);
      } else {
        L += gridDim.x;
        t = tile_job<C>(p, L, tiles_n, limit);
        if (t.e >= 0) issue_tile<C>(sm, buf ^ 1, t.ga, t.ra, t.ras, t.B, 0, wave, lane);
      }
      if (works) tile_stage<C, 0>(rd, acc);
      wait_vm_barrier<0>();
      // the other buffer
      const uint32_t step = buf ? 0u - C::BM * C::RB : C::BM * C::RB, sstep = buf ? 0u - C::BM * C::SB : C::BM * C::SB;
#pragma unroll
      for (int k = 0; k < ReadAddr<C>::kS; ++k) {
        rd.a[k] += step;
        rd.b[k] += step;
      }
      rd.as += sstep;
      rd.bs += sstep;
      buf ^= 1;
    }
    if (works) finish_tile<C>(p, out, acc, rows);
    if (t.e < 0) return;
  }
}

template <bool GATED>
static void launch_tile(const MxGroupedLaunch& p, hipStream_t stream) {
  typedef CfgExperts<GATED> C;
  const int64_t cols = GATED ? p.N / 2 : p.N, kCols = C::kBRows;
  const int64_t tiles = most_tiles(p.rows, p.E, C::BM) * ((cols + kCols - 1) / kCols);
  hipLaunchKernelGGL(k_mx_grouped_tile<C>, dim3((unsigned)(tiles < kCUs ? tiles : kCUs)), dim3(C::kThreads), 0, stream, p);
}

void launch_mx_grouped_tile(const MxGroupedLaunch& p, bool gated, hipStream_t stream) {
  if (gated) launch_tile<true>(p, stream);
  else launch_tile<false>(p, stream);
}

}  // namespace nvfp4
