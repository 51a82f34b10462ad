// Register-streamed NVFP4 / MXFP4 tiles: operand loads straight into
// registers and the K-group main loop, shared by the plain GEMM (gemm.hip)
// and the GEMMs with a fused epilogue (block/).  Device functions only; each
// kernel instantiation lives in the one source that launches it.
#pragma once

#include "gemm_tile.h"

namespace nvfp4 {

// Whole-line operand loads: two 16-byte loads per lane cover a 16-row block of
// one 256-K unit (128 bytes per row) as 8 whole lines each, lane l reading row
// l % 8 (words 0..3) and row 8 + l % 8 (words 4..7), chunk l / 8 of each.
// Exchange with the lane 8 away in the same row of 16 so that lane 16 g + r
// holds row r, chunk 2 g in words 0..3 and chunk 2 g + 1 in words 4..7: the
// 16x16x32 MFMA operand layout, with K permuted the same way for A and B.
__device__ __forceinline__ void kreg_exchange(uint32_t (&w)[8], bool lo8) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t p = w[j], q = w[4 + j];
    const uint32_t give = lo8 ? q : p;
    const uint32_t recv = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x128, 0xF, 0xF, false);  // row_ror:8
    w[j] = lo8 ? p : recv;
    w[4 + j] = lo8 ? recv : q;
  }
}

// Scale layouts the register-streamed kernels can read in place
// (nvfp4_gemm_sf, nvfp4_grouped_gemm_sf): 0 linear [rows][K/16]; 1 the 128 x
// 4 tiled layout (512-byte tiles of 128 rows x 4 scale columns, row-major
// tile order; row r, column c at byte (r % 32) 16 + ((r % 128) / 32) 4 + c %
// 4); 2 the 8 x 4 one (32-byte tiles of 8 rows x 4 columns; row r, column c
// at byte (r % 8) 4 + c % 4).  In both tiled layouts the 4 scales of columns
// 4 j .. 4 j + 3 of a row are one aligned word, the word a lane loads, so
// only its address changes.
template <int SFL>
struct SfLayout {
  static_assert(SFL >= 0 && SFL <= 2, "scale layout");
  // bytes between consecutive 256-element units of one row (4 words)
  static constexpr uint32_t kUnitStep = SFL == 0 ? 16 : (SFL == 1 ? 4 * 512 : 4 * 32);
  // Rows [r0, r0 + rows_valid) of a scale matrix with lds = K/16 bytes per
  // row (r0 counts rows from the matrix start, any alignment): a descriptor
  // bounded by the bytes of the row groups those rows occupy, and the offset
  // of word j of local row r in unit 0.
  static __device__ __forceinline__ rsrc_t rsrc(const uint8_t* sf, int64_t r0, int rows_valid, int64_t lds) {
    if constexpr (SFL == 0) return make_rsrc(sf + r0 * lds, (uint32_t)(rows_valid * lds));
    else if constexpr (SFL == 1)
      return make_rsrc(sf + (r0 >> 7) * 128 * lds, (uint32_t)(((r0 & 127) + rows_valid + 127) / 128 * 128 * lds));
    else return make_rsrc(sf + (r0 >> 3) * 8 * lds, (uint32_t)(((r0 & 7) + rows_valid + 7) / 8 * 8 * lds));
  }
  static __device__ __forceinline__ uint32_t offset(int64_t r0, int r, int j, int64_t lds) {
    if constexpr (SFL == 0) return (uint32_t)(r * lds + 4 * j);
    else if constexpr (SFL == 1) {
      const int q = (int)(r0 & 127) + r;
      return (uint32_t)((q >> 7) * 128 * lds + 512 * j + (q & 31) * 16 + ((q >> 5) & 3) * 4);
    } else {
      const int q = (int)(r0 & 7) + r;
      return (uint32_t)((q >> 3) * 8 * lds + 32 * j + (q & 7) * 4);
    }
  }
};

// ---------------------------------------------------------------------------
// Register-streamed K-group GEMM for small and mid M (no LDS staging).  A
// work-group owns one BM x BN output tile and a K range (all of K, or split z
// of S); its KS waves are K-groups: wave w takes the 256-element K units w,
// w + KS, w + 2 KS, ... of the range.  Every lane loads its 16-byte code
// chunks and scale words straight into registers, D units ahead, dequantises
// them and issues 16x16x32 f16 MFMAs on its wave's full tile.  The KS partial
// tiles are summed through LDS in wave order (deterministic); with S > 1 the
// last split to finish sums the S partials in split order.
//
// A unit is 128 bytes of codes per row, one cache line.  Each 16-row block is
// loaded with two instructions that each cover 8 whole lines: lane l reads
// row l % 8 (then row 8 + l % 8), bytes 16 (l / 8) .. 16 (l / 8) + 15.  On a
// cold call the number of outstanding requests per CU is what limits the
// rate, and whole-line requests carry twice the bytes of the half lines a
// 16-row instruction would fetch.  One DPP rotation by 8 lanes within each
// row of 16 then gives lane l = 16 g + r row r with chunks 2 g (words 0..3)
// and 2 g + 1 (words 4..7), K elements 64 g .. 64 g + 63 of the unit; its
// scale word is bytes 4 g .. 4 g + 3 of the row's 16 unit scales.  MFMA t of
// chunk c multiplies elements 8 t .. 8 t + 7 of that chunk, the same K set
// for A and B.
//
// MX tiles (MXFP4: one E8M0 scale per 32 elements) use the same loads and
// exchange and no dequantisation: chunk c of every lane (32 codes, one MX
// block) is the lane's operand of one v_mfma_scale_f32_16x16x128_f8f6f4
// (lane 16 g + r: row r, K block g of the MFMA; its scale operand's low byte
// applies to that row and block; the output layout is that of the 16x16 f16
// MFMA).  Lane 16 g + r loads scale word g / 2 of the row's 8 unit scales;
// bytes 2 g and 2 g + 1 of the unit are those of its chunks.
//
// GATED tiles pair two weight matrices stored one after the other in B
// ([N / 2] gate rows, then [N / 2] up rows): column blocks 0 .. TN / 2 - 1 of
// the tile are gate rows n0 .., blocks TN / 2 .. TN - 1 the same up rows, so a
// tile covers BN / 2 gate columns and holds the product's two factors.  With
// GATED 2 every column block holds 8 gate rows and the same 8 up rows instead
// (the two whole-line loads of a block read 8 rows each as it is), for tiles
// of 8 outputs; the scales of both matrices then lie in one descriptor, so
// N K / 32 < 2^31.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int KS_, int D_, int OCC_, int MX_ = 0, int GATED_ = 0>
struct KCfg {
  static constexpr bool kGated = GATED_ != 0, kHalves = GATED_ == 2;
  static constexpr int BM = BM_, BN = BN_, KS = KS_, D = D_, OCC = OCC_;
  static constexpr bool kMx = MX_ != 0;
  static constexpr int SBLK = kMx ? 32 : 16;        // elements per scale
  static constexpr int TM = BM / 16, TN = BN / 16;
  static constexpr int kBlkN = GATED_ == 1 ? TN / 2 : TN;  // column blocks of one B matrix
  static constexpr int kThreads = KS * 64;
  static constexpr int kTileFloats = BM * BN;        // one wave's partial tile
  static constexpr int kUnit = 256;                  // K elements per unit
  static_assert(BM % 16 == 0 && BN % 16 == 0, "16-row MFMA blocks");
  static_assert(!kGated || ((TN % 2 == 0 || kHalves) && !kMx), "gated tiles pair NVFP4 column blocks");
  static_assert(KS >= 1 && KS <= 16, "waves per work-group");
  static_assert(KS * kTileFloats * 4 <= 65536, "partial tiles fit in 64 KB of LDS");
};

template <class C>
struct KRegs {
  uint32_t aq[C::D][C::TM][8], bq[C::D][C::TN][8];  // two 16-byte code chunks as words
  uint32_t as[C::D][C::TM], bs[C::D][C::TN];        // scale words (4 e4m3)
};

// Loads of unit `unit` into slot u; dead units (past the end of the range)
// read out of range, which returns zero without a memory access, so every
// iteration issues the same loads.
template <class C, int SFL>
__device__ __forceinline__ void kreg_load(KRegs<C>& R, int u, int unit, bool live, const rsrc_t& ra,
                                          const rsrc_t& ras, const rsrc_t& rb, const rsrc_t& rbs,
                                          const rsrc_t& rb2, const rsrc_t& rbs2,
                                          const uint32_t (&va)[C::TM][2], const uint32_t (&vas)[C::TM],
                                          const uint32_t (&vb)[C::TN][2], const uint32_t (&vbs)[C::TN]) {
  constexpr uint32_t kOut = 0x80000000u;
  const int so = unit * (C::kUnit / 2);
  const int sso = unit * (SFL == 0 ? C::kUnit / C::SBLK : (int)SfLayout<SFL>::kUnitStep);
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u4_t v = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, live ? va[tm][h] : kOut, so, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) R.aq[u][tm][4 * h + j] = v[j];
    }
    R.as[u][tm] = __builtin_amdgcn_raw_buffer_load_b32(ras, live ? vas[tm] : kOut, sso, 0);
  }
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u4_t v = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(tn < C::kBlkN && !(C::kHalves && h) ? rb : rb2, live ? vb[tn][h] : kOut, so, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) R.bq[u][tn][4 * h + j] = v[j];
    }
    R.bs[u][tn] = __builtin_amdgcn_raw_buffer_load_b32(tn < C::kBlkN ? rbs : rbs2, live ? vbs[tn] : kOut, sso, 0);
  }
}

// Multiply-accumulate slot u's unit into acc.
template <class C>
__device__ __forceinline__ void kreg_unit(KRegs<C>& R, int u, bool lo8, int g, Mfma<16>::Acc (&acc)[C::TM][C::TN]) {
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) kreg_exchange(R.aq[u][tm], lo8);
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn) kreg_exchange(R.bq[u][tn], lo8);
  if constexpr (C::kMx) {
    typedef int v8i_t __attribute__((ext_vector_type(8)));
    const int ssh = 16 * (g & 1);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      v8i_t bv[C::TN];
      int sb[C::TN];
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) {
        const uint32_t* w = R.bq[u][tn] + 4 * c;
        bv[tn] = v8i_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        sb[tn] = (int)(R.bs[u][tn] >> (ssh + 8 * c));
      }
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
        const uint32_t* w = R.aq[u][tm] + 4 * c;
        const v8i_t av = v8i_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        const int sa = (int)(R.as[u][tm] >> (ssh + 8 * c));
#pragma unroll
        for (int tn = 0; tn < C::TN; ++tn)
          acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv[tn], acc[tm][tn], 4, 4, 0, sa, 0,
                                                                         sb[tn]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      h2_t asp[C::TM], bsp[C::TN];
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) asp[tm] = e4m3x2_to_h2(R.as[u][tm] >> (16 * c));
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) bsp[tn] = e4m3x2_to_h2(R.bs[u][tn] >> (16 * c));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        h8_t bf[C::TN];
#pragma unroll
        for (int tn = 0; tn < C::TN; ++tn) bf[tn] = dequant8(R.bq[u][tn][4 * c + t], scale_pair(bsp[tn], t >> 1));
#pragma unroll
        for (int tm = 0; tm < C::TM; ++tm) {
          const h8_t af = dequant8(R.aq[u][tm][4 * c + t], scale_pair(asp[tm], t >> 1));
#pragma unroll
          for (int tn = 0; tn < C::TN; ++tn) acc[tm][tn] = Mfma<16>::run(af, bf[tn], acc[tm][tn]);
        }
      }
    }
  }
}

// Split z of S (all of K when S is 1) of the BM x BN tile at row m0 of A and row n0
// of B into this wave's accumulators (its K-group's share; the caller sums
// the KS waves).  rows_a, rows_b: valid rows of each operand in the tile
// (of each matrix in a gated tile); rows past them read as zero.
template <class C, int SFL, bool SKIP = false>
__device__ __forceinline__ void kreg_accumulate(const GemmLaunch& p, int64_t m0, int64_t n0, int rows_a, int rows_b,
                                                int z, int S, Mfma<16>::Acc (&acc)[C::TM][C::TN]) {
  const int64_t ld = p.K / 2, lds = p.K / C::SBLK;
  const rsrc_t ra = make_rsrc(p.a + m0 * ld, (uint32_t)(rows_a * ld));
  const rsrc_t ras = SfLayout<SFL>::rsrc(p.a_sf, m0, rows_a, lds);
  const rsrc_t rb = make_rsrc(p.b + n0 * ld, (uint32_t)(rows_b * ld));
  const rsrc_t rbs = C::kHalves ? make_rsrc(p.b_sf + n0 * lds, (uint32_t)((p.N / 2 + rows_b) * lds))
                                : SfLayout<SFL>::rsrc(p.b_sf, n0, rows_b, lds);
  // the second matrix of a gated tile
  const int64_t n2 = C::kGated ? p.N / 2 + n0 : n0;
  const rsrc_t rb2 = C::kGated ? make_rsrc(p.b + n2 * ld, (uint32_t)(rows_b * ld)) : rb;
  const rsrc_t rbs2 = C::kGated ? SfLayout<SFL>::rsrc(p.b_sf, n2, rows_b, lds) : rbs;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r_in = lane & 15, g = lane >> 4;
  // code offsets: rows lane % 8 and 8 + lane % 8 of each 16-row block, bytes
  // 16 (lane / 8) of the unit; scale word g (MX: g / 2) of row r_in
  const int sw = C::kMx ? 4 * (g >> 1) : 4 * g;
  uint32_t va[C::TM][2], vas[C::TM], vb[C::TN][2], vbs[C::TN];
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = tm * 16 + 8 * h + (lane & 7);
      va[tm][h] = r < rows_a ? (uint32_t)(r * ld + 16 * (lane >> 3)) : 0x80000000u;
    }
    const int r = tm * 16 + r_in;
    if constexpr (SFL == 0) vas[tm] = r < rows_a ? (uint32_t)(r * lds + sw) : 0x80000000u;
    else vas[tm] = r < rows_a ? SfLayout<SFL>::offset(m0, r, g, lds) : 0x80000000u;
  }
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn) {
    if constexpr (C::kHalves) {
      static_assert(SFL == 0 || !C::kHalves, "linear scales");
      const int r = tn * 8 + (lane & 7);
      vb[tn][0] = vb[tn][1] = r < rows_b ? (uint32_t)(r * ld + 16 * (lane >> 3)) : 0x80000000u;
      vbs[tn] = r < rows_b ? (uint32_t)((r + (lane & 8 ? p.N / 2 : 0)) * lds + sw) : 0x80000000u;
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (tn % C::kBlkN) * 16 + 8 * h + (lane & 7);
      vb[tn][h] = r < rows_b ? (uint32_t)(r * ld + 16 * (lane >> 3)) : 0x80000000u;
    }
    const int r = (tn % C::kBlkN) * 16 + r_in;
    if constexpr (SFL == 0) vbs[tn] = r < rows_b ? (uint32_t)(r * lds + sw) : 0x80000000u;
    else vbs[tn] = r < rows_b ? SfLayout<SFL>::offset(tn < C::kBlkN ? n0 : n2, r, g, lds) : 0x80000000u;
  }
  // this work-group's K units [u_lo, u_hi): all of K, or split z of S
  const int nu_all = (int)(p.K / C::kUnit);
  const int u_lo = (int)((int64_t)z * nu_all / S), u_hi = (int)((int64_t)(z + 1) * nu_all / S);
  const int nu = u_hi - u_lo;
  // every wave runs the same number of iterations (a multiple of D); units
  // past the end are dead
  const int per_wave = (nu + C::KS - 1) / C::KS;
  const int iters = (per_wave + C::D - 1) / C::D * C::D;
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) acc[tm][tn] = Mfma<16>::Acc{0.f, 0.f, 0.f, 0.f};
  KRegs<C> R;
#pragma unroll
  for (int u = 0; u < C::D; ++u) {
    const int unit = wave + u * C::KS;
    kreg_load<C, SFL>(R, u, u_lo + unit, unit < nu, ra, ras, rb, rbs, rb2, rbs2, va, vas, vb, vbs);
    __builtin_amdgcn_sched_barrier(0);
  }
  const bool lo8 = (lane & 8) == 0;
  for (int i0 = 0; i0 < iters; i0 += C::D) {
#pragma unroll
    for (int u = 0; u < C::D; ++u) {
      // SKIP: a unit past the end of the range adds zeros; leave them out
      if (!SKIP || wave + (i0 + u) * C::KS < nu) kreg_unit<C>(R, u, lo8, g, acc);
      // the slot's reload stays after its last reads (old and new contents
      // share registers; no copies that would wait on the load)
      __builtin_amdgcn_sched_barrier(0);
      const int unit = wave + (i0 + u + C::D) * C::KS;
      kreg_load<C, SFL>(R, u, u_lo + unit, unit < nu, ra, ras, rb, rbs, rb2, rbs2, va, vas, vb, vbs);
    }
  }
}

}  // namespace nvfp4
