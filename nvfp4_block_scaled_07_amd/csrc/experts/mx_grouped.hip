// Grouped products of MXFP4 operands: each expert's rows of A with the
// expert's own weights, for a mixture-of-experts layer.
//
//   plain: d[r][n] = bf16( alpha[e] sum_k A[row(r)][k] B_e[n][k] + bias[e][n] )
//   gated: h[r][i] = act(alpha[2e] sum A G_e + bias) (alpha[2e + 1] sum A U_e + bias),
//          B_e being I gate rows, then I up rows; h to MXFP4
//
// A few rows meet all weights of an expert, so the weight stream from HBM
// bounds the call.  Every weight is used by one wave only and goes straight to
// registers: a unit (256 elements of K, one 128-byte line a row) of a wave's 32
// rows is 4 whole-line loads, kU units ahead.  What the waves of a work-group
// share, the rows of A and the scales of both operands, is staged in LDS one
// chunk of kU units ahead (double buffer, one barrier a chunk); waiting for it
// leaves the weights in flight.  No dequantisation: the scaled FP4 MFMA takes
// the codes and the E8M0 bytes as they are.
//
// Measured: 64 tokens on 8 of 256 experts of 2 x 2048 x 6144, 2.97 GB of weights
// in 452 us (6.6 TB/s; a sum over 2 GB reads 6.1), down projections of 6144 x 2048
// 219 us (6.8); one token 21 and 14 us.
//
// The weights are the MFMA's first operand, so a lane ends with four
// consecutive columns of one row, and an MXFP4 block lies in the registers of
// 4 lanes of two waves.
#include "../block/epilogue.h"
#include "expert_tile.h"
#include "mx_block.h"

namespace nvfp4 {

// 0, 1 + the first expert whose offsets are wrong, or -(1 + the first covered
// row whose token is outside [0, T)).
__global__ __launch_bounds__(1024) void k_expert_status(const int32_t* __restrict__ offsets, int E,
                                                        const int32_t* __restrict__ tok, int64_t rows, int64_t T,
                                                        int32_t* status) {
  __shared__ int bad, first;
  if (threadIdx.x == 0) bad = first = INT32_MAX;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) {
    const int64_t lo = offsets[e], hi = offsets[e + 1];
    if (lo < 0 || hi < lo || hi > rows) atomicMin(&bad, e);
  }
  __syncthreads();
  if (tok && bad == INT32_MAX) {
    const int64_t end = E > 0 ? offsets[E] : 0;
    for (int64_t i = (E > 0 ? offsets[0] : 0) + threadIdx.x; i < end; i += 1024) {
      const int64_t t = tok[i];
      if (t < 0 || t >= T) atomicMin(&first, (int)i);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *status = bad != INT32_MAX ? bad + 1 : first != INT32_MAX ? -(first + 1) : 0;
}

template <int BM_, bool GATED_, int WAVES_, int OCC_>
struct StreamCfg {
  static constexpr int BM = BM_, TM = BM / 16, TN = 2;
  static constexpr bool kGated = GATED_;
  static constexpr int kOcc = OCC_;                // waves per SIMD that the registers must leave room for
  static constexpr int kWaves = WAVES_, kThreads = 64 * kWaves;
  static constexpr int kU = 4;                     // units of a chunk, and in flight a wave
  static constexpr int kRow = 8 * kU;              // 16-byte pieces of a row in a chunk
  static constexpr int kBRows = 32 * kWaves;       // weight rows of a tile
  static constexpr int kCols = GATED_ ? kBRows / 2 : kBRows;  // output columns
  static constexpr int kPieces = BM * kRow / kThreads;  // pieces of A a thread stages
  static constexpr int kASf = (BM * kU + kThreads - 1) / kThreads;  // 8-byte pieces of A's scales
  static constexpr int kASRows = kASf * kThreads / kU;  // rows that those cover (no branch around the last)
  static constexpr int kBSf = kBRows * kU / kThreads;
  static_assert(kPieces * kThreads == BM * kRow && kThreads / kU % 32 == 0, "whole shares");
  static constexpr int kOut = kCols * 2 + 16;      // bytes of an output row in LDS (16 more: other banks)
};

template <class C>
struct StreamSmem {
  union {
    struct {
      // [row][pieces of 16 bytes], piece p of row r at slot p ^ (r & 15)
      uint8_t a[2][C::BM * C::kRow * 16];
      uint8_t asf[2][C::kASRows * C::kU * 8], bsf[2][C::kBRows * C::kU * 8];
    };
    uint8_t out[C::BM * C::kOut];  // bf16 outputs of a tile, once the products are done
    uint32_t peak[C::kWaves][C::BM];
  };
};

template <class C>
struct Staged {
  u4_t a[C::kPieces];
  u2_t as[C::kASf], bs[C::kBSf];
};

constexpr uint32_t kOutside = 0x80000000u;
constexpr int kStreaming = 2;  // buffer loads that leave the caches to others (non-temporal)

// LDS accesses of this wave done, then a work-group barrier; loads in flight
// are left alone.
__device__ __forceinline__ void stage_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// bf16 values p[0 .. 3], the first n of them (else 0)
__device__ __forceinline__ void load_bias4(float (&b)[4], const uint16_t* p, int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = j < n ? __uint_as_float((uint32_t)p[j] << 16) : 0.0f;
}

// The outputs of a tile.  Lane 16 g + r holds row r of each 16 rows, columns 4 g
// .. 4 g + 3 of each column block: the tile goes through LDS, so that whole runs
// of a row are stored (8-byte stores straight from the accumulators cost 4096 rows
// of 6144 columns, 50 MB, 46 us of 351; like this it is 6).
template <class C>
__device__ __forceinline__ void store_plain(const MxGroupedLaunch& p, int e, int64_t mc, int rows_c, int64_t n0, int valid,
                                            const Mfma<16>::Acc (&acc)[C::TM][C::TN], uint8_t* out) {
  const int lane = threadIdx.x & 63, wave = wave_id(), r_in = lane & 15, g = lane >> 4;
  const float alpha = p.alpha ? p.alpha[e] : 1.0f;
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn) {
    const int col = 32 * wave + 16 * tn + 4 * g;
    float b[4];
    if (p.bias) load_bias4(b, p.bias + (int64_t)e * p.N + n0 + col, valid - col);
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = p.bias ? alpha * acc[tm][tn][j] + b[j] : alpha * acc[tm][tn][j];
      *(u2_t*)(out + (tm * 16 + r_in) * C::kOut + 2 * col) = u2_t{f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3])};
    }
  }
  stage_barrier();
  constexpr int kRuns = C::kCols / 8;  // 16-byte runs of a row
  for (int i = threadIdx.x; i < rows_c * kRuns; i += C::kThreads) {
    const int row = i / kRuns, col = i % kRuns * 8;
    if (col >= valid) continue;
    const u4_t w = *(const u4_t*)(out + row * C::kOut + 2 * col);
    uint16_t* to = p.d + (mc + row) * p.N + n0 + col;
    // non-temporal: 4096 rows of 6144 columns on 256 experts 324 -> 307 us
    if (col + 8 <= valid) __builtin_nontemporal_store(w, (u4_any_t*)to);
    else
      for (int j = 0; j < valid - col; ++j) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

// The same for a gated tile: column block 0 is the gate, 1 the up projection of
// columns 16 wave + 4 g ..; a block of 32 is in two waves, whose peaks meet in
// LDS.
template <class C>
__device__ __forceinline__ void store_gated(const MxGroupedLaunch& p, int e, int64_t mc, int rows_c, int64_t n0, int valid,
                                            const Mfma<16>::Acc (&acc)[C::TM][C::TN], uint32_t (&peak)[C::kWaves][C::BM]) {
  const int lane = threadIdx.x & 63, wave = wave_id(), r_in = lane & 15, g = lane >> 4;
  const float a0 = p.alpha ? p.alpha[2 * e] : 1.0f, a1 = p.alpha ? p.alpha[2 * e + 1] : 1.0f;
  const int col = 16 * wave + 4 * g;
  const bool in = col < valid;  // blocks of 32 are whole
  const int64_t I = p.N / 2, n = n0 + col;
  float bg[4], bu[4];
  const bool bias = p.bias && in;
  if (bias) {
    load_bias4(bg, p.bias + (int64_t)e * p.N + n, 4);
    load_bias4(bu, p.bias + (int64_t)e * p.N + I + n, 4);
  }
  float h[C::TM][4];
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[tm][j] = bias ? a0 * acc[tm][0][j] + bg[j] : a0 * acc[tm][0][j];
    activate<4>(h[tm], p.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[tm][j] *= bias ? a1 * acc[tm][1][j] + bu[j] : a1 * acc[tm][1][j];
      top = umax(top, magnitude(h[tm][j]));
    }
    top = umax(top, (uint32_t)__shfl_xor((int)top, 16));
    top = umax(top, (uint32_t)__shfl_xor((int)top, 32));
    if (g == 0) peak[wave][tm * 16 + r_in] = top;
  }
  stage_barrier();
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) {
    const int row = tm * 16 + r_in;
    const MxScale s = mx_scale(umax(peak[wave][row], peak[wave ^ 1][row]), p.rule);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h[tm][0] * s.r, h[tm][1] * s.r, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, h[tm][2] * s.r, h[tm][3] * s.r, 1.0f, 1);
    if (row < rows_c && in) {
      const int64_t r = mc + row;
      *(uint16_t*)(p.q + r * (I / 2) + n / 2) = (uint16_t)(w & s.keep);
      if (g == 0 && (wave & 1) == 0) p.sf[r * (I / 32) + n / 32] = (uint8_t)s.byte;
    }
  }
}

template <class C>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::kOcc))) void k_mx_grouped(MxGroupedLaunch p) {
  typedef int v8i_t __attribute__((ext_vector_type(8)));
  __shared__ __attribute__((aligned(16))) StreamSmem<C> sm;
  const int64_t cols = C::kGated ? p.N / 2 : p.N;
  const int tiles_n = (int)((cols + C::kCols - 1) / C::kCols);
  // column tiles of one row tile follow each other, so they are spread over the
  // XCDs (with a run of tiles to each XCD, experts of unequal rows leave some idle:
  // 16 tokens on 256 experts 268 us against 228)
  const int L = (int)blockIdx.x, q = L / tiles_n;
  const ExpertTile at = find_tile<C::BM>(p, q);
  if (at.expert < 0) return;
  const int e = at.expert;
  const int64_t n0 = (int64_t)(L % tiles_n) * C::kCols, mc = at.lo + (int64_t)(q - at.first) * C::BM;
  const int rows_c = (int)min<int64_t>(C::BM, at.hi - mc);
  const int64_t ld = p.K / 2, lds = p.K / 32;
  const int nu = (int)(p.K / 256), chunks = (nu + C::kU - 1) / C::kU;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int r_in = lane & 15, g = lane >> 4;
  const bool lo8 = (lane & 8) == 0;

  // weight rows: column block tn of wave w is rows 32 w + 16 tn .. of the tile,
  // or (gated) rows 16 w .. of the tile in matrix tn; rows past the tile's last
  // lie past the end of its buffer
  const int valid = (int)min<int64_t>(C::kCols, cols - n0);
  const uint8_t* b0 = p.b + ((int64_t)e * p.N + n0) * ld;
  const uint8_t* s0 = p.b_sf + ((int64_t)e * p.N + n0) * lds;
  const int64_t second = C::kGated ? p.N / 2 : 0;  // rows from the first matrix to the second
  const rsrc_t rs = make_rsrc(s0, (uint32_t)(valid * lds)), rs2 = make_rsrc(s0 + second * lds, (uint32_t)(valid * lds));
  uint32_t vb[C::TN][2];
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      vb[tn][h] = (uint32_t)(((C::kGated ? 16 * wave : 32 * wave + 16 * tn) + 8 * h + (lane & 7)) * ld + 16 * (lane >> 3));
  // 8-byte pieces of the weights' scales: row tid / kU of the tile's LDS order
  // (wave, block, row), unit tid % kU of the chunk
  uint32_t vbs[C::kBSf];
  const int su = tid % C::kU, pc = tid % C::kRow;
#pragma unroll
  for (int i = 0; i < C::kBSf; ++i) {
    const int row = tid / C::kU + i * (C::kThreads / C::kU);
    const int w = row >> 5, tn = (row >> 4) & 1, r = row & 15;
    vbs[i] = (uint32_t)((C::kGated ? 16 * w + r : 32 * w + 16 * tn + r) * lds + 8 * su);
  }
  // the matrix of this thread's scale pieces: rows 16 .. 31 of a wave's 32 are the second's
  const bool odd_block = C::kGated && (tid / C::kU >> 4 & 1);

  rsrc_t ra, ras;
  if (p.row_token) {
    // never empty, so that no chunk's scalar offset lies past the end (without
    // tokens every row's vector offset does)
    const int64_t most = max(p.T, (int64_t)1);
    ra = make_rsrc(p.a, (uint32_t)(most * ld));
    ras = make_rsrc(p.a_sf, (uint32_t)(most * lds));
  } else {
    ra = make_rsrc(p.a + mc * ld, (uint32_t)(rows_c * ld));
    ras = make_rsrc(p.a_sf + mc * lds, (uint32_t)(rows_c * lds));
  }
  const auto source = [&](int r) -> int64_t {  // row r's row of a, or -1
    if (r >= rows_c) return -1;
    if (!p.row_token) return r;
    const int64_t t = p.row_token[mc + r];
    return t >= 0 && t < p.T ? t : -1;
  };
  uint32_t va[C::kPieces], vas[C::kASf];
#pragma unroll
  for (int i = 0; i < C::kPieces; ++i) {
    const int64_t t = source(tid / C::kRow + i * (C::kThreads / C::kRow));
    va[i] = t >= 0 ? (uint32_t)(t * ld + 16 * pc) : kOutside;
  }
#pragma unroll
  for (int i = 0; i < C::kASf; ++i) {
    const int r = tid / C::kU + i * (C::kThreads / C::kU);
    const int64_t t = r < C::BM ? source(r) : -1;
    vas[i] = t >= 0 ? (uint32_t)(t * lds + 8 * su) : kOutside;
  }

  Staged<C> st;
  u4_t bq[C::kU][C::TN][2];
  Mfma<16>::Acc acc[C::TM][C::TN];
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) acc[tm][tn] = Mfma<16>::Acc{0.f, 0.f, 0.f, 0.f};

  // units past the end of K read out of range: zero codes and scales.  The chunk
  // behind the last one has no scalar offset, which may lie past a buffer's end.
  const auto stage_load = [&](int c) {
    const int at = c < chunks ? c : 0;
    const bool piece = C::kU * c + (pc >> 3) < nu, scale = C::kU * c + su < nu;
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i)
      st.a[i] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, piece ? va[i] : kOutside, at * C::kRow * 16, 0));
#pragma unroll
    for (int i = 0; i < C::kASf; ++i)
      st.as[i] = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(ras, scale ? vas[i] : kOutside, at * C::kU * 8, 0));
#pragma unroll
    for (int i = 0; i < C::kBSf; ++i) {
      const uint32_t off = scale ? vbs[i] : kOutside;
      if constexpr (C::kGated) {
        // a thread's rows are of one matrix: it loads from its own
        const u2_t x = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs, odd_block ? kOutside : off, at * C::kU * 8, 0));
        const u2_t y = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs2, odd_block ? off : kOutside, at * C::kU * 8, 0));
        st.bs[i] = odd_block ? y : x;
      } else {
        st.bs[i] = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs, off, at * C::kU * 8, 0));
      }
    }
  };
  const auto stage_store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
      const int r = tid / C::kRow + i * (C::kThreads / C::kRow);
      *(u4_t*)(sm.a[buf] + (r * C::kRow + (pc ^ (r & 15))) * 16) = st.a[i];
    }
#pragma unroll
    for (int i = 0; i < C::kASf; ++i) {
      const int r = tid / C::kU + i * (C::kThreads / C::kU);
      *(u2_t*)(sm.asf[buf] + (r * C::kU + su) * 8) = st.as[i];
    }
#pragma unroll
    for (int i = 0; i < C::kBSf; ++i) {
      const int r = tid / C::kU + i * (C::kThreads / C::kU);
      *(u2_t*)(sm.bsf[buf] + (r * C::kU + su) * 8) = st.bs[i];
    }
  };
  const auto unit_load = [&](int u, int unit) {
    const bool live = unit < nu;  // uniform: an empty buffer and no offset else
    // kStreaming: the weights of an expert of one row tile are used once.  16 tokens on
    // 256 experts 341 -> 310 us (both products), 37 rows an expert on 64 experts 274 ->
    // 257; 64 rows, where every other expert has two tiles, 356 -> 368: at every tile
    // height, as the rows of single experts are not known here.
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) {
      const rsrc_t r = make_rsrc(C::kGated && tn ? b0 + second * ld : b0, live ? (uint32_t)(valid * ld) : 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        bq[u][tn][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, vb[tn][h], live ? unit * 128 : 0, kStreaming));
    }
  };
  const auto unit_compute = [&](int buf, int u) {
    v8i_t bv[C::TN][2];
    int sb[C::TN];
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = bq[u][tn][0][j];
        w[4 + j] = bq[u][tn][1][j];
      }
      kreg_exchange(w, lo8);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        bv[tn][c] = v8i_t{(int)w[4 * c], (int)w[4 * c + 1], (int)w[4 * c + 2], (int)w[4 * c + 3], 0, 0, 0, 0};
      sb[tn] = *(const uint16_t*)(sm.bsf[buf] + ((wave * 32 + tn * 16 + r_in) * C::kU + u) * 8 + 2 * g);
    }
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm) {
      const int row = tm * 16 + r_in;
      const int sa = *(const uint16_t*)(sm.asf[buf] + (row * C::kU + u) * 8 + 2 * g);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const u4_t x = *(const u4_t*)(sm.a[buf] + (row * C::kRow + ((8 * u + 2 * g + c) ^ r_in)) * 16);
        const v8i_t av = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
#pragma unroll
        for (int tn = 0; tn < C::TN; ++tn)
          acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[tn][c], av, acc[tm][tn], 4, 4, 0,
                                                                         sb[tn] >> (8 * c), 0, sa >> (8 * c));
      }
      // computed here: not moved down to where a tile ends (no instruction reads it)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) asm volatile("" : "+v"(acc[tm][tn]));
    }
  };

  stage_load(0);
#pragma unroll
  for (int u = 0; u < C::kU; ++u) {
    unit_load(u, u);
    __builtin_amdgcn_sched_barrier(0);
  }
  stage_store(0);
  stage_barrier();
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    stage_load(c + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < C::kU; ++u) {
      unit_compute(c & 1, u);
      // the slot's reload stays behind its last reads
      __builtin_amdgcn_sched_barrier(0);
      unit_load(u, C::kU * (c + 1) + u);
    }
    stage_store((c + 1) & 1);
    stage_barrier();
  }
  if constexpr (C::kGated) store_gated<C>(p, e, mc, rows_c, n0, valid, acc, sm.peak);
  else store_plain<C>(p, e, mc, rows_c, n0, valid, acc, sm.out);
}

template <int BM, bool GATED>
static void launch_stream(const MxGroupedLaunch& p, hipStream_t stream) {
  // three work-groups a CU where the registers allow it (a fourth wave a SIMD,
  // or a third of the 64-row tile, spills and is slower)
  typedef StreamCfg<BM, GATED, 4, BM == 16 ? 3 : 2> C;
  const int64_t cols = GATED ? p.N / 2 : p.N;
  const unsigned grid = (unsigned)((cols + C::kCols - 1) / C::kCols * most_tiles(p.rows, p.E, BM));
  hipLaunchKernelGGL(k_mx_grouped<C>, dim3(grid), dim3(C::kThreads), 0, stream, p);
}

template <bool GATED>
static void launch_rows(const MxGroupedLaunch& p, hipStream_t stream) {
  // The host knows rows and E, whose quotient is the average rows of an expert if
  // all rows are these experts'.  With a range of the experts, rows that others have
  // count as well, and the tiles may be too high: 32 of 256 experts of 2 x 2048 x 6144,
  // 8 a token, both products by top_k T rows and by those that exist, 16 tokens 55 and
  // 55 us, 64 106 and 102, 128 123 and 109, 512 188 and 113.  Measured (us, both
  // products of a feed-forward of 2048 x 6144, rows on average, by tile height
  // 16 / 32 / 64 / 256, with weight loads that stay in the caches): 2 rows 727 / 734 /
  // 792, 16 rows 1113 / 926 / 973, 64 rows 729 / 448 / 356 / 377, 80 rows 436 / 383 by
  // the last two, 128 rows 543 / 417 (256 experts up to 16 rows, 64 from there).  As
  // they are now: 16 rows by 32 867, 37 rows by 64 257, 64 rows 368 by 64 and by 256.
  if (p.rows <= 4 * (int64_t)p.E) launch_stream<16, GATED>(p, stream);
  else if (p.rows <= 24 * (int64_t)p.E) launch_stream<32, GATED>(p, stream);
  else if (p.rows <= 64 * (int64_t)p.E) launch_stream<64, GATED>(p, stream);
  else launch_mx_grouped_tile(p, GATED, stream);
}

hipError_t launch_mx_grouped(const MxGroupedLaunch& p, bool gated, hipStream_t stream) {
  if (gated) launch_rows<true>(p, stream);
  else launch_rows<false>(p, stream);
  return hipGetLastError();
}

hipError_t launch_expert_status(const int32_t* offsets, int E, const int32_t* row_token, int64_t rows, int64_t T,
                                int32_t* status, hipStream_t stream) {
  hipLaunchKernelGGL(k_expert_status, dim3(1), dim3(1024), 0, stream, offsets, E, row_token, rows, T, status);
  return hipGetLastError();
}

}  // namespace nvfp4
