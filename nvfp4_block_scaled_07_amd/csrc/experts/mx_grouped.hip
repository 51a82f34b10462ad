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
// rows is 4 whole-line loads, kD units ahead.  What the waves of a work-group
// share, the rows of A and the scales of both operands, is staged in LDS one
// chunk of kD units ahead (double buffer, one barrier a chunk); waiting for it
// leaves the weights in flight.  No dequantisation: the scaled FP4 MFMA takes
// the codes and the E8M0 bytes as they are.
//
// The weights are the MFMA's first operand, so a lane ends with four
// consecutive columns of one row: four bf16 outputs are one store, and an
// MXFP4 block lies in the registers of 4 lanes of two waves.
#include "../block/epilogue.h"
#include "experts.h"
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

template <int BM_, bool GATED_>
struct StreamCfg {
  static constexpr int BM = BM_, TM = BM / 16, TN = 2;
  static constexpr bool kGated = GATED_;
  static constexpr int kWaves = 4, kThreads = 64 * kWaves;
  static constexpr int kD = 4;                     // units in flight a wave, units of a chunk
  static constexpr int kCols = GATED_ ? 64 : 128;  // output columns of a work-group
  static constexpr int kBRows = 128;               // weight rows of a work-group
  static constexpr int kPieces = BM / 8;           // 16-byte pieces of A a thread stages
  static constexpr int kASf = (BM * 4 + kThreads - 1) / kThreads;  // 8-byte pieces of A's scales
  static constexpr int kASRows = kASf * kThreads / 4;  // rows that those cover (no branch around the last)
  static constexpr int kBSf = kBRows * 4 / kThreads;
};

template <class C>
struct StreamSmem {
  // [row][32 pieces of 16 bytes], piece p of row r at slot p ^ (r & 15)
  uint8_t a[2][C::BM * 512];
  uint8_t asf[2][C::kASRows * 32], bsf[2][C::kBRows * 32];
  uint32_t peak[C::kWaves][C::BM];
};

template <class C>
struct Staged {
  u4_t a[C::kPieces];
  u2_t as[C::kASf], bs[C::kBSf];
};

constexpr uint32_t kOutside = 0x80000000u;

// LDS accesses of this wave done, then a work-group barrier; loads in flight
// are left alone.
__device__ __forceinline__ void stage_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <class C>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_mx_grouped(MxGroupedLaunch p) {
  typedef int v8i_t __attribute__((ext_vector_type(8)));
  __shared__ __attribute__((aligned(16))) StreamSmem<C> sm;
  const int64_t cols = C::kGated ? p.N / 2 : p.N;
  const int tiles_n = (int)((cols + C::kCols - 1) / C::kCols);
  const int L = xcd_remap(blockIdx.x, tiles_n * p.E);
  const int e = L / tiles_n;
  const int64_t n0 = (int64_t)(L % tiles_n) * C::kCols;
  const int64_t lo = p.offsets[e], hi = p.offsets[e + 1];
  if (lo < 0 || hi <= lo || hi > p.rows) return;  // empty or invalid expert
  const int64_t ld = p.K / 2, lds = p.K / 32;
  const int nu = (int)(p.K / 256), chunks = (nu + C::kD - 1) / C::kD;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int r_in = lane & 15, g = lane >> 4;
  const bool lo8 = (lane & 8) == 0;

  // weight rows: column block tn of wave w is rows 32 w + 16 tn .. of the tile,
  // or (gated) rows 16 w .. of the tile in matrix tn
  const int valid = (int)min<int64_t>(C::kCols, cols - n0);  // columns of the tile
  const uint8_t* b0 = p.b + ((int64_t)e * p.N + n0) * ld;
  const uint8_t* s0 = p.b_sf + ((int64_t)e * p.N + n0) * lds;
  const int64_t second = C::kGated ? p.N / 2 : 0;  // rows from the first matrix to the second
  const rsrc_t rb[2] = {make_rsrc(b0, (uint32_t)(valid * ld)), make_rsrc(b0 + second * ld, (uint32_t)(valid * ld))};
  const rsrc_t rs[2] = {make_rsrc(s0, (uint32_t)(valid * lds)), make_rsrc(s0 + second * lds, (uint32_t)(valid * lds))};
  uint32_t vb[C::TN][2];
#pragma unroll
  for (int tn = 0; tn < C::TN; ++tn)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (C::kGated ? 16 * wave : 32 * wave + 16 * tn) + 8 * h + (lane & 7);
      vb[tn][h] = r < valid ? (uint32_t)(r * ld + 16 * (lane >> 3)) : kOutside;
    }
  // 8-byte pieces of the weights' scales: row id / 4 of the tile's LDS order
  // (wave, block, row), unit id % 4 of the chunk
  uint32_t vbs[C::kBSf];
  const int su = tid & 3;
#pragma unroll
  for (int i = 0; i < C::kBSf; ++i) {
    const int row = (tid >> 2) + i * (C::kThreads / 4);
    const int w = row >> 5, tn = (row >> 4) & 1, r = row & 15;
    const int at = C::kGated ? 16 * w + r : 32 * w + 16 * tn + r;
    vbs[i] = at < valid ? (uint32_t)(at * lds + 8 * su) : kOutside;
  }
  const bool odd_block = C::kGated && ((tid >> 6) & 1);  // the piece's matrix: rows 16 .. 31 of a wave's 32

#pragma unroll 1
  for (int64_t mc = lo; mc < hi; mc += C::BM) {
    const int rows_c = (int)min<int64_t>(C::BM, hi - mc);
    rsrc_t ra, ras;
    if (p.row_token) {
      ra = make_rsrc(p.a, (uint32_t)(p.T * ld));
      ras = make_rsrc(p.a_sf, (uint32_t)(p.T * lds));
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
      const int64_t t = source((tid >> 5) + 8 * i);
      va[i] = t >= 0 ? (uint32_t)(t * ld + 16 * (tid & 31)) : kOutside;
    }
#pragma unroll
    for (int i = 0; i < C::kASf; ++i) {
      const int r = (tid >> 2) + i * (C::kThreads / 4);
      const int64_t t = r < C::BM ? source(r) : -1;
      vas[i] = t >= 0 ? (uint32_t)(t * lds + 8 * su) : kOutside;
    }

    Staged<C> st;
    u4_t bq[C::kD][C::TN][2];
    Mfma<16>::Acc acc[C::TM][C::TN];
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) acc[tm][tn] = Mfma<16>::Acc{0.f, 0.f, 0.f, 0.f};

    // units past the end of K read out of range: zero codes and scales
    const auto stage_load = [&](int c) {
      const bool piece = C::kD * c + ((tid & 31) >> 3) < nu, scale = C::kD * c + su < nu;
#pragma unroll
      for (int i = 0; i < C::kPieces; ++i)
        st.a[i] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, piece ? va[i] : kOutside, c * 512, 0));
#pragma unroll
      for (int i = 0; i < C::kASf; ++i)
        st.as[i] = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(ras, scale ? vas[i] : kOutside, c * 32, 0));
#pragma unroll
      for (int i = 0; i < C::kBSf; ++i) {
        const uint32_t off = scale ? vbs[i] : kOutside;
        if constexpr (C::kGated) {
          // a quarter wave's rows are of one matrix: each lane loads from its own
          const u2_t x = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs[0], odd_block ? kOutside : off, c * 32, 0));
          const u2_t y = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs[1], odd_block ? off : kOutside, c * 32, 0));
          st.bs[i] = odd_block ? y : x;
        } else {
          st.bs[i] = __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(rs[0], off, c * 32, 0));
        }
      }
    };
    const auto stage_store = [&](int buf) {
#pragma unroll
      for (int i = 0; i < C::kPieces; ++i) {
        const int r = (tid >> 5) + 8 * i;
        *(u4_t*)(sm.a[buf] + r * 512 + (((tid & 31) ^ (r & 15)) << 4)) = st.a[i];
      }
#pragma unroll
      for (int i = 0; i < C::kASf; ++i) {
        const int r = (tid >> 2) + i * (C::kThreads / 4);
        *(u2_t*)(sm.asf[buf] + r * 32 + 8 * su) = st.as[i];
      }
#pragma unroll
      for (int i = 0; i < C::kBSf; ++i) {
        const int r = (tid >> 2) + i * (C::kThreads / 4);
        *(u2_t*)(sm.bsf[buf] + r * 32 + 8 * su) = st.bs[i];
      }
    };
    const auto unit_load = [&](int u, int unit) {
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          bq[u][tn][h] = __builtin_bit_cast(
              u4_t, __builtin_amdgcn_raw_buffer_load_b128(rb[C::kGated ? tn : 0], unit < nu ? vb[tn][h] : kOutside, unit * 128, 0));
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
        sb[tn] = *(const uint16_t*)(sm.bsf[buf] + (wave * 32 + tn * 16 + r_in) * 32 + 8 * u + 2 * g);
      }
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
        const int row = tm * 16 + r_in;
        const int sa = *(const uint16_t*)(sm.asf[buf] + row * 32 + 8 * u + 2 * g);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u4_t x = *(const u4_t*)(sm.a[buf] + row * 512 + (((8 * u + 2 * g + c) ^ r_in) << 4));
          const v8i_t av = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
#pragma unroll
          for (int tn = 0; tn < C::TN; ++tn)
            acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[tn][c], av, acc[tm][tn], 4, 4, 0,
                                                                           sb[tn] >> (8 * c), 0, sa >> (8 * c));
        }
      }
    };

    stage_load(0);
#pragma unroll
    for (int u = 0; u < C::kD; ++u) {
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
      for (int u = 0; u < C::kD; ++u) {
        unit_compute(c & 1, u);
        // the slot's reload stays behind its last reads
        __builtin_amdgcn_sched_barrier(0);
        unit_load(u, C::kD * (c + 1) + u);
      }
      stage_store((c + 1) & 1);
      stage_barrier();
    }

    // lane: row r_in of each row block, columns 4 g .. 4 g + 3 of each column block
    if constexpr (C::kGated) {
      const float a0 = p.alpha ? p.alpha[2 * e] : 1.0f, a1 = p.alpha ? p.alpha[2 * e + 1] : 1.0f;
      const int col = 16 * wave + 4 * g;
      const bool in = col < valid;  // blocks of 32 are whole
      const int64_t I = cols;
      float h[C::TM][4];
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
        float u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[tm][j] = a0 * acc[tm][0][j];
          u[j] = a1 * acc[tm][1][j];
        }
        if (p.bias && in) {
          const uint16_t* bg = p.bias + (int64_t)e * p.N + n0 + col;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[tm][j] += __uint_as_float((uint32_t)bg[j] << 16);
            u[j] += __uint_as_float((uint32_t)bg[I + j] << 16);
          }
        }
        activate<4>(h[tm], p.act);
        uint32_t peak = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[tm][j] *= u[j];
          peak = umax(peak, magnitude(h[tm][j]));
        }
        peak = umax(peak, (uint32_t)__shfl_xor((int)peak, 16));
        peak = umax(peak, (uint32_t)__shfl_xor((int)peak, 32));
        if (g == 0) sm.peak[wave][tm * 16 + r_in] = peak;
      }
      __syncthreads();
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
        const int row = tm * 16 + r_in;
        const MxScale s = mx_scale(umax(sm.peak[wave][row], sm.peak[wave ^ 1][row]), p.rule);
        uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h[tm][0] * s.r, h[tm][1] * s.r, 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, h[tm][2] * s.r, h[tm][3] * s.r, 1.0f, 1);
        if (row < rows_c && in) {
          const int64_t r = mc + row, n = n0 + col;
          *(uint16_t*)(p.q + r * (I / 2) + n / 2) = (uint16_t)(w & s.keep);
          if (g == 0 && (wave & 1) == 0) p.sf[r * (I / 32) + n / 32] = (uint8_t)s.byte;
        }
      }
      __syncthreads();  // the next rows' peaks
    } else {
      const float alpha = p.alpha ? p.alpha[e] : 1.0f;
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) {
        const int col = 32 * wave + 16 * tn + 4 * g;
        if (col >= valid) continue;
        const int n = min(4, valid - col);
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias)
          for (int j = 0; j < 4; ++j)
            if (j < n) b[j] = __uint_as_float((uint32_t)p.bias[(int64_t)e * p.N + n0 + col + j] << 16);
#pragma unroll
        for (int tm = 0; tm < C::TM; ++tm) {
          const int row = tm * 16 + r_in;
          if (row >= rows_c) continue;
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = p.bias ? alpha * acc[tm][tn][j] + b[j] : alpha * acc[tm][tn][j];
          const u2_t w = {f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3])};
          uint16_t* out = p.d + (mc + row) * p.N + n0 + col;
          if (n == 4) *(u2_any_t*)out = w;
          else
            for (int j = 0; j < n; ++j) out[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  }
}

template <int BM, bool GATED>
static void launch_stream(const MxGroupedLaunch& p, hipStream_t stream) {
  typedef StreamCfg<BM, GATED> C;
  const int64_t cols = GATED ? p.N / 2 : p.N;
  const unsigned grid = (unsigned)((cols + C::kCols - 1) / C::kCols) * (unsigned)p.E;
  hipLaunchKernelGGL(k_mx_grouped<C>, dim3(grid), dim3(C::kThreads), 0, stream, p);
}

template <bool GATED>
static void launch_rows(const MxGroupedLaunch& p, hipStream_t stream) {
  // the host knows the average rows of an expert only
  if (p.rows <= 4 * (int64_t)p.E) launch_stream<16, GATED>(p, stream);
  else if (p.rows <= 24 * (int64_t)p.E) launch_stream<32, GATED>(p, stream);
  else launch_stream<64, GATED>(p, stream);
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
