// The norms before and after a block, fused with its gate and residual:
//
//   u = post(x)                      post(x) = norm of x with post_w, post_b; or x
//   r = beta res + gate u            gate: one row for all, or one per gate_group rows; or 1
//   y = norm(r) with w, b            to bf16 and / or NVFP4
//
//   norm(v) = (v - m) rstd w + b,  rstd = 1 / sqrt(mean((v - m)^2) + eps),
//   m = mean(v) (layer norm) or 0 (RMS norm)
//
// One pass over memory: a row's chunks of 8 columns stay in the registers of
// the threads that own them from the first load to the last store, so x and
// res are read once and r, y written once.  Bound by HBM for long inputs and by one
// memory round trip plus the launch for a few rows.
//
// Arithmetic: the sums of a row (mean, mean square) and rstd are in fp64 and
// rstd is rounded once to fp32, which makes it independent of the order of
// the sum to within one rounding in 2^29; everything else is fp32, one
// rounding per step in the formulas' order (r is not rounded to bf16 before
// the second norm).  Built without fp contraction, so a plain evaluation of
// the same steps gives the same bits, the NVFP4 codes and scales among them.
// The fp64 sums cost an RMS norm two instructions an element (a conversion and
// a fused multiply-add), far below the memory time; a layer norm also adds for
// its mean and subtracts it before the square and again, with a conversion, in
// its output, which a call of a few hundred rows waits for as well.
#include "block.h"
#include "quantize_block.h"
#include "vec8.h"

namespace nvfp4 {

// The columns of a row's TPR threads: thread tid holds chunks tid, TPR + tid,
// ... of 8 columns, one 16-byte access each whatever the row's alignment.
// When H is no multiple of 8 the last chunk is either
//  * kOverlap (H >= 8): moved back to the row's last 8 columns, so that no
//    access is shorter (a branch around one would make its wave wait for each
//    operand's load in turn: one row of 1545 columns 5.2 us against 3.6 for
//    1544).  The columns it shares with the chunk before are computed twice,
//    to the same bits, and counted once; nothing may be stored before every
//    thread of the row has loaded;
//  * kShort: loaded and stored in shorter pieces.
enum Tail { kNone, kOverlap, kShort };

template <int TPR, int TAIL>
struct Columns {
  int tid, H;
  // columns of chunk i before its start is moved back, and the columns it is moved by
  __device__ __forceinline__ int first(int i) const { return (i * TPR + tid) * 8; }
  __device__ __forceinline__ int shared(int i) const { return TAIL == kOverlap ? max(first(i) - (H - 8), 0) : 0; }
  __device__ __forceinline__ int col(int i) const { return first(i) - shared(i); }
  __device__ __forceinline__ bool any(int i) const { return first(i) < H; }
  // whether element e of chunk i counts in the row's sums
  __device__ __forceinline__ bool counts(int i, int e) const {
    if (TAIL == kOverlap) return any(i) && e >= shared(i);
    return first(i) + (TAIL == kShort ? e : 0) < H;
  }
  // f(e, whether element e counts) for the elements of chunk i.  Rows of whole
  // chunks skip absent ones with one test (layer norms before and after, 8192 x
  // 4096: 50.7 us against 52.3 with a select an element; 4096 x 16384: 140 against
  // 149); where a row ends inside a chunk the selects are faster (777 x 1545: 6.3
  // against 6.6).
  template <class F>
  __device__ __forceinline__ void each(int i, F&& f) const {
    if (TAIL == kNone && !any(i)) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) f(e, TAIL == kNone || counts(i, e));
  }
  // chunk i of a row or vector as packed bf16; columns past H are 0
  __device__ __forceinline__ u4_t load(const uint16_t* row, int i) const {
    if (TAIL == kShort && any(i) && first(i) + 8 > H) return load_tail8(row + first(i), H & 7);
    return any(i) ? load8(row + col(i)) : u4_t{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void store(uint16_t* row, int i, const float (&v)[8]) const {
    if (TAIL == kShort && any(i) && first(i) + 8 > H) store_tail8(row + first(i), to_bf16x8(v), H & 7);
    else if (any(i)) store8(row + col(i), to_bf16x8(v));
  }
};

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// v + its value in the neighbouring group of 16 or 32 lanes: a swap of a value
// with itself leaves both groups' values in every lane.
__device__ __forceinline__ double join(u2_t lo, u2_t hi) {
  return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) +
         __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
}
__device__ __forceinline__ double add_swap16(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  return join(__builtin_bit_cast(u2_t, __builtin_amdgcn_permlane16_swap(lo, lo, false, false)),
              __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane16_swap(hi, hi, false, false)));
}
__device__ __forceinline__ double add_swap32(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  return join(__builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(lo, lo, false, false)),
              __builtin_bit_cast(u2_t, __builtin_amdgcn_permlane32_swap(hi, hi, false, false)));
}

// Sum over the TPR threads of a row, in a fixed order, to all of them.  Every
// step adds a lane's value and its partner's, so all lanes get the same bits.
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* cell) {
  v = dpp_add<0xB1>(v);   // lane ^ 1
  v = dpp_add<0x4E>(v);   // lane ^ 2
  v = dpp_add<0x141>(v);  // mirror of 8 lanes
  v = dpp_add<0x140>(v);  // mirror of 16 lanes
  v = add_swap16(v);
  v = add_swap32(v);
  if constexpr (TPR > 64) {
    __syncthreads();  // the cells' last readers are done
    if ((threadIdx.x & 63) == 0) cell[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += cell[w];
  }
  return v;
}

// mean (0 for RMS) and rstd of one row
struct Stats {
  double mean;
  float rstd;
};

// 1 / sqrt(ms + eps), in fp64 rounded once to fp32: the hardware estimate and
// two Newton steps (each at least doubles its 23 bits), a quarter of the
// latency of a square root and a division.  An infinite sum gives 0.
__device__ __forceinline__ float rstd_of(double ms, float eps) {
  const double v = ms + (double)eps;
  const double y0 = __builtin_amdgcn_rsq(v);
  const double h = 0.5 * v;
  double y = y0 * __builtin_fma(-h * y0, y0, 1.5);
  y = y * __builtin_fma(-h * y, y, 1.5);
  return (float)(v < 1e300 && v > 1e-300 ? y : y0);
}

// Absent vectors stand for values that change no bit: weights and gates of 1,
// biases of -0.
constexpr uint32_t kOnes = 0x3F803F80u, kMinusZeros = 0x80008000u;

template <bool LAYER>
__device__ __forceinline__ float normed(float v, const Stats& s, float w, float b) {
  return (LAYER ? (float)((double)v - s.mean) : v) * s.rstd * w + b;
}

template <class C>
__device__ __forceinline__ u4_t load_or(const C& at, const uint16_t* row, int i, uint32_t absent) {
  return row ? at.load(row, i) : u4_t{absent, absent, absent, absent};
}

// Statistics of a row held as V chunks of 8 per thread.
template <int TPR, int V, int TAIL, bool LAYER>
__device__ __forceinline__ Stats row_stats(const float (&v)[V][8], const Columns<TPR, TAIL>& at, const NormLaunch& p,
                                           double* cell) {
  Stats s{0.0, 0.0f};
  if constexpr (LAYER) {
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) at.each(i, [&](int e, bool in) { a += in ? (double)v[i][e] : 0.0; });
    s.mean = row_sum<TPR>(a, cell) * p.inv_h;
  }
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    at.each(i, [&](int e, bool in) {
      const double d = in ? (LAYER ? (double)v[i][e] - s.mean : (double)v[i][e]) : 0.0;
      q = __builtin_fma(d, d, q);
    });
  s.rstd = rstd_of(row_sum<TPR>(q, cell) * p.inv_h, p.eps);
  return s;
}

// y of one chunk, to bf16 and NVFP4
template <int TPR, int TAIL>
__device__ __forceinline__ void store_y(const NormLaunch& p, const Columns<TPR, TAIL>& at, int64_t t, int i,
                                        const float (&y)[8], float gs) {
  if (p.y) at.store(p.y + t * p.ldy, i, y);
  if constexpr (TAIL == kNone) {
    const int c = at.col(i);
    if (p.q && c < at.H) {
      // H % 16 == 0: the lanes of a pair hold the two halves of a block
      uint32_t codes;
      const uint32_t sf = quantize_pair16(f4_t{y[0], y[1], y[2], y[3]}, f4_t{y[4], y[5], y[6], y[7]}, gs, codes);
      *(uint32_t*)(p.q + t * (p.H / 2) + c / 2) = codes;
      if (c % 16 == 0) p.sf[t * (p.H / 16) + c / 16] = (uint8_t)sf;
    }
  }
}

// The vectors (weights, biases, gate) are loaded where they are used, not with
// the row: they come from L2, and the registers they would hold cost rows in
// flight per CU, which are what hides the sums' barriers (16384 x 6144 with
// both norms and a gate: 164 us against 225 with every load issued first; a
// single row was not slower either).  Layer and RMS norms are kernels of their
// own for the same reason: 84 registers instead of 130 at 256 x 3, 151 us (5.3
// TB/s, what a copy of the same bytes takes).
template <int TPR>
constexpr int kRowsPerGroup = TPR == 64 ? 4 : 1;  // rows of one work-group

template <int TPR, int V, int TAIL, bool LAYER>
__global__ __launch_bounds__(TPR * kRowsPerGroup<TPR>) void k_residual_norm(NormLaunch p) {
  __shared__ double cell[TPR / 64];
  const int64_t t = p.t0 + (int64_t)blockIdx.x * kRowsPerGroup<TPR> + threadIdx.x / TPR;
  if (t >= p.T) return;  // whole waves: a row has 64 threads, or the work-group
  const Columns<TPR, TAIL> at{(int)threadIdx.x % TPR, (int)p.H};
  const uint16_t* gate = p.gate ? p.gate + (p.gate_group > 0 ? t / p.gate_group : 0) * p.H : nullptr;
  u4_t x[V], res[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = at.load(p.x + t * p.ldx, i);
    if (p.res) res[i] = at.load(p.res + t * p.ldres, i);
  }
  float v[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = bf16_at(x[i], e);
  if (p.post_w) {
    const Stats s = row_stats<TPR, V, TAIL, LAYER>(v, at, p, cell);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const u4_t w = at.load(p.post_w, i), b = load_or(at, p.post_b, i, kMinusZeros);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = normed<LAYER>(v[i][e], s, bf16_at(w, e), bf16_at(b, e));
    }
  }
  if (gate) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const u4_t g = at.load(gate, i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = bf16_at(g, e) * v[i][e];
    }
  }
  if (p.res) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = p.beta * bf16_at(res[i], e) + v[i][e];
  }
  const bool norm = p.y || p.q;
  if (TAIL == kOverlap && TPR > 64) __syncthreads();  // the whole row is loaded: r may be x or res
  if (p.r) {
#pragma unroll
    for (int i = 0; i < V; ++i) at.store(p.r + t * p.ldr, i, v[i]);
  }
  if (!norm) return;
  const Stats s = row_stats<TPR, V, TAIL, LAYER>(v, at, p, cell);
  const float gs = p.q && p.gs ? *p.gs : 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const u4_t w = load_or(at, p.w, i, kOnes), b = load_or(at, p.b, i, kMinusZeros);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = normed<LAYER>(v[i][e], s, bf16_at(w, e), bf16_at(b, e));
    store_y(p, at, t, i, v[i], gs);
  }
}

// Rows too long for the registers: the same steps with the row read again for
// each sum, one work-group per row.  A thread stores only columns it reads,
// after its last read of them, so r may be x or res here too.  A residual and an
// RMS norm read both inputs twice, mostly from cache the second time (1000 x
// 20480: 40 us, 4.1 TB/s of the four arrays; 1000 x 32768 65 us); with layer norms
// before and after, x is read five times and the residual three (74 and 111 us).
// The widest rows that registers hold, 1000 x 16384: 27 and 38 us.
template <int TAIL, bool LAYER>
__global__ __launch_bounds__(1024) void k_residual_norm_long(NormLaunch p) {
  constexpr int TPR = 1024;
  __shared__ double cell[TPR / 64];
  const int64_t t = p.t0 + blockIdx.x, H = p.H;
  const Columns<TPR, TAIL> at{(int)threadIdx.x, (int)H};
  const uint16_t* gate = p.gate ? p.gate + (p.gate_group > 0 ? t / p.gate_group : 0) * H : nullptr;
  const int n = (int)((H + 8 * TPR - 1) / (8 * TPR));
  Stats sx{0.0, 0.0f}, sr{0.0, 0.0f};
  auto x_chunk = [&](int i, float (&v)[8]) {
    const u4_t x = at.load(p.x + t * p.ldx, i);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bf16_at(x, e);
  };
  auto r_chunk = [&](int i, float (&v)[8]) {
    const u4_t res = load_or(at, p.res ? p.res + t * p.ldres : nullptr, i, 0u);
    x_chunk(i, v);
    if (p.post_w) {
      const u4_t w = at.load(p.post_w, i), b = load_or(at, p.post_b, i, kMinusZeros);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = normed<LAYER>(v[e], sx, bf16_at(w, e), bf16_at(b, e));
    }
    const u4_t g = load_or(at, gate, i, kOnes);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = bf16_at(g, e) * v[e];
      if (p.res) v[e] = p.beta * bf16_at(res, e) + v[e];
    }
  };
  auto stats = [&](auto&& chunk) {
    Stats s{0.0, 0.0f};
    float v[8];
    if constexpr (LAYER) {
      double a = 0.0;
      for (int i = 0; i < n; ++i) {
        chunk(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at.counts(i, e)) a += (double)v[e];
      }
      s.mean = row_sum<TPR>(a, cell) * p.inv_h;
    }
    double q = 0.0;
    for (int i = 0; i < n; ++i) {
      chunk(i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double d = (double)v[e] - s.mean;
        if (at.counts(i, e)) q = __builtin_fma(d, d, q);
      }
    }
    s.rstd = rstd_of(row_sum<TPR>(q, cell) * p.inv_h, p.eps);
    return s;
  };
  const bool norm = p.y || p.q;
  if (p.post_w) sx = stats(x_chunk);
  if (norm) sr = stats(r_chunk);
  const float gs = p.q && p.gs ? *p.gs : 1.0f;
  for (int i = 0; i < n; ++i) {
    float v[8];
    r_chunk(i, v);
    if (p.r) at.store(p.r + t * p.ldr, i, v);
    if (!norm) continue;
    const u4_t w = load_or(at, p.w, i, kOnes), b = load_or(at, p.b, i, kMinusZeros);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = normed<LAYER>(v[e], sr, bf16_at(w, e), bf16_at(b, e));
    store_y(p, at, t, i, v, gs);
  }
}

// Rows of one launch: a launch has fewer than 2^32 threads.
static constexpr int64_t kLaunchRows = int64_t(1) << 21;
static int64_t launch_rows(const NormLaunch& p) { return p.T - p.t0 < kLaunchRows ? p.T - p.t0 : kLaunchRows; }

template <int TPR, int V, bool LAYER>
static void launch_norm_as(const NormLaunch& p, hipStream_t stream) {
  constexpr int R = kRowsPerGroup<TPR>;
  const dim3 grid((unsigned)((launch_rows(p) + R - 1) / R)), block(TPR * R);
  if (p.H % 8 == 0) hipLaunchKernelGGL((k_residual_norm<TPR, V, kNone, LAYER>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((k_residual_norm<TPR, V, kOverlap, LAYER>), grid, block, 0, stream, p);
}

template <int TPR, int V>
static void launch_norm(const NormLaunch& p, hipStream_t stream) {
  if (p.layer) launch_norm_as<TPR, V, true>(p, stream);
  else launch_norm_as<TPR, V, false>(p, stream);
}

static void launch_norm_short(const NormLaunch& p, hipStream_t stream) {
  const dim3 grid((unsigned)((launch_rows(p) + 3) / 4)), block(256);
  if (p.layer) hipLaunchKernelGGL((k_residual_norm<64, 1, kShort, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((k_residual_norm<64, 1, kShort, false>), grid, block, 0, stream, p);
}

static void launch_norm_long(const NormLaunch& p, hipStream_t stream) {
  const dim3 grid((unsigned)launch_rows(p)), block(1024);
  const bool whole = p.H % 8 == 0;
  if (whole && p.layer) hipLaunchKernelGGL((k_residual_norm_long<kNone, true>), grid, block, 0, stream, p);
  else if (whole) hipLaunchKernelGGL((k_residual_norm_long<kNone, false>), grid, block, 0, stream, p);
  else if (p.layer) hipLaunchKernelGGL((k_residual_norm_long<kShort, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((k_residual_norm_long<kShort, false>), grid, block, 0, stream, p);
}

// Threads per row and chunks per thread.  Up to 2048 columns a chunk a thread
// is best at every number of rows, and up to 12288 two at most.  Where rows are
// many (more than two per CU) and both a wide and a narrow shape fit, the
// narrow one has more rows in flight per CU between the barriers of the sums
// (16276 rows of 6144, both norms and a gate: 256 x 3 151 us, 384 x 2 157, 768 x 1
// 164; 6103 of 16384: 512 x 4 160, 1024 x 2 176); where they are few the wide one
// is the shorter chain (one row of 6144: 768 x 1 2.85 us, 256 x 3 3.53).
static void launch_norm_rows(const NormLaunch& p, hipStream_t stream) {
  const int64_t n8 = (p.H + 7) / 8;
  const bool many = p.T > 2 * kCUs;
  if (n8 > 2048) launch_norm_long(p, stream);
  else if (p.H < 8) launch_norm_short(p, stream);
  else if (n8 <= 64) launch_norm<64, 1>(p, stream);
  else if (n8 <= 128) launch_norm<128, 1>(p, stream);
  else if (n8 <= 256) launch_norm<256, 1>(p, stream);
  else if (n8 <= 512) many ? launch_norm<256, 2>(p, stream) : launch_norm<512, 1>(p, stream);
  else if (n8 <= 768) many ? launch_norm<256, 3>(p, stream) : launch_norm<768, 1>(p, stream);
  else if (n8 <= 1024) launch_norm<512, 2>(p, stream);
  else if (n8 <= 1536) launch_norm<768, 2>(p, stream);
  else many ? launch_norm<512, 4>(p, stream) : launch_norm<1024, 2>(p, stream);
}

hipError_t launch_residual_norm(NormLaunch p, hipStream_t stream) {
  for (p.t0 = 0; p.t0 < p.T; p.t0 += kLaunchRows) launch_norm_rows(p, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
