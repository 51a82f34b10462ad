// Row order of a mixture-of-experts layer: a stable counting sort of the
// chosen experts ids[T][top_k] (i = t top_k + j):
//   offsets[e] = number of ids below expert e, offsets[E] = number of valid ids
//   row(i)     = offsets[id(i)] + number of i' < i with the same id
//   row_token[row(i)] = t, token_rows[i] = row(i) (-1: id outside the range)
// No atomics on memory and no order that depends on timing: the same rows every
// time.
//
// Few ids (k_sort_few): one work-group an expert.  Every work-group counts the
// ids below its own and its own in a first pass over all ids, which gives its
// first row without a word from the others, and places its own in a second: one
// launch, no workspace, but every CU reads all ids twice.
//
// Many ids, up to 1024 experts: the ids are cut into runs, one a wave.
// k_sort_count writes each run's number of ids of each expert; k_sort_place,
// which has 16 runs a work-group, adds up the counts of all runs before its own
// and of all experts, and every wave goes through its run 64 ids at a time: the
// lanes that hold the same expert are found by comparing the bits of the ids in
// ballots, and the first of them moves the expert's next row on.
#include "experts.h"
#include "mx_block.h"

namespace nvfp4 {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int below(uint64_t mask, int lane) { return __popcll(mask & ((1ull << lane) - 1)); }

// Four consecutive ids from i as expert numbers; those at n and beyond are
// none.  32-bit wrap-around: an id below `first` becomes a large number.
__device__ __forceinline__ void four_ids(const SortLaunch& p, int64_t i, int64_t n, uint32_t (&id)[4]) {
  typedef uint32_t any4_t __attribute__((ext_vector_type(4), aligned(4)));
  if (i + 4 <= n) {
    const any4_t v = *(const any4_t*)(p.ids + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = v[j] - (uint32_t)p.first;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = i + j < n ? (uint32_t)p.ids[i + j] - (uint32_t)p.first : 0xFFFFFFFFu;
  }
}

// Each wave takes one contiguous run of the ids, 256 at a time.
__global__ __launch_bounds__(kSortThreads) void k_sort_few(SortLaunch p) {
  __shared__ int own[kSortWaves], low[kSortWaves], top[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t e = blockIdx.x, E = (uint32_t)p.E;
  const int64_t per = ((p.n + kSortWaves - 1) / kSortWaves + 255) / 256 * 256;
  const int64_t lo = min(wave * per, p.n), hi = min(lo + per, p.n);
  int mine = 0, less = 0, all = 0;
  for (int64_t i = lo + 4 * lane; i < hi; i += 256) {
    uint32_t id[4];
    four_ids(p, i, hi, id);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mine += id[j] == e;
      less += id[j] < e;
      all += id[j] < E;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    mine += __shfl_xor(mine, o);
    less += __shfl_xor(less, o);
    all += __shfl_xor(all, o);
  }
  if (lane == 0) {
    own[wave] = mine;
    low[wave] = less;
    top[wave] = all;
  }
  __syncthreads();
  int row = 0, valid = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    row += low[w];
    valid += top[w];
  }
  if (threadIdx.x == 0) {
    p.offsets[e] = row;
    if (e == 0) p.offsets[p.E] = valid;
  }
  for (int w = 0; w < wave; ++w) row += own[w];
  if (mine == 0 && e != 0) return;
  for (int64_t i0 = lo; i0 < hi; i0 += 256) {
    const int64_t i = i0 + 4 * lane;
    uint32_t id[4];
    four_ids(p, i, hi, id);
    int hits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) hits += id[j] == e;
    if (e == 0) {  // the ids left out
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < hi && id[j] >= E) p.token_rows[i + j] = -1;
    }
    // hits of the lanes before, from the bits of their numbers
    const uint64_t b0 = __ballot(hits & 1), b1 = __ballot(hits & 2), b2 = __ballot(hits & 4);
    int at = row + below(b0, lane) + 2 * below(b1, lane) + 4 * below(b2, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id[j] == e) {
        p.row_token[at] = (int32_t)((uint32_t)(i + j) / (uint32_t)p.top_k);
        p.token_rows[i + j] = at++;
      }
    row += __popcll(b0) + 2 * __popcll(b1) + 4 * __popcll(b2);
  }
}

// Runs: 512 ids or more each, 1024 of them where that keeps them below 2^15 ids
// (their counts are 16-bit).
struct SortRuns {
  int runs;
  int64_t per;
};
constexpr int kManyRuns = 1024;
constexpr int kAhead = 8;  // steps of 64 ids that a wave loads at once
static SortRuns sort_runs(int64_t n) {
  SortRuns r;
  r.per = (n + kManyRuns - 1) / kManyRuns;
  r.per = r.per < 512 ? 512 : r.per > 32768 ? 32768 : (r.per + 63) / 64 * 64;
  r.runs = (int)((n + r.per - 1) / r.per);
  return r;
}

// EP: the number of experts rounded up to a power of two.
template <int EP>
__global__ __launch_bounds__(256) void k_sort_count(SortLaunch p, int runs, int64_t per) {
  __shared__ int count[4][EP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, run = blockIdx.x * 4 + wave;
  for (int e = lane; e < EP; e += 64) count[wave][e] = 0;
  __builtin_amdgcn_wave_barrier();
  const int64_t lo = min(run * per, p.n), hi = min(lo + per, p.n);
  for (int64_t i = lo + 4 * lane; i < hi; i += 256) {
    uint32_t id[4];
    four_ids(p, i, hi, id);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id[j] < (uint32_t)p.E) atomicAdd(&count[wave][id[j]], 1);
  }
  __builtin_amdgcn_wave_barrier();
  if (run < runs)
    for (int e = lane; e < p.E; e += 64) p.ws[(int64_t)run * p.E + e] = (uint16_t)count[wave][e];
}

template <int EP>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortLaunch p, int runs, int64_t per) {
  __shared__ int next[kSortWaves][EP];  // an expert's next row, for each run of the work-group
  __shared__ int total[kSortThreads], before[kSortThreads], sums[kSortWaves];
  constexpr int kParts = kSortThreads / EP;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = tid % EP, part = tid / EP, first = blockIdx.x * kSortWaves;  // first run
  // ids of expert e in a part of the runs, and in those before the work-group's
  int all = 0, mine = 0;
  if (e < p.E) {
    const int u1 = (part + 1) * runs / kParts;
#pragma unroll 16
    for (int u = part * runs / kParts; u < u1; ++u) {
      const int c = p.ws[(int64_t)u * p.E + e];
      all += c;
      mine += u < first ? c : 0;
    }
  }
  int own[kSortWaves];  // of the work-group's runs
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) own[w] = tid < p.E && first + w < runs ? p.ws[(int64_t)(first + w) * p.E + e] : 0;
  total[tid] = all;
  before[tid] = mine;
  __syncthreads();
  if (tid < EP) {
    for (int q = 1; q < kParts; ++q) {
      all += total[q * EP + e];
      mine += before[q * EP + e];
    }
  } else {
    all = 0;
  }
  // rows of the experts before
  int upto = all;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int row = upto - all;
  for (int w = 0; w < wave; ++w) row += sums[w];
  if (tid < p.E) {
    if (blockIdx.x == 0) {
      p.offsets[e] = row;
      if (e == p.E - 1) p.offsets[p.E] = row + all;
    }
    row += mine;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      next[w][e] = row;
      row += own[w];
    }
  }
  __syncthreads();
  const int64_t lo = min((int64_t)(first + wave) * per, p.n), hi = min(lo + per, p.n);
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kAhead) {
    uint32_t ids[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t i = i0 + 64 * a + lane;
      ids[a] = i < hi ? (uint32_t)p.ids[i] - (uint32_t)p.first : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t i = i0 + 64 * a + lane;
      const uint32_t id = ids[a];
      const bool in = id < (uint32_t)p.E;
      uint64_t same = __ballot(in);  // lanes with this lane's expert
#pragma unroll
      for (int b = 1; b < EP; b *= 2) {
        const uint64_t set = __ballot(id & b);
        same &= id & b ? set : ~set;
      }
      if (in) {
        const int at = next[wave][id], rank = below(same, lane), number = __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (rank == 0) next[wave][id] = at + number;
        p.row_token[at + rank] = (int32_t)((uint32_t)i / (uint32_t)p.top_k);
        p.token_rows[i] = at + rank;
      } else if (i < hi) {
        p.token_rows[i] = -1;
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Whether the second form is taken.  256 experts, us by the first and the second
// form: 8192 ids 5.1 and 12.6, 32768 ids 11.0 and 13.3, 49152 ids 15.1 and 15.8, 65536
// ids 19.7 and 14.6, 131072 ids 36.8 and 17.1, a million 288 and 40.  At 40960 ids, 16
// experts 17.4 and 11.7, 64 15.4 and 12.4, 128 14.2 and 14.4, 512 18.5 and 16.3, 1024
// 31.6 and 18.1: the border is that of 128 to 256 experts, others meet earlier (16 at
// 24576 ids, 512 at 32768, 1024 at 16384).
static bool many_ids(int64_t n, int E) { return n > 40960 && E <= kMostSorted; }

size_t moe_sort_workspace(int64_t n, int E) {
  return many_ids(n, E) ? (size_t)sort_runs(n).runs * (size_t)E * sizeof(uint16_t) : 0;
}

template <int EP>
static hipError_t sort_many(const SortLaunch& p, hipStream_t stream) {
  const SortRuns r = sort_runs(p.n);
  hipLaunchKernelGGL(k_sort_count<EP>, dim3((unsigned)((r.runs + 3) / 4)), dim3(256), 0, stream, p, r.runs, r.per);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_sort_place<EP>, dim3((unsigned)((r.runs + kSortWaves - 1) / kSortWaves)),
                     dim3(kSortThreads), 0, stream, p, r.runs, r.per);
  return hipGetLastError();
}

hipError_t launch_moe_sort(const SortLaunch& p, hipStream_t stream) {
  if (many_ids(p.n, p.E)) {
    if (p.E <= 64) return sort_many<64>(p, stream);
    if (p.E <= 256) return sort_many<256>(p, stream);
    return sort_many<1024>(p, stream);
  }
  hipLaunchKernelGGL(k_sort_few, dim3((unsigned)p.E), dim3(kSortThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
