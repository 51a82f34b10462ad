// Row order of a mixture-of-experts layer: a stable counting sort of the
// chosen experts ids[T][top_k] (i = t top_k + j):
//   offsets[e] = number of ids below expert e, offsets[E] = number of valid ids
//   row(i)     = offsets[id(i)] + number of i' < i with the same id
//   row_token[row(i)] = t, token_rows[i] = row(i) (-1: id outside the range)
//
// One work-group an expert: every work-group counts the ids below its own and
// its own in a first pass over all ids, which gives its first row without a
// word from the others, and places its own in a second.  No workspace, no
// atomics, one launch; each CU reads all ids twice.
#include "experts.h"
#include "mx_block.h"

namespace nvfp4 {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int below(uint64_t mask, int lane) { return __popcll(mask & ((1ull << lane) - 1)); }

// Each wave takes one contiguous run of the ids, 64 at a time.
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(SortLaunch p) {
  __shared__ int own[kSortWaves], low[kSortWaves], top[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
  const int64_t per = ((p.n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t lo = min(wave * per, p.n), hi = min(lo + per, p.n);
  int mine = 0, less = 0, all = 0;
  for (int64_t i = lo + lane; i < hi; i += 64) {
    // 32-bit wrap-around: an id below `first` becomes a large number
    const uint32_t id = (uint32_t)p.ids[i] - (uint32_t)p.first;
    mine += id == (uint32_t)e;
    less += id < (uint32_t)e;
    all += id < (uint32_t)p.E;
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
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const uint32_t id = i < hi ? (uint32_t)p.ids[i] - (uint32_t)p.first : 0xFFFFFFFFu;
    const bool hit = i < hi && id == (uint32_t)e;
    const uint64_t hits = __ballot(hit);
    if (hit) {
      const int at = row + below(hits, lane);
      p.row_token[at] = (int32_t)(i / p.top_k);
      p.token_rows[i] = at;
    }
    if (e == 0 && i < hi && id >= (uint32_t)p.E) p.token_rows[i] = -1;
    row += __popcll(hits);
  }
}

size_t moe_sort_workspace(int64_t, int) { return 0; }

hipError_t launch_moe_sort(const SortLaunch& p, hipStream_t stream) {
  hipLaunchKernelGGL(k_moe_sort, dim3((unsigned)p.E), dim3(kSortThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
