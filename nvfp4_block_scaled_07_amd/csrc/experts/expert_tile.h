// Row tiles of experts: which expert, and which of its rows, a work-group has
// when the rows of each expert are cut into tiles of BM.
#pragma once
#include "experts.h"

namespace nvfp4 {

struct ExpertTile {
  int expert;      // -1: no such tile
  int first;       // tiles of the experts before
  int tiles;       // of this expert
  int64_t lo, hi;  // its rows
};

// Most row tiles that `rows` rows of E experts have: every expert with rows may
// have one that is not full.
__host__ __device__ inline int64_t most_tiles(int64_t rows, int E, int bm) { return rows / bm + (rows < E ? rows : E); }

// The expert of row tile q, the same in all lanes.  Every wave finds it for
// itself: lane l counts the tiles of EPL consecutive experts (four at a time,
// whose offsets are loaded together), a prefix sum over the lanes follows, and
// the lane that holds q tells.  Experts whose offsets are wrong have no tiles.  Offsets
// that decrease can add up to any number of tiles: q is below most_tiles, which
// fits kMostTiles (the entry points see to it), and a lane's count stops there.
// Counting leaves out experts without rows, which are most of them when a few
// tokens meet many experts (one token, 8 of 256 experts, 2 x 2048 x 6144: 36 us
// with a work-group for every expert, 22 like this), and spreads an expert of
// many rows over the GPU.
constexpr int kMostTiles = 1 << 24;

template <int BM>
__device__ __forceinline__ ExpertTile find_tile(const MxGroupedLaunch& p, int q) {
  const int lane = threadIdx.x & 63;
  const int epl = ((p.E + 63) / 64 + 3) / 4 * 4, e0 = lane * epl;
  int at[5], n[4];  // four experts: their offsets and tiles
  const auto load4 = [&](int e) {
#pragma unroll
    for (int i = 0; i < 5; ++i) at[i] = p.offsets[min(e + i, p.E)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool good = e + i < p.E && at[i] >= 0 && at[i + 1] > at[i] && at[i + 1] <= p.rows;
      n[i] = good ? (at[i + 1] - at[i] + BM - 1) / BM : 0;
    }
  };
  int mine = 0;
  for (int e = 0; e < epl; e += 4) {
    load4(e0 + e);
    mine = min(mine + min(n[0], kMostTiles) + min(n[1], kMostTiles) + min(n[2], kMostTiles) + min(n[3], kMostTiles), kMostTiles);
  }
  int upto = mine;  // inclusive prefix sum
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  const uint64_t after = __ballot(upto > q);
  ExpertTile t{-1, 0, 0, 0, 0};
  if (after == 0) return t;
  const int owner = __builtin_ctzll(after);
  // in every lane, of which the owner's counts
  int first = upto - mine, e = -1, lo = 0, hi = 0, tiles = 0, before = 0;
  for (int b = 0; b < epl; b += 4) {
    if (epl > 4) load4(e0 + b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e < 0 && q - first < n[i]) {
        e = e0 + b + i;
        lo = at[i];
        hi = at[i + 1];
        tiles = n[i];
        before = first;
      }
      first += e < 0 ? n[i] : 0;
    }
  }
  t.expert = __builtin_amdgcn_readlane(e, owner);
  t.first = __builtin_amdgcn_readlane(before, owner);
  t.tiles = __builtin_amdgcn_readlane(tiles, owner);
  t.lo = __builtin_amdgcn_readlane(lo, owner);
  t.hi = __builtin_amdgcn_readlane(hi, owner);
  return t;
}

}  // namespace nvfp4
