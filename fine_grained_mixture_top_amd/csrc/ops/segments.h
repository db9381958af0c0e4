// Row tiles of a plan's segments.
#pragma once

#include "../device_common.h"

namespace moe {

// n rows from row o on, as far as they lie in the `total` rows of the buffers (rows past
// them are never touched)
__device__ __forceinline__ int rows_inside(int total, int o, int n) {
  return o < 0 || o >= total ? 0 : max(0, min(n, total - o));
}

// The tile number `mg` when every segment's rows are cut into tiles of BM: its expert,
// first row and rows (at most BM), the same in all lanes of the wave.  False when there
// is none.  offsets null: one segment of `total` rows.
//   Lanes scan `per` experts each, four at a time (loads of four in flight; up to 256
// experts they stay in registers).
template <int BM>
__device__ __forceinline__ bool segment_tile(const int32_t* offsets, const int32_t* counts, int E, int total, int mg,
                                             int lane, int& e, int& row0, int& rows) {
  const int per = (E + 63) >> 6;
  int first[4], rws[4];
  int mine = 0;
  for (int x0 = 0; x0 < per; x0 += 4) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = lane * per + x0 + x;
      const bool is = x0 + x < per && i < E;
      first[x] = is && offsets ? offsets[i] : 0;
      rws[x] = is ? (offsets ? counts[i] : total) : 0;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      rws[x] = rows_inside(total, first[x], rws[x]);
      mine += (rws[x] + BM - 1) / BM;
    }
  }
  int incl = mine;
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(incl, s, 64);
    if (lane >= s) incl += y;
  }
  const uint64_t past = __ballot(incl > mg);
  if (past == 0) return false;
  const int src = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
  int left = mg - (__builtin_amdgcn_readlane(incl, src) - __builtin_amdgcn_readlane(mine, src));
  int n = 0;
  e = src * per;
  row0 = 0;
  if (per <= 4) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int nx = __builtin_amdgcn_readlane(rws[x], src), tiles = (nx + BM - 1) / BM;
      if (left >= 0 && left < tiles) {
        e = src * per + x;
        n = nx;
        row0 = __builtin_amdgcn_readlane(first[x], src) + left * BM;
        n -= left * BM;
        left = -1;
      }
      if (left >= 0) left -= tiles;
    }
  } else {
    for (;; ++e) {
      row0 = __builtin_amdgcn_readfirstlane(offsets[e]);
      n = rows_inside(total, row0, __builtin_amdgcn_readfirstlane(counts[e]));
      const int tiles = (n + BM - 1) / BM;
      if (left < tiles) break;
      left -= tiles;
    }
    row0 += left * BM;
    n -= left * BM;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  rows = min(__builtin_amdgcn_readfirstlane(n), BM);
  return true;
}

}  // namespace moe
