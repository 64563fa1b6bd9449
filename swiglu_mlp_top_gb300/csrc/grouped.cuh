// Row groups of the experts' products, read from the device tables of a sort.
#pragma once

#include "mm_kernels.cuh"

namespace mm {

// Rows [r0, r1) belong to the group, the first n of them hold an assignment
// and the rest are padding.  The tables are a caller's: whatever they hold,
// the rows stay inside [0, rows).
struct GroupSpan {
  int r0, r1, n;
};

__device__ __forceinline__ GroupSpan group_span(const GroupTables& g, int e) {
  const int R = static_cast<int>(g.rows);
  if (g.offsets == nullptr) return GroupSpan{0, R, R};
  GroupSpan s;
  s.r0 = min(max(g.offsets[e], 0), R);
  s.r1 = min(max(g.offsets[e + 1], s.r0), R);
  s.n = min(max(g.counts[e], 0), s.r1 - s.r0);
  return s;
}

// Where the tile with index t lies among tiles of `block` rows of every group
// in order, `cols` tiles to a row of tiles.  Called by a full warp; every lane
// gets the answer; e < 0: there is no such tile.
struct GroupTile {
  int e, mb, nb;
  GroupSpan s;
};

__device__ __forceinline__ GroupTile find_group_tile(const GroupTables& g, int64_t t, int block,
                                                     int cols) {
  static_assert(MM_MAX_EXPERTS <= 64, "two groups a lane");
  const int lane = threadIdx.x & 31;
  GroupSpan s[2];
  int rows_of[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * lane + i;
    s[i] = e < g.E ? group_span(g, e) : GroupSpan{0, 0, 0};
    rows_of[i] = (s[i].r1 - s[i].r0 + block - 1) / block;
  }
  const int mine = rows_of[0] + rows_of[1];
  int before = mine;                           // inclusive prefix over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  before -= mine;
  const int64_t row = t / cols;
  const bool here = row >= before && row < before + mine;
  const uint32_t who = __ballot_sync(0xffffffffu, here);
  GroupTile r{-1, 0, 0, {0, 0, 0}};
  if (who == 0) return r;
  const int src = __ffs(who) - 1;
  const int local = static_cast<int>(row) - before;
  const int second = local >= rows_of[0];
  r.e = __shfl_sync(0xffffffffu, 2 * lane + second, src);
  r.mb = __shfl_sync(0xffffffffu, second ? local - rows_of[0] : local, src);
  r.nb = static_cast<int>(t % cols);
  r.s.r0 = __shfl_sync(0xffffffffu, second ? s[1].r0 : s[0].r0, src);
  r.s.r1 = __shfl_sync(0xffffffffu, second ? s[1].r1 : s[0].r1, src);
  r.s.n = __shfl_sync(0xffffffffu, second ? s[1].n : s[0].n, src);
  return r;
}

}  // namespace mm
