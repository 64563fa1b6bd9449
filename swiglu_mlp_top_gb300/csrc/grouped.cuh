// Row groups of the experts' products, read from the device tables of a sort.
#pragma once

#include <algorithm>

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

// The groups' rows in chunks of at most MOST, group after group: chunk c
// belongs to the last group whose `first` is not above c.  PADDING: a group's
// padding is cut up with its rows; else a group that has padding alone is one
// chunk.  By the block's first warp.
struct GroupChunks {
  GroupSpan span[MM_MAX_EXPERTS];
  int first[MM_MAX_EXPERTS];                   // behind the last group: their number
  int count;
};

template <int MOST, bool PADDING>
__device__ __forceinline__ void group_chunks(const GroupTables& g, GroupChunks* t) {
  static_assert(MM_MAX_EXPERTS == 64, "two groups a lane");
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  GroupSpan s[2];
  int mine[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * lane + i;
    s[i] = e < g.E ? group_span(g, e) : GroupSpan{0, 0, 0};
    mine[i] = s[i].r1 == s[i].r0 ? 0 : PADDING ? (s[i].r1 - s[i].r0 + MOST - 1) / MOST : max(1, (s[i].n + MOST - 1) / MOST);
  }
  int upto = mine[0] + mine[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  t->span[2 * lane] = s[0];
  t->span[2 * lane + 1] = s[1];
  t->first[2 * lane] = upto - mine[1] - mine[0];
  t->first[2 * lane + 1] = upto - mine[1];
  if (lane == 31) t->count = upto;
}

// The group of chunk c < count; by a full warp.
__device__ __forceinline__ int chunk_group(const GroupChunks& t, int c) {
  const int lane = threadIdx.x & 31;
  return __popc(__ballot_sync(0xffffffffu, t.first[lane] <= c)) + __popc(__ballot_sync(0xffffffffu, t.first[lane + 32] <= c)) - 1;
}

// Chunks of `most` rows that any grouping of the rows can give.
inline int64_t most_chunks(const GroupTables& g, int most) {
  const int64_t groups = std::min<int64_t>(g.E, g.rows);
  return groups + (g.rows - groups) / most;
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

// Schedule of the tensor-core kernels: CTA pairs make tiles of 256 rows (of a
// group, or of a weight gradient) x nt columns.
struct GmTables {
  int r0[MM_MAX_EXPERTS], r1[MM_MAX_EXPERTS], n[MM_MAX_EXPERTS], tstart[MM_MAX_EXPERTS + 1];
  uint8_t order[MM_MAX_EXPERTS];   // wgrad: groups by descending rows
};

struct GmTile {
  int e, m0, mrows, mvalid, n0, k0, krows;
};

// Reads the tables, one group a lane (two rounds); the tiles' prefix sums.
template <int OP>
__device__ __forceinline__ void gm_tables(const GroupTables& g, GmTables& s, int ntn) {
  const int lane = threadIdx.x & 31, E = g.E;
  for (int e = lane; e < E; e += 32) {
    const GroupSpan sp = group_span(g, e);
    s.r0[e] = sp.r0;
    s.r1[e] = sp.r1;
    s.n[e] = sp.n;
  }
  __syncwarp();
  if constexpr (OP == kGroupedWgrad) {
    for (int e = lane; e < E; e += 32) {
      int pos = 0;
      for (int o = 0; o < E; ++o) pos += (s.n[o] > s.n[e] || (s.n[o] == s.n[e] && o < e)) ? 1 : 0;
      s.order[pos] = static_cast<uint8_t>(e);
    }
  } else {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int mine = e < E ? ((s.r1[e] - s.r0[e] + 255) / 256) * ntn : 0;
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e < E) s.tstart[e] = base + inc - mine;
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) s.tstart[E] = base;
  }
}

template <int OP>
__device__ __forceinline__ GmTile gm_tile(int t, int E, int M, int K, const GmTables& s, int ntn, int nt, int rank) {
  GmTile ti;
  if constexpr (OP == kGroupedWgrad) {
    const int per = ((M + 255) / 256) * ntn;
    ti.e = s.order[t / per];
    const int local = t % per;
    ti.m0 = (local / ntn) * 256 + rank * 128;
    ti.mrows = ti.mvalid = min(128, M - ti.m0);
    ti.n0 = (local % ntn) * nt;
    ti.k0 = s.r0[ti.e];
    ti.krows = s.n[ti.e];
  } else {
    int lo = 0, hi = E - 1;              // last group with tstart <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.tstart[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int local = t - s.tstart[lo];
    ti.e = lo;
    ti.m0 = s.r0[lo] + (local / ntn) * 256 + rank * 128;
    ti.mrows = s.r1[lo] - ti.m0;             // may be negative for the odd CTA
    ti.mvalid = s.r0[lo] + s.n[lo] - ti.m0;
    ti.n0 = (local % ntn) * nt;
    ti.k0 = 0;
    ti.krows = K;
  }
  return ti;
}

// The j-th tile of pair c of nc.  wgrad: rounds alternately forwards and
// backwards over the groups in descending length, so that the pairs with a
// round's longest tiles take the next one's shortest.
template <int OP>
__device__ __forceinline__ int gm_index(int j, int c, int nc) {
  if constexpr (OP == kGroupedWgrad) return j * nc + ((j & 1) ? nc - 1 - c : c);
  return j * nc + c;
}

// Eight fp32 values times 2^24 as three bf16 parts, each the nearest of what the
// ones before leave.  fp32 numbers are whole multiples of 2^-149, so that the
// scaled ones' parts are multiples of 2^-125, and what is left of 24 bits behind
// two parts has eight: nothing is lost, however small a value is.  Products come
// out times 2^48 (kSplitUnscale takes that away).  Values from kSplitMost on (of
// which the first part may round to infinity), infinities and NaN have no such
// parts; one of their parts is not finite then, and no sum with it is.
constexpr float kSplitScale = 0x1p24f, kSplitUnscale = 0x1p-48f, kSplitMost = 0x1p103f;

__device__ __forceinline__ void split_vector(const float (&x)[8], uint4 (&planes)[3]) {
  uint32_t p[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // rounded by name, or the compiler subtracts the first part in one operation
    // with the scaling and keeps both values (60 rows, E = 8, K = N = 2048: 65 us, 45)
    float a = __fmul_rn(x[2 * j], kSplitScale), b = __fmul_rn(x[2 * j + 1], kSplitScale);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      p[q][j] = pack_bf16x2(a, b);
      a -= __uint_as_float(p[q][j] << 16);
      b -= __uint_as_float(p[q][j] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) planes[q] = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
}

// A warp's 32 rows x 64 columns of bf16 (a row a lane) out through its stage of
// 128-byte rows (16-byte chunk q of row i at chunk q ^ (i & 7)); `rem` rows are
// the group's.
__device__ __forceinline__ void store_rows_bf16(const uint32_t (&pk)[32], uint8_t* wstage, const CUtensorMap* map,
                                                void* outp, int aligned, int row, int col, int rem, int N, int lane) {
  if (lane == 0) bulk_wait_read();                 // the previous piece's store has read the stage
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<uint4*>(wstage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
        make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
  if (aligned && rem == 32) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, wstage, col, row);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  uint16_t* o = static_cast<uint16_t*>(outp) + static_cast<int64_t>(row) * N + col;
  if (aligned) {
    // a group's ragged end: 16 bytes a lane, four rows at once
    if (col + 8 * (lane & 7) < N)
      for (int i = lane >> 3; i < rem; i += 4)
        *reinterpret_cast<uint4*>(o + static_cast<int64_t>(i) * N + 8 * (lane & 7)) =
            *reinterpret_cast<const uint4*>(wstage + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
    return;
  }
  // rows that start anywhere: element by element
  for (int i = 0; i < rem; ++i)
#pragma unroll
    for (int c = lane; c < 64; c += 32)
      if (col + c < N)
        o[static_cast<int64_t>(i) * N + c] =
            *reinterpret_cast<const uint16_t*>(wstage + i * 128 + ((((c >> 3) ^ (i & 7)) << 4) | ((c & 7) << 1)));
}

// ---------------------------------------------------------------- host side
// Result rows in bf16: store boxes of `box` columns (64 or 32) x 32 rows, swizzled
// over the box's row.
inline bool map_out_rows(CUtensorMap* m, void* p, int cols, int64_t rows, int box) {
  const uint64_t d[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, s[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t b[2] = {static_cast<uint32_t>(box), 32};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, reinterpret_cast<uint64_t>(p), d, s, b,
                  box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}
// Tiles of 256 rows that any grouping of the rows can need.
inline int64_t row_tiles256(const GroupTables& g) {
  return g.offsets ? std::min<int64_t>(g.rows, g.rows / 256 + g.E) : (g.rows + 255) / 256;
}

// Columns of a tile: 128 where that is all, or where tiles of 256 would fill at
// most half the pairs of SMs (512 rows, K = 2048, N = 4096: 14.9 -> 13.1 us; 200
// rows, E = 8, K = 768, N = 1024: 9.5 -> 8.6, with 4-bit weights 12.9 -> 9.5).
// Up to all the pairs they mostly lose what they gain in a second round (N =
// 8192: 16.6 -> 22.1; fp32, 1000 rows, N = 2432: 50.5 -> 53.6), so that 400 rows,
// E = 4, N = 2432, which would gain (10.3 -> 9.0), stay with 256.
inline int gm_columns(int64_t row_tiles, int cols) {
  return cols <= 128 || 2 * row_tiles * ((cols + 255) / 256) <= num_sms() / 2 ? 128 : 256;
}

}  // namespace mm
