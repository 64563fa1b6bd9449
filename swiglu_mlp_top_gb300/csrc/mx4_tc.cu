// Products of rows and weights in microscaled 4-bit floating point on the
// 5th-generation tensor cores: ys = v(xs) v(w[e])^T, fp32 accumulators.
//
// tcgen05.mma kind::mxf4 over a CTA pair multiplies 256 rows x 256 columns x
// 64 packed e2m1 elements and scales each group of 32 by its power of two,
// which it reads from TMEM.  As for bf16 (grouped_tc.cu): tiles of 256 rows,
// operands by TMA into a ring of stages of 128 bytes a row (256 elements),
// half of the weights' rows in each CTA.  A tile has up to 224 columns: an even
// share of N in multiples of 32.
//
// Scales.  The four scale bytes of 128 columns of a row are one word, and a
// TMEM column holds the words of 32 rows.  tcgen05.cp takes 32 x 16 bytes from
// shared memory to four columns, where the 16 bytes at l are the words of rows
// l, l + 32, l + 64, l + 96.  A word's rows lie next to each other in memory
// ([columns / 128, rows, 4]), so a warp reads 32 of them at once and any first
// row will do.  Five warps take a stage each in turn (all 256 columns' scales
// in each CTA: a CTA scales its own half of the rows): they load a stage's
// words before its place in the ring is free, and store 16 bytes a lane.  (Two
// warps that copied every stage word by word with cp.async made the stages
// follow each other at 2000 cycles, most of it the way of one stage's words.)
//
// TMEM: two accumulators of up to 224 columns, so that the epilogue of a tile
// runs under the products of the next, and two stages of scales, 24 columns
// each.  (One accumulator of 256: the tensor cores wait 4000 cycles a tile for
// the epilogue of both CTAs.)
//
// The MMA warp goes through its loop as a whole and issues from one lane, so
// that descriptors stay in uniform registers: issued from a loop of one lane,
// the eleven instructions of a stage take 950 cycles, twice the tensor cores'
// time.
#include "grouped.cuh"
#include "mx4.cuh"

namespace mm {

constexpr int kMtStages = 5;
constexpr int kMtMaxN = 224;                          // columns of a tile
constexpr int kMtTileA = 128 * 128;                   // 16 KiB: 128 rows x 256 elements
constexpr int kMtTileB = kMtMaxN / 2 * 128;
constexpr int kMtSc = 2 * (128 + 256) * 4;            // scale words of a stage: of 128 rows and 256 columns, twice
constexpr int kMtStageBytes = kMtTileA + kMtTileB + kMtSc;
constexpr int kMtEpiWarps = 8;
constexpr int kMtWarpProducer = kMtEpiWarps, kMtWarpMma = kMtEpiWarps + 1, kMtWarpScales = kMtEpiWarps + 2;
constexpr int kMtScaleWarps = 5;
static_assert(kMtScaleWarps <= kMtStages, "a stage has one warp at a time: a wait tells two neighbouring phases apart");
constexpr int kMtThreads = 32 * (kMtEpiWarps + 2 + kMtScaleWarps);
constexpr int kMtEpi = 2 * 32 * 64;                   // per warp: two pieces of 32 rows x 32 columns
constexpr int kMtSmem = kMtStages * kMtStageBytes + kMtEpiWarps * kMtEpi + 1024 + 256;
static_assert(kMtSmem + sizeof(GmTables) + 64 <= 232448, "shared memory budget");
constexpr uint32_t kMtScales = 2 * kMtMaxN, kMtScaleCols = 24;   // TMEM: 8 columns of A's, 16 of B's
static_assert(kMtScales + 2 * kMtScaleCols <= 512, "TMEM columns");

struct MtParams {
  CUtensorMap a, b, out;
  GroupTables g;
  const uint8_t* a_sc;      // [words, rows, 4]
  const uint8_t* b_sc;      // [words, E * N, 4]
  int N;                    // columns of the result
  int nt;                   // columns of a tile, a multiple of 32
  int stages;               // stages of 256 elements
  int words;                // scale words of a row
  int out_aligned;
  void* outp;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMtThreads, 1)
mx4_tc_kernel(const __grid_constant__ MtParams P, WsHeader* hdr) {
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = sA + kMtStages * kMtTileA;
  uint8_t* sEpi = sB + kMtStages * kMtTileB;
  uint8_t* sSc = sEpi + kMtEpiWarps * kMtEpi;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSc + kMtStages * kMtSc);
  uint64_t* full = bars;                   // [stages] even CTA: both CTAs' bytes and scales
  uint64_t* empty = bars + kMtStages;      // [stages] each CTA: released by the pair's MMAs
  uint64_t* tfull = bars + 2 * kMtStages;  // [2] each CTA: accumulator ready
  uint64_t* tempty = tfull + 2;            // [2] even CTA: both CTAs' epilogues have read it
  uint64_t* drained = tempty + 2;          // even CTA: all MMAs finished
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ GmTables s_tab;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = blockIdx.x >> 1, nc = gridDim.x >> 1;
  const int ntn = (P.N + P.nt - 1) / P.nt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMtStages; ++s) {
      mbar_init(&full[s], 1 + 2);          // the bytes, and each CTA's scales
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kMtEpiWarps);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 0) {
    // tables and operands may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    gm_tables<kGroupedForward>(P.g, s_tab, ntn);
  }
  if (warp == kMtWarpMma) {
    tmem_alloc_cta2(&s_tmem, 512);
    tmem_relinquish_cta2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int total = s_tab.tstart[P.g.E];
  volatile int* abort = &s_abort;

  if (warp == kMtWarpProducer) {
    // ------------------------------------------------ TMA (both CTAs)
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = cluster; ok && tile < total; tile += nc) {
        const GmTile ti = gm_tile<kGroupedForward>(tile, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
        for (int kb = 0; kb < P.stages; ++kb, ++it) {
          const int s = it % kMtStages;
          const uint32_t ph = (it / kMtStages) & 1;
          if (!mbar_wait(&empty[s], ph ^ 1, abort, hdr, 121)) { ok = false; break; }
          const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kMtTileA + P.nt * 128);
          tma_load_2d_cta2(sA + s * kMtTileA, &P.a, fb, kb * 128, ti.m0);
          tma_load_3d_cta2(sB + s * kMtTileB, &P.b, fb, kb * 128, ti.n0 + P.nt / 2 * rank, ti.e);
        }
      }
      if (!ok && rank == 0) {
        // a wait gave up: the copies in flight land before the block ends
        for (int j = 0; j < kMtStages; ++j) {
          const int i2 = it - 1 - j;
          if (i2 < 0) break;
          mbar_wait(&full[i2 % kMtStages], (i2 / kMtStages) & 1, nullptr, hdr, 122);
        }
      }
    }
    __syncwarp();
  } else if (warp >= kMtWarpScales) {
    // ------------------------------------------------ scales (both CTAs): a warp a stage, in turn
    const int64_t a_rows = P.g.rows, b_rows = static_cast<int64_t>(P.g.E) * P.N;
    const uint32_t* a_sc = reinterpret_cast<const uint32_t*>(P.a_sc);
    const uint32_t* b_sc = reinterpret_cast<const uint32_t*>(P.b_sc);
    const int mine = total > cluster ? (total - cluster + nc - 1) / nc * P.stages : 0;      // stages of all tiles
    int have = -1;
    GmTile ti;
    for (int it = warp - kMtWarpScales; it < mine; it += kMtScaleWarps) {
      const int nth = it / P.stages, kb = it - nth * P.stages;
      if (nth != have) ti = gm_tile<kGroupedForward>(cluster + nth * nc, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
      have = nth;
      // a lane's words of rows lane, + 32, + 64, + 96 of each 128; where there is
      // nothing, zeros: 2^-127, which scales zeros or rows that are not stored
      uint32_t w[6][4];
      const int64_t b0 = static_cast<int64_t>(ti.e) * P.N + ti.n0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int word = 2 * kb + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 32 + lane;
          w[3 * c][i] = word < P.words && ti.m0 + r < a_rows ? a_sc[word * a_rows + ti.m0 + r] : 0u;
          w[3 * c + 1][i] = word < P.words && ti.n0 + r < P.N ? b_sc[word * b_rows + b0 + r] : 0u;
          w[3 * c + 2][i] = word < P.words && ti.n0 + 128 + r < P.N ? b_sc[word * b_rows + b0 + 128 + r] : 0u;
        }
      }
      const int s = it % kMtStages;
      const uint32_t ph = (it / kMtStages) & 1;
      if (!warp_wait(&empty[s], ph ^ 1, abort, hdr, 123)) break;
      uint4* to = reinterpret_cast<uint4*>(sSc + s * kMtSc) + lane;
#pragma unroll
      for (int q = 0; q < 6; ++q) to[32 * q] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
      fence_proxy_async_smem();                // visible to the tensor core, and told to the even CTA
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&full[s]);
        // a release of all writes would keep the lane from its next stage (dense
        // 8192 x 4096 x 8192: 119 us, 86 without)
        else mbar_release_smem_cluster(mapa_shared(smem_u32(&full[s]), 0));
      }
    }
    __syncwarp();
  } else if (warp == kMtWarpMma) {
    // ------------------------------------------------ MMA (even CTA)
    if (rank == 0) {
      const bool leader = elect_one();
      const int tiles = __shfl_sync(0xffffffffu, total, 0);
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t id0 = idesc_mxf4(256, 0, 0) | (static_cast<uint32_t>(P.nt >> 3) << 17);
      const uint32_t id2 = idesc_mxf4(256, 0, 2) | (static_cast<uint32_t>(P.nt >> 3) << 17);
      const uint64_t da = smem_desc_sw128(smem_u32(sA)), db = smem_desc_sw128(smem_u32(sB));
      const uint64_t ds = smem_desc_rows16(smem_u32(sSc));
      int s = 0, used = 0;
      uint32_t ph = 0, sc = base + kMtScales;
      bool ok = true;
      for (int tile = cluster; ok && tile < tiles; tile += nc, ++used) {
        ok = warp_wait<true>(&tempty[used & 1], ((used >> 1) & 1) ^ 1, abort, hdr, 124);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = base + (used & 1) * kMtMaxN;
        for (int kb = 0; kb < P.stages; ++kb) {
          ok = warp_wait<true>(&full[s], ph, abort, hdr, 125);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t dss = ds + static_cast<uint64_t>(s * (kMtSc / 16));
            const uint64_t das = da + static_cast<uint64_t>(s * (kMtTileA / 16));
            const uint64_t dbs = db + static_cast<uint64_t>(s * (kMtTileB / 16));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tmem_cp_scales_cta2(sc + 4 * c, dss + 96 * c);
              tmem_cp_scales_cta2(sc + 8 + 8 * c, dss + 96 * c + 32);
              tmem_cp_scales_cta2(sc + 8 + 8 * c + 4, dss + 96 * c + 64);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_mxf4_cta2(d, das + 2 * kk, dbs + 2 * kk, (kk & 1) ? id2 : id0, sc + 4 * (kk >> 1), sc + 8 + 8 * (kk >> 1),
                             (kb | kk) ? 1u : 0u);
            umma_commit_cta2_mc(&empty[s], 0x3);
            if (kb + 1 == P.stages) umma_commit_cta2_mc(&tfull[used & 1], 0x3);
          }
          __syncwarp();
          sc ^= (base + kMtScales) ^ (base + kMtScales + kMtScaleCols);
          if (++s == kMtStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (leader) umma_commit_cta2_mc(drained, 0x1);
      __syncwarp();
      warp_wait(drained, 0, nullptr, hdr, 126);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (warps 0-7, both CTAs)
    const int quad = warp & 3, half = warp >> 2;
    uint8_t* wstage = sEpi + warp * kMtEpi;
    const uint32_t te0 = mapa_shared(smem_u32(&tempty[0]), 0), te1 = mapa_shared(smem_u32(&tempty[1]), 0);
    int used = 0;
    for (int tile = cluster; tile < total; tile += nc, ++used) {
      const GmTile ti = gm_tile<kGroupedForward>(tile, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
      if (!warp_wait(&tfull[used & 1], (used >> 1) & 1, abort, hdr, 127)) break;
      tc_fence_after();
      const int rem = min(32, ti.mrows - quad * 32);            // rows of the group in this warp's 32
      const bool counts = quad * 32 + lane < ti.mvalid;         // this lane's row is not padding
      const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (used & 1) * kMtMaxN;
      const int row = ti.m0 + quad * 32;
      // every other piece of 32 columns, packed, so that the accumulator is free before the stores
      uint32_t pk[4][16];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int c = 32 * half + 64 * p;
        if (c >= P.nt) continue;                   // warp-uniform
        uint32_t r[32];
        tmem_ld_32x32b_x32(tb + c, r);             // every lane (warp-collective)
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q)
          pk[p][q] = counts ? pack_bf16x2(__uint_as_float(r[2 * q]), __uint_as_float(r[2 * q + 1])) : 0u;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_signal_cluster((used & 1) ? te1 : te0);
      if (rem <= 0) continue;                      // warp-uniform
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        const int c0 = ti.n0 + 32 * half + 64 * b; // two pieces at once: columns c0 and c0 + 64
        if (32 * half + 64 * b >= P.nt || c0 >= P.N) break;
        const bool two = 32 * half + 64 * b + 64 < P.nt && c0 + 64 < P.N;
        if (lane == 0) bulk_wait_read();           // the stores before have read the stage
        __syncwarp();
        // 64-byte rows, 16-byte chunk q of row i at chunk q ^ ((i >> 1) & 3)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(wstage + p * (kMtEpi / 2) + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pk[b + p][4 * q], pk[b + p][4 * q + 1], pk[b + p][4 * q + 2], pk[b + p][4 * q + 3]);
        if (P.out_aligned && rem == 32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&P.out, wstage, c0, row);
            if (two) tma_store_2d(&P.out, wstage + kMtEpi / 2, c0 + 64, row);
            bulk_commit();
          }
          continue;
        }
        __syncwarp();
        for (int p = 0; p < 1 + two; ++p) {
          const uint8_t* stage = wstage + p * (kMtEpi / 2);
          const int col = c0 + 64 * p;
          uint16_t* o = static_cast<uint16_t*>(P.outp) + static_cast<int64_t>(row) * P.N + col;
          if (P.out_aligned) {
            // a group's ragged end: 16 bytes a lane, eight rows at once
            if (col + 8 * (lane & 3) < P.N)
              for (int i = lane >> 2; i < rem; i += 8)
                *reinterpret_cast<uint4*>(o + static_cast<int64_t>(i) * P.N + 8 * (lane & 3)) =
                    *reinterpret_cast<const uint4*>(stage + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
          } else if (col + lane < P.N) {
            // rows that start anywhere: element by element
            for (int i = 0; i < rem; ++i)
              o[static_cast<int64_t>(i) * P.N + lane] =
                  *reinterpret_cast<const uint16_t*>(stage + i * 64 + ((((lane >> 3) ^ ((i >> 1) & 3)) << 4) | ((lane & 7) << 1)));
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's tensor stores have landed
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kMtWarpMma) tmem_dealloc_cta2(tmem, 512);
}

// ===================================================== bf16 rows, 4-bit weights
// ys = x v(w[e])^T with x in bf16: the forward kernel of grouped_tc.cu (tiles of
// 256 x 256 or 256 x 128, slices of 64, kind::f16), whose B tiles are made from
// codes instead of loaded.  Six warps take a stage each in turn: a lane loads
// the 32 bytes of codes and the scale word of four rows (one stage ahead of the
// one that it converts), multiplies (mx4.cuh, 19 instructions for 8 values) and
// stores 16 bytes at a time where the swizzled TMA layout has them.  The
// weights are read and converted in 4 bits for each tile of 256 rows that needs
// them, once where an expert has no more rows; with a bf16 copy of the weights
// first (and no copy of x) T = 256, E = 8, K = 768, N = 4864 took 28 us.
constexpr int kMwRing = 6, kMwTile = 128 * 64 * 2;
constexpr int kMwWarpConvert = kMtEpiWarps + 2, kMwConverters = 6;
static_assert(kMwConverters <= kMwRing, "a stage has one warp at a time: a wait tells two neighbouring phases apart");
constexpr int kMwThreads = 32 * (kMtEpiWarps + 2 + kMwConverters);
constexpr int kMwStage = 32 * 128;                    // epilogue: 32 rows x 128 bytes per warp
constexpr int kMwSmem = kMwRing * 2 * kMwTile + kMtEpiWarps * kMwStage + 1024 + 256;
static_assert(kMwSmem + sizeof(GmTables) + 64 <= 232448, "shared memory budget");

struct MwParams {
  CUtensorMap a, out;
  GroupTables g;
  const uint8_t* w;         // codes [E * N, 16 groups]
  const uint32_t* sc;       // [words, E * N]
  int N, K, nt, groups;
  int out_aligned;
  void* outp;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMwThreads, 1)
mx4w_tc_kernel(const __grid_constant__ MwParams P, WsHeader* hdr) {
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = sA + kMwRing * kMwTile;
  uint8_t* sEpi = sB + kMwRing * kMwTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + kMtEpiWarps * kMwStage);
  uint64_t* full = bars;                   // [stages] even CTA: both CTAs' rows and weights
  uint64_t* empty = bars + kMwRing;        // [stages] each CTA: released by the pair's MMAs
  uint64_t* tfull = bars + 2 * kMwRing;    // [2] each CTA: accumulator ready
  uint64_t* tempty = tfull + 2;            // [2] even CTA: both CTAs' epilogues have read it
  uint64_t* drained = tempty + 2;          // even CTA: all MMAs finished
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ GmTables s_tab;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = blockIdx.x >> 1, nc = gridDim.x >> 1;
  const int ntn = (P.N + P.nt - 1) / P.nt, slices = (P.K + 63) / 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMwRing; ++s) {
      mbar_init(&full[s], 1 + 2);          // the bytes of A, and each CTA's converted weights
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kMtEpiWarps);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 0) {
    // tables and operands may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    gm_tables<kGroupedForward>(P.g, s_tab, ntn);
  }
  if (warp == kMtWarpMma) {
    tmem_alloc_cta2(&s_tmem, 512);
    tmem_relinquish_cta2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int total = s_tab.tstart[P.g.E];
  volatile int* abort = &s_abort;

  if (warp == kMtWarpProducer) {
    // ------------------------------------------------ TMA: rows of x (both CTAs)
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = cluster; ok && tile < total; tile += nc) {
        const GmTile ti = gm_tile<kGroupedForward>(tile, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
        for (int kb = 0; kb < slices; ++kb, ++it) {
          const int s = it % kMwRing;
          const uint32_t ph = (it / kMwRing) & 1;
          if (!mbar_wait(&empty[s], ph ^ 1, abort, hdr, 131)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kMwTile);
          tma_load_2d_cta2(sA + s * kMwTile, &P.a, mapa_shared(smem_u32(&full[s]), 0), kb * 64, ti.m0);
        }
      }
      if (!ok && rank == 0) {
        // a wait gave up: the copies in flight land before the block ends
        for (int j = 0; j < kMwRing; ++j) {
          const int i2 = it - 1 - j;
          if (i2 < 0) break;
          mbar_wait(&full[i2 % kMwRing], (i2 / kMwRing) & 1, nullptr, hdr, 132);
        }
      }
    }
    __syncwarp();
  } else if (warp >= kMwWarpConvert) {
    // ------------------------------------------------ weights (both CTAs): a warp a stage, in turn
    const int64_t rows = static_cast<int64_t>(P.g.E) * P.N, pitch = 16 * static_cast<int64_t>(P.groups);
    const int mine = total > cluster ? (total - cluster + nc - 1) / nc * slices : 0;      // stages of all tiles
    const int per = P.nt / 64;             // rows of a lane
    struct Loaded {
      uint4 c[4][2];
      uint32_t sc[4];
    };
    // the codes of stage `it`: two groups of rows lane, + 32, + 64, + 96
    auto load = [&](int it, Loaded& v) {
      const int nth = it / slices, kb = it - nth * slices;
      const GmTile ti = gm_tile<kGroupedForward>(cluster + nth * nc, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
      const int n0 = ti.n0 + P.nt / 2 * rank;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * i + lane;
        const bool in = i < per && n < P.N;
        const int64_t r = static_cast<int64_t>(ti.e) * P.N + n;
        const uint4* from = reinterpret_cast<const uint4*>(P.w + r * pitch) + 2 * kb;
        // where there is nothing, zeros of scale 2^-127
        v.c[i][0] = in ? __ldg(from) : make_uint4(0u, 0u, 0u, 0u);
        v.c[i][1] = in && 2 * kb + 1 < P.groups ? __ldg(from + 1) : make_uint4(0u, 0u, 0u, 0u);
        v.sc[i] = in ? __ldg(P.sc + (kb >> 1) * rows + r) >> (16 * (kb & 1)) : 0u;
      }
    };
    auto convert = [&](int it, const Loaded& v) {
      const int s = it % kMwRing;
      const uint32_t ph = (it / kMwRing) & 1;
      if (!warp_wait(&empty[s], ph ^ 1, abort, hdr, 133)) return false;
      uint8_t* tile = sB + s * kMwTile;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= per) break;
        const int r = 32 * i + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t byte = (v.sc[i] >> (8 * h)) & 255u;
          uint32_t f1, f2;
          mx4_factors(byte, f1, f2);
          const bool two = __any_sync(0xffffffffu, byte > 128u);
          const uint32_t c[4] = {v.c[i][h].x, v.c[i][h].y, v.c[i][h].z, v.c[i][h].w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            // 128-byte rows, 16-byte chunk j of row r at chunk j ^ (r & 7)
            *reinterpret_cast<uint4*>(tile + r * 128 + (((4 * h + q) ^ (r & 7)) << 4)) =
                two ? e2m1_bf16<true>(c[q], f1, f2) : e2m1_bf16<false>(c[q], f1, 0u);
        }
      }
      fence_proxy_async_smem();            // where this SM's tensor core reads them
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&full[s]);
        else mbar_release_smem_cluster(mapa_shared(smem_u32(&full[s]), 0));
      }
      return true;
    };
    Loaded a, b;
    int it = warp - kMwWarpConvert;
    if (it < mine) load(it, a);
    while (it < mine) {
      if (it + kMwConverters < mine) load(it + kMwConverters, b);
      if (!convert(it, a)) break;
      it += kMwConverters;
      if (it >= mine) break;
      if (it + kMwConverters < mine) load(it + kMwConverters, a);
      if (!convert(it, b)) break;
      it += kMwConverters;
    }
    __syncwarp();
  } else if (warp == kMtWarpMma) {
    // ------------------------------------------------ MMA (even CTA)
    if (rank == 0) {
      const bool leader = elect_one();
      const int tiles = __shfl_sync(0xffffffffu, total, 0);
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc = idesc_bf16_f32(256, 0) | (static_cast<uint32_t>(P.nt >> 3) << 17);
      const uint64_t da = smem_desc_sw128(smem_u32(sA)), db = smem_desc_sw128(smem_u32(sB));
      int s = 0, used = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cluster; ok && tile < tiles; tile += nc, ++used) {
        ok = warp_wait<true>(&tempty[used & 1], ((used >> 1) & 1) ^ 1, abort, hdr, 134);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = base + (used & 1) * 256;
        for (int kb = 0; kb < slices; ++kb) {
          ok = warp_wait<true>(&full[s], ph, abort, hdr, 135);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t as = da + static_cast<uint64_t>(s * (kMwTile / 16)), bs = db + static_cast<uint64_t>(s * (kMwTile / 16));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_f16_cta2(d, as + 2 * kk, bs + 2 * kk, idesc, (kb | kk) ? 1u : 0u);
            umma_commit_cta2_mc(&empty[s], 0x3);
            if (kb + 1 == slices) umma_commit_cta2_mc(&tfull[used & 1], 0x3);
          }
          __syncwarp();
          if (++s == kMwRing) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (leader) umma_commit_cta2_mc(drained, 0x1);
      __syncwarp();
      warp_wait(drained, 0, nullptr, hdr, 136);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (warps 0-7, both CTAs)
    const int quad = warp & 3, half = warp >> 2, hc = P.nt / 2;
    uint8_t* wstage = sEpi + warp * kMwStage;
    const uint32_t te0 = mapa_shared(smem_u32(&tempty[0]), 0), te1 = mapa_shared(smem_u32(&tempty[1]), 0);
    int used = 0;
    for (int tile = cluster; tile < total; tile += nc, ++used) {
      const GmTile ti = gm_tile<kGroupedForward>(tile, P.g.E, 0, 0, s_tab, ntn, P.nt, rank);
      if (!warp_wait(&tfull[used & 1], (used >> 1) & 1, abort, hdr, 137)) break;
      tc_fence_after();
      const int rem = min(32, ti.mrows - quad * 32);            // rows of the group in this warp's 32
      const bool counts = quad * 32 + lane < ti.mvalid;         // this lane's row is not padding
      const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (used & 1) * 256 + half * hc;
#pragma unroll 1
      for (int c = 0; c < hc; c += 64) {
        uint32_t pk[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tb + c + 32 * h, r);  // every lane (warp-collective)
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 16; ++q)
            pk[16 * h + q] = counts ? pack_bf16x2(__uint_as_float(r[2 * q]), __uint_as_float(r[2 * q + 1])) : 0u;
        }
        if (c + 64 == hc) {                        // the accumulator is read: the next tile may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_signal_cluster((used & 1) ? te1 : te0);
        }
        const int col = ti.n0 + half * hc + c;
        if (rem > 0 && col < P.N)
          store_rows_bf16(pk, wstage, &P.out, P.outp, P.out_aligned, ti.m0 + quad * 32, col, rem, P.N, lane);
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's tensor stores have landed
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kMtWarpMma) tmem_dealloc_cta2(tmem, 512);
}

// =============================================================== host side
cudaError_t launch_mx4_tc(const Mx4MatmulArgs& a, WsHeader* hdr, cudaStream_t st) {
  MtParams p;
  memset(&p, 0, sizeof(p));
  const int groups = (a.K + 31) / 32;
  p.g = a.g;
  p.a_sc = a.x_exps;
  p.b_sc = a.w_exps;
  p.N = a.N;
  p.words = (groups + 3) / 4;
  p.stages = (groups + 7) / 8;
  p.outp = a.out;
  p.out_aligned = a.N % 8 == 0;
  const uint64_t row = 16 * static_cast<uint64_t>(groups);
  const uint64_t da[2] = {row, static_cast<uint64_t>(a.g.rows)}, sa[1] = {row};
  const uint64_t db[3] = {row, static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.g.E)}, sb[2] = {row, row * a.N};
  // an even share of the columns
  const int ntn = (a.N + kMtMaxN - 1) / kMtMaxN;
  p.nt = ((a.N + ntn - 1) / ntn + 31) / 32 * 32;
  const uint32_t boxa[2] = {128, 128}, boxb[3] = {128, static_cast<uint32_t>(p.nt / 2), 1};
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!make_map(&p.a, u8, 2, reinterpret_cast<uint64_t>(a.x), da, sa, boxa, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.b, u8, 3, reinterpret_cast<uint64_t>(a.w), db, sb, boxb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (p.out_aligned && !map_out_rows(&p.out, a.out, a.N, a.g.rows, 32)))
    return cudaErrorInvalidValue;
  const int64_t tiles = row_tiles256(a.g) * ntn;
  if (tiles * p.stages > 0x3fffffff) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(mx4_tc_kernel), kMtSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms() / 2));
  return launch_dependent_kernel(mx4_tc_kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(kMtThreads), kMtSmem, st,
                                 p, hdr);
}

cudaError_t launch_mx4w_tc(const Mx4MatmulArgs& a, WsHeader* hdr, cudaStream_t st) {
  MwParams p;
  memset(&p, 0, sizeof(p));
  p.g = a.g;
  p.w = static_cast<const uint8_t*>(a.w);
  p.sc = reinterpret_cast<const uint32_t*>(a.w_exps);
  p.N = a.N;
  p.K = a.K;
  p.groups = (a.K + 31) / 32;
  p.nt = gm_columns(row_tiles256(a.g), a.N);
  p.outp = a.out;
  p.out_aligned = a.N % 8 == 0;
  const uint64_t da[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.g.rows)}, sa[1] = {2 * static_cast<uint64_t>(pitch8(a.K))};
  const uint32_t box[2] = {64, 128};
  if (!make_map(&p.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, reinterpret_cast<uint64_t>(a.x), da, sa, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (p.out_aligned && !map_out_rows(&p.out, a.out, a.N, a.g.rows, 64)))
    return cudaErrorInvalidValue;
  const int64_t tiles = row_tiles256(a.g) * ((a.N + p.nt - 1) / p.nt);
  if (tiles * ((a.K + 63) / 64) > 0x3fffffff) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(mx4w_tc_kernel), kMwSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms() / 2));
  return launch_dependent_kernel(mx4w_tc_kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(kMwThreads), kMwSmem, st, p,
                                 hdr);
}

}  // namespace mm
