// Experts' products of bf16 rows on the 5th-generation tensor cores, fp32
// accumulators in TMEM:
//   forward  ys = xs w[e]^T       A = xs  [rows, K]  K-major,   B = w[e] [N, K] K-major
//   dgrad    dxs = dys w[e]       A = dys [rows, N]  K-major,   B = w[e] with its K contiguous (MN-major)
//   wgrad    dw[e] = dys^T xs     A = dys, B = xs, both MN-major; the summed index is the group's rows
//
// A CTA pair makes a tile of 256 x 256 (tcgen05.mma.cta_group::2: 128 rows of
// A and half of B in each CTA's shared memory), in slices of 64 of the summed
// index through a ring of six stages; two accumulators, so that the epilogue
// of one tile runs under the products of the next.  Warps: 8 epilogue, 1 TMA,
// 1 MMA (even CTA).
//
// Groups start and end at any row, which only the device knows.  Where rows
// are the M index, a tile reads rows past its group (rows of A have no
// influence on one another) and must not write them: a warp whose 32 rows all
// belong to the group writes them with one tensor store, others row by row.
// Where rows are summed, what stands behind the group must not count, and may
// be NaN: the TMA brings a group's last slice to a barrier of its own CTA, the
// producer warp writes zeros over the rows behind the group, in both operands,
// and hands the slice on.
#include "grouped.cuh"

namespace mm {

constexpr int kGmStages = 6;
constexpr int kGmTile = 128 * 64 * 2;                 // 16 KiB: 128 rows x one slice
constexpr int kGmEpiWarps = 8;
constexpr int kGmThreads = 32 * (kGmEpiWarps + 2);
constexpr int kGmWarpProducer = kGmEpiWarps, kGmWarpMma = kGmEpiWarps + 1;
constexpr int kGmStage = 32 * 128;                    // epilogue: 32 rows x 128 bytes per warp
constexpr int kGmSmem = kGmStages * 2 * kGmTile + kGmEpiWarps * kGmStage + 1024 + 256;

// Slices of the summed index per accumulation in TMEM.  The tensor cores cut
// off where they add to the accumulator; a weight gradient, kept in fp32 and
// summed over thousands of rows, adds chunks of 512 rows in fp32 registers.
template <int OP> constexpr int kGmChunk = OP == kGroupedWgrad ? 8 : 1 << 30;

struct GmParams {
  CUtensorMap a, b, out;
  GroupTables g;
  int M;              // wgrad: rows of a dw matrix
  int N;              // columns of the result
  int K;              // forward, dgrad: length of the sum
  int a_blocks, b_blocks;   // the MN-major map has 64-column blocks as a dimension: one box for both
  int out_aligned;    // the result's rows start on 16 bytes: tensor stores
  void* outp;
};

// with the static arrays within the 227 KiB of a block
static_assert(kGmSmem + sizeof(GmTables) + 64 <= 232448, "shared memory budget");

template <int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGmThreads, 1)
grouped_tc_kernel(const __grid_constant__ GmParams P, WsHeader* hdr) {
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kGmStages * kGmTile;
  uint8_t* sEpi = sB + kGmStages * kGmTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + kGmEpiWarps * kGmStage);
  uint64_t* full = bars;                   // [stages] even CTA: both CTAs' bytes
  uint64_t* empty = bars + kGmStages;      // [stages] each CTA: released by the pair's MMAs
  uint64_t* tfull = bars + 2 * kGmStages;  // [2] each CTA: accumulator ready
  uint64_t* tempty = tfull + 2;            // [2] even CTA: both CTAs' epilogues done
  uint64_t* drained = tempty + 2;          // even CTA: all MMAs finished
  uint64_t* part = drained + 1;            // wgrad, each CTA: a group's last slice has landed
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ GmTables s_tab;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = blockIdx.x >> 1, nc = gridDim.x >> 1;
  const int ntn = (P.N + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGmStages; ++s) {
      mbar_init(&full[s], OP == kGroupedWgrad ? 2 : 1);   // wgrad: each CTA's producer arrives
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kGmEpiWarps);
    }
    mbar_init(drained, 1);
    mbar_init(part, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == 0) {
    // tables and operands may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    gm_tables<OP>(P.g, s_tab, ntn);
  }
  if (warp == kGmWarpMma) {
    tmem_alloc_cta2(&s_tmem, 512);
    tmem_relinquish_cta2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int total = OP == kGroupedWgrad ? P.g.E * ((P.M + 255) / 256) * ntn : s_tab.tstart[P.g.E];
  volatile int* abort = &s_abort;

  if (warp == kGmWarpProducer) {
    // ------------------------------------------------ TMA (both CTAs)
    int it = 0, parts = 0;
    bool ok = true;
    for (int j = 0; ok && j * nc < total; ++j) {
      const int tile = gm_index<OP>(j, cluster, nc);
      if (tile >= total) continue;               // the last round's missing tiles
      const GmTile ti = gm_tile<OP>(tile, P.g.E, P.M, P.K, s_tab, ntn, 256, rank);
      const int ncol = ti.n0 + 128 * rank;       // this CTA's half of the columns
      const int nkb = (ti.krows + 63) / 64;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int s = it % kGmStages;
        const uint32_t ph = (it / kGmStages) & 1;
        ok = lane != 0 || mbar_wait(&empty[s], ph ^ 1, abort, hdr, 111);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
        uint8_t* a = sA + s * kGmTile;
        uint8_t* b = sB + s * kGmTile;
        if constexpr (OP == kGroupedWgrad) {
          const int krow = ti.k0 + kb * 64, rows = ti.krows - kb * 64;
          if (rows >= 64) {
            if (lane == 0) {
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 4 * kGmTile);
              else mbar_signal_cluster(fb);
              if (P.a_blocks) {
                tma_load_3d_cta2(a, &P.a, fb, 0, krow, ti.m0 / 64);
              } else {
                tma_load_2d_cta2(a, &P.a, fb, ti.m0, krow);
                tma_load_2d_cta2(a + kGmTile / 2, &P.a, fb, ti.m0 + 64, krow);
              }
              if (P.b_blocks) {
                tma_load_3d_cta2(b, &P.b, fb, 0, krow, ncol / 64);
              } else {
                tma_load_2d_cta2(b, &P.b, fb, ncol, krow);
                tma_load_2d_cta2(b + kGmTile / 2, &P.b, fb, ncol + 64, krow);
              }
            }
          } else {
            if (lane == 0) {
              mbar_arrive_expect_tx(part, 2 * kGmTile);
              if (P.a_blocks) {
                tma_load_3d(a, &P.a, part, 0, krow, ti.m0 / 64);
              } else {
                tma_load_2d(a, &P.a, part, ti.m0, krow);
                tma_load_2d(a + kGmTile / 2, &P.a, part, ti.m0 + 64, krow);
              }
              if (P.b_blocks) {
                tma_load_3d(b, &P.b, part, 0, krow, ncol / 64);
              } else {
                tma_load_2d(b, &P.b, part, ncol, krow);
                tma_load_2d(b + kGmTile / 2, &P.b, part, ncol + 64, krow);
              }
            }
            ok = warp_wait(part, parts & 1, abort, hdr, 117);
            ++parts;
            if (!ok) break;
            // a half tile is 64 rows of 128 bytes: rows [rows, multiple of 16) become zeros
            const int clear = ((rows + 15) / 16 * 16 - rows) * 8;        // 16-byte vectors of a half
            for (int v = lane; v < 4 * clear; v += 32) {
              const int h = v / clear;
              uint8_t* half = (h & 2 ? b : a) + (h & 1) * (kGmTile / 2);
              reinterpret_cast<uint4*>(half + rows * 128)[v - h * clear] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(&full[s]);
              else mbar_arrive_cluster(fb);
            }
          }
        } else if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 4 * kGmTile);
          tma_load_2d_cta2(a, &P.a, fb, kb * 64, ti.m0);
          if constexpr (OP == kGroupedForward) {
            tma_load_3d_cta2(b, &P.b, fb, kb * 64, ncol, ti.e);
          } else if (P.b_blocks) {
            tma_load_4d_cta2(b, &P.b, fb, 0, kb * 64, ncol / 64, ti.e);
          } else {
            tma_load_3d_cta2(b, &P.b, fb, ncol, kb * 64, ti.e);
            tma_load_3d_cta2(b + kGmTile / 2, &P.b, fb, ncol + 64, kb * 64, ti.e);
          }
        }
      }
    }
    if (!ok && lane == 0 && rank == 0) {
      // a wait gave up: the copies in flight land before the block ends
      for (int j = 0; j < kGmStages; ++j) {
        const int i2 = it - 1 - j;
        if (i2 < 0) break;
        mbar_wait(&full[i2 % kGmStages], (i2 / kGmStages) & 1, nullptr, hdr, 112);
      }
    }
    __syncwarp();
  } else if (warp == kGmWarpMma) {
    // ------------------------------------------------ MMA (even CTA)
    if (rank == 0 && lane == 0) {
      constexpr uint32_t kAMn = OP == kGroupedWgrad ? 1u : 0u, kBMn = OP == kGroupedForward ? 0u : 1u;
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256) | (kAMn << 15) | (kBMn << 16);
      int it = 0, used = 0;
      bool ok = true;
      for (int j = 0; ok && j * nc < total; ++j) {
        const int tile = gm_index<OP>(j, cluster, nc);
        if (tile >= total) continue;
        const GmTile ti = gm_tile<OP>(tile, P.g.E, P.M, P.K, s_tab, ntn, 256, 0);
        const int nkb = (ti.krows + 63) / 64;      // 0: an empty group, zeros from the epilogue
        uint32_t d = 0;
        int acc = 0;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const bool first = kb % kGmChunk<OP> == 0;
          if (first) {
            acc = used & 1;
            const uint32_t aph = (used >> 1) & 1;
            ++used;
            if (!mbar_wait(&tempty[acc], aph ^ 1, abort, hdr, 113)) { ok = false; break; }
            tc_fence_after();
            d = tmem + acc * 256;
          }
          const int s = it % kGmStages;
          const uint32_t ph = (it / kGmStages) & 1;
          if (!mbar_wait<OP == kGroupedWgrad>(&full[s], ph, abort, hdr, 114)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * kGmTile);
          const uint32_t b0 = smem_u32(sB + s * kGmTile);
          // wgrad: the steps of 16 rows that hold one of the group's
          const int steps = OP == kGroupedWgrad ? min(4, (ti.krows - kb * 64 + 15) / 16) : 4;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= steps) break;
            const uint64_t ad = kAMn ? smem_desc_sw128_mn(a0 + kk * 2048) : smem_desc_sw128(a0 + kk * 32);
            const uint64_t bd = kBMn ? smem_desc_sw128_mn(b0 + kk * 2048) : smem_desc_sw128(b0 + kk * 32);
            umma_f16_cta2(d, ad, bd, idesc, (!first || kk) ? 1u : 0u);
          }
          umma_commit_cta2_mc(&empty[s], 0x3);
          if (kb + 1 == nkb || (kb + 1) % kGmChunk<OP> == 0) umma_commit_cta2_mc(&tfull[acc], 0x3);
        }
      }
      umma_commit_cta2_mc(drained, 0x1);
      mbar_wait(drained, 0, nullptr, hdr, 115);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (warps 0-7, both CTAs)
    const int quad = warp & 3, half = warp >> 2;
    uint8_t* wstage = sEpi + warp * kGmStage;
    const uint32_t te0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t te1 = mapa_shared(smem_u32(&tempty[1]), 0);
    int used = 0;
    for (int j = 0; j * nc < total; ++j) {
      const int tile = gm_index<OP>(j, cluster, nc);
      if (tile >= total) continue;
      const GmTile ti = gm_tile<OP>(tile, P.g.E, P.M, P.K, s_tab, ntn, 256, rank);
      const int rem = min(32, ti.mrows - quad * 32);            // rows of the group in this warp's 32
      const int col0 = ti.n0 + half * 128;
      const int row = ti.m0 + quad * 32;
      if constexpr (OP == kGroupedWgrad) {
        // the sums of all slices, chunk by chunk in registers
        float sum[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) sum[c] = 0.f;
        const int chunks = ((ti.krows + 63) / 64 + kGmChunk<OP> - 1) / kGmChunk<OP>;
        bool ok = true;
        for (int i = 0; i < chunks; ++i) {
          const int acc = used & 1;
          const uint32_t aph = (used >> 1) & 1;
          ++used;
          ok = warp_wait(&tfull[acc], aph, abort, hdr, 116);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(tb + 16 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 16; ++q) sum[16 * c + q] += __uint_as_float(r[q]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_signal_cluster(acc ? te1 : te0);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = col0 + 32 * c;
          if (rem <= 0 || col >= P.N) continue;    // warp-uniform
          if (lane == 0) bulk_wait_read();         // the previous piece's store has read the stage
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(wstage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_float4(sum[32 * c + 4 * q], sum[32 * c + 4 * q + 1], sum[32 * c + 4 * q + 2], sum[32 * c + 4 * q + 3]);
          if (P.out_aligned) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&P.out, wstage, col, row, ti.e);
              bulk_commit();
            }
          } else {
            // rows that start anywhere: element by element
            __syncwarp();
            float* o = static_cast<float*>(P.outp) + (static_cast<int64_t>(ti.e) * P.M + row) * P.N + col + lane;
            if (col + lane < P.N)
              for (int i = 0; i < rem; ++i)
                o[static_cast<int64_t>(i) * P.N] =
                    *reinterpret_cast<const float*>(wstage + i * 128 + ((((lane >> 2) ^ (i & 7)) << 4) | ((lane & 3) << 2)));
          }
        }
      } else {
        const int acc = used & 1;
        const uint32_t aph = (used >> 1) & 1;
        ++used;
        if (!warp_wait(&tfull[acc], aph, abort, hdr, 116)) break;
        tc_fence_after();
        const bool counts = quad * 32 + lane < ti.mvalid;       // this lane's row is not padding
        const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * 128;
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t lo[32], hi[32];
          tmem_ld_32x32b_x32(tb + c, lo);          // every lane (warp-collective)
          tmem_ld_32x32b_x32(tb + c + 32, hi);
          tmem_ld_wait();
          if (c == 64) {                           // the accumulator is read: the next tile may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_signal_cluster(acc ? te1 : te0);
          }
          if (rem <= 0 || col0 + c >= P.N) continue;            // warp-uniform
          uint32_t pk[32];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            pk[q] = counts ? pack_bf16x2(__uint_as_float(lo[2 * q]), __uint_as_float(lo[2 * q + 1])) : 0u;
            pk[16 + q] = counts ? pack_bf16x2(__uint_as_float(hi[2 * q]), __uint_as_float(hi[2 * q + 1])) : 0u;
          }
          store_rows_bf16(pk, wstage, &P.out, P.outp, P.out_aligned, row, col0 + c, rem, P.N, lane);
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's tensor stores have landed
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kGmWarpMma) tmem_dealloc_cta2(tmem, 512);
}

// Rows of 2-byte elements that start anywhere -> rows of pitch8(cols), zeros
// behind the row; a 16-byte vector a thread, from the two aligned vectors that
// hold it (K = 1001, 16.7 MB: REPITCH us).
__global__ void __launch_bounds__(256)
repitch_kernel(const uint16_t* __restrict__ src, uint4* __restrict__ dst, const int64_t vectors, const int64_t elements,
               const int cols, const int per_row) {
  pdl_enter();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= vectors) return;
  const int64_t row = vectors <= 0xffffffffll ? static_cast<uint32_t>(v) / static_cast<uint32_t>(per_row) : v / per_row;
  const int c = static_cast<int>(v - row * per_row) * 8;
  const int64_t at = row * cols + c;           // first element
  const int64_t base = at & ~int64_t{7};
  uint32_t out[4];
  if (base + 16 <= elements) {
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src + base)), hi = __ldg(reinterpret_cast<const uint4*>(src + base) + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int shift = static_cast<int>(at - base);           // elements, 0..7
    uint32_t u[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) u[j] = shift & 4 ? w[j + 2] : w[j];
    uint32_t t[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) t[j] = shift & 2 ? u[j + 1] : u[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = shift & 1 ? __funnelshift_r(t[j], t[j + 1], 16) : t[j];
  } else {                                     // the tensor ends inside the second vector
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = at + 2 * j < elements ? src[at + 2 * j] : 0u, b = at + 2 * j + 1 < elements ? src[at + 2 * j + 1] : 0u;
      out[j] = a | b << 16;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {                // columns behind the row
    if (c + 2 * j >= cols) out[j] = 0u;
    else if (c + 2 * j + 1 >= cols) out[j] &= 0xffffu;
  }
  dst[v] = make_uint4(out[0], out[1], out[2], out[3]);
}

// =============================================================== host side
cudaError_t launch_repitch(const void* src, void* dst, int64_t rows, int cols, cudaStream_t st) {
  const int per_row = pitch8(cols) / 8;
  const int64_t vectors = rows * per_row, blocks = (vectors + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(repitch_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                                 static_cast<const uint16_t*>(src), static_cast<uint4*>(dst), vectors, rows * cols, cols, per_row);
}

static const CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
static const CUtensorMapSwizzle kSw = CU_TENSOR_MAP_SWIZZLE_128B;

// [rows, cols] K-major, rows of `pitch` elements: box 64 x 128.
static bool map_kmajor(CUtensorMap* m, const void* p, int cols, int64_t rows, int64_t pitch) {
  const uint64_t d[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, s[1] = {static_cast<uint64_t>(pitch) * 2};
  const uint32_t b[2] = {64, 128};
  return make_map(m, kBf, 2, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [E, N, K] K-major: box 64 x 128 x 1.
static bool map_weights(CUtensorMap* m, const void* p, int K, int64_t pitch, int N, int E) {
  const uint64_t d[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t s[2] = {static_cast<uint64_t>(pitch) * 2, static_cast<uint64_t>(pitch) * 2 * N};
  const uint32_t b[3] = {64, 128, 1};
  return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [E, N, K] with K as the operand's M / N index: boxes of 64 columns x 64 rows,
// two at once where the columns are whole blocks of 64.
static bool map_weights_mn(CUtensorMap* m, const void* p, int K, int64_t pitch, int N, int E, bool blocks) {
  const uint64_t row = static_cast<uint64_t>(pitch) * 2;
  if (blocks) {
    const uint64_t d[4] = {64, static_cast<uint64_t>(N), static_cast<uint64_t>(K / 64), static_cast<uint64_t>(E)};
    const uint64_t s[3] = {row, 128, row * N};
    const uint32_t b[4] = {64, 64, 2, 1};
    return make_map(m, kBf, 4, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
  }
  const uint64_t d[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t s[2] = {row, row * N};
  const uint32_t b[3] = {64, 64, 1};
  return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [rows, cols] with the rows as the summed index: boxes of 64 columns x 64
// rows, two at once where the columns are whole blocks of 64.
static bool map_rows_mn(CUtensorMap* m, const void* p, int cols, int64_t rows, int64_t pitch, bool blocks) {
  const uint64_t row = static_cast<uint64_t>(pitch) * 2;
  if (blocks) {
    const uint64_t d[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols / 64)};
    const uint64_t s[2] = {row, 128};
    const uint32_t b[3] = {64, 64, 2};
    return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
  }
  const uint64_t d[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, s[1] = {row};
  const uint32_t b[2] = {64, 64};
  return make_map(m, kBf, 2, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// Weight gradients fp32 [E, N, K]: store boxes of 32 x 32.
static bool map_out_weights(CUtensorMap* m, void* p, int K, int N, int E) {
  const uint64_t d[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t s[2] = {static_cast<uint64_t>(K) * 4, static_cast<uint64_t>(K) * 4 * N};
  const uint32_t b[3] = {32, 32, 1};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}

template <int OP>
static cudaError_t gm_launch(const GmParams& p, int64_t tiles, WsHeader* hdr, cudaStream_t st) {
  auto fn = grouped_tc_kernel<OP>;
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), kGmSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms() / 2));
  return launch_dependent_kernel(fn, dim3(static_cast<unsigned>(2 * pairs)), dim3(kGmThreads), kGmSmem, st, p, hdr);
}

cudaError_t launch_grouped_tc(int op, const GroupedArgs& a, WsHeader* hdr, cudaStream_t st) {
  GmParams p;
  memset(&p, 0, sizeof(p));
  p.g = a.g;
  p.outp = a.out;
  const int64_t kp = pitch8(a.K), np = pitch8(a.N);
  bool ok;
  if (op == kGroupedWgrad) {
    p.M = a.N;
    p.N = a.K;
    p.a_blocks = a.N % 64 == 0;
    p.b_blocks = a.K % 64 == 0;
    p.out_aligned = a.K % 4 == 0;
    ok = map_rows_mn(&p.a, a.dys, a.N, a.g.rows, np, p.a_blocks) &&
         map_rows_mn(&p.b, a.xs, a.K, a.g.rows, kp, p.b_blocks) &&
         (!p.out_aligned || map_out_weights(&p.out, a.out, a.K, a.N, a.g.E));
    const int64_t tiles = a.g.E * ((a.N + 255) / 256) * static_cast<int64_t>((a.K + 255) / 256);
    return ok ? gm_launch<kGroupedWgrad>(p, tiles, hdr, st) : cudaErrorInvalidValue;
  }
  const bool fwd = op == kGroupedForward;
  p.N = fwd ? a.N : a.K;
  p.K = fwd ? a.K : a.N;
  p.out_aligned = p.N % 8 == 0;
  p.b_blocks = !fwd && a.K % 64 == 0;
  ok = fwd ? map_kmajor(&p.a, a.xs, a.K, a.g.rows, kp) && map_weights(&p.b, a.w, a.K, kp, a.N, a.g.E)
           : map_kmajor(&p.a, a.dys, a.N, a.g.rows, np) && map_weights_mn(&p.b, a.w, a.K, kp, a.N, a.g.E, p.b_blocks);
  ok = ok && (!p.out_aligned || map_out_rows(&p.out, a.out, p.N, a.g.rows, 64));
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = row_tiles256(a.g) * ((p.N + 255) / 256);
  return fwd ? gm_launch<kGroupedForward>(p, tiles, hdr, st) : gm_launch<kGroupedDgrad>(p, tiles, hdr, st);
}

}  // namespace mm
