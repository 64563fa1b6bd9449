// Experts' products of bf16 and fp32 rows on the 5th-generation tensor cores,
// fp32 accumulators in TMEM:
//   forward  ys = xs w[e]^T       A = xs  [rows, K]  K-major,   B = w[e] [N, K] K-major
//   dgrad    dxs = dys w[e]       A = dys [rows, N]  K-major,   B = w[e] with its K contiguous (MN-major)
//   wgrad    dw[e] = dys^T xs     A = dys, B = xs, both MN-major; the summed index is the group's rows
//
// A CTA pair makes a tile of 256 x 256, or 256 x 128 where those fit into half
// the pairs of SMs (tcgen05.mma.cta_group::2: 128 rows of A and half of B in
// each CTA's shared memory), in slices of 64 of the summed index through a
// ring of six stages; two accumulators, so that the epilogue
// of one tile runs under the products of the next.  Warps: 8 epilogue, 1 TMA,
// 1 MMA (even CTA; it goes through its loop as a whole and issues from one
// lane, which keeps descriptors in uniform registers).
//
// Groups start and end at any row, which only the device knows.  Where rows
// are the M index, a tile reads rows past its group (rows of A have no
// influence on one another) and must not write them: a warp whose 32 rows all
// belong to the group writes them with one tensor store, others row by row.
// Where rows are summed, what stands behind the group must not count, and may
// be NaN: the TMA brings a group's last slice to a barrier of its own CTA, the
// producer warp writes zeros over the rows behind the group, in both operands,
// and hands the slice on.
//
// fp32 operands come as three bf16 planes (split_kernel): 2^24 x = h + m + l, each
// the nearest bf16 of what the ones before leave, so that 24 bits are kept, of
// the smallest numbers too; of the nine products the three below 2^-25 are left
// out.  h h' adds up in one accumulator and the five smaller products in the
// other; both are added in fp32 registers every 256 of the summed index, and the
// result is scaled back by 2^-48.  What is not finite on the way (large operands,
// sums of 2^80 and more) sets a flag, and the CUDA cores do the operation.
//
// Few tiles with a long sum are cut into `splits` parts of the sum, each an
// fp32 tile of its own in the workspace, and join_kernel adds them in order.
#include "grouped.cuh"

namespace mm {

constexpr int kGmRing = 6;                            // tiles of A (and of B) in the ring
constexpr int kGmTile = 128 * 64 * 2;                 // 16 KiB: 128 rows x one slice
constexpr int kGmEpiWarps = 8;
constexpr int kGmThreads = 32 * (kGmEpiWarps + 2);
constexpr int kGmWarpProducer = kGmEpiWarps, kGmWarpMma = kGmEpiWarps + 1;
constexpr int kGmStage = 32 * 128;                    // epilogue: 32 rows x 128 bytes per warp
constexpr int kGmSmem = kGmRing * 2 * kGmTile + kGmEpiWarps * kGmStage + 1024 + 256;
// with the static arrays within the 227 KiB of a block
static_assert(kGmSmem + sizeof(GmTables) + 64 <= 232448, "shared memory budget");

// Slices of the summed index per accumulation in TMEM.  The tensor cores cut
// off where they add to the accumulator; results in fp32 add chunks of 256 in
// fp32 registers.  Relative to their root mean square, results over 2048 and
// more are 2.4e-7 off (3.2e-7 where all terms have one sign), with chunks of 512
// 4.8e-7 (7.1e-7), with 128 1.4e-7 (1.5e-7).  fp32 products, which have one pair of accumulators, take
// 3 to 5% more time than with 512 and 128 takes 8 to 10% more again; weight gradients of bf16 rows, which have two
// by turns, as long as with 512, with 128 12% longer (T = 16384, 2432 -> 768).
template <bool F32> constexpr int kGmChunk = F32 ? 4 : 1 << 30;

struct GmParams {
  CUtensorMap a, b, out;
  GroupTables g;
  int M;              // wgrad: rows of a dw matrix
  int N;              // columns of the result
  int nt;             // columns of a tile: 256 or 128
  int K;              // forward, dgrad: length of the sum
  int a_blocks, b_blocks;   // the MN-major map has 64-column blocks as a dimension: so many in a box
  int a_plane, b_plane;     // three planes: rows (b of forward and dgrad: experts) from one to the next
  int splits;         // parts of the sum
  int out_plane;      // rows (wgrad: experts) of a part's result
  int out_aligned;    // the result's rows start on 16 bytes: tensor stores
  void* outp;
  int64_t ldo;        // elements from one row of the result to the next
  const int* skip;    // not null: nothing is done where it holds something
  int* over;          // not null: set where a result is not finite
};

// OP, PLANES: 1 (bf16) or 3 (fp32).  F32: the result, or its parts, in fp32.
template <int OP, int PLANES, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGmThreads, 1)
grouped_tc_kernel(const __grid_constant__ GmParams P, WsHeader* hdr) {
  constexpr int kStages = kGmRing / PLANES;
  constexpr int kAccs = PLANES == 1 ? 2 : 1;   // accumulators by turns; three planes: one pair of them
  constexpr int kStep = PLANES * kGmTile;      // bytes of an operand's stage
  constexpr bool kWgrad = OP == kGroupedWgrad;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kGmRing * kGmTile;
  uint8_t* sEpi = sB + kGmRing * kGmTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + kGmEpiWarps * kGmStage);
  uint64_t* full = bars;                   // [stages] even CTA: both CTAs' bytes
  uint64_t* empty = bars + kStages;        // [stages] each CTA: released by the pair's MMAs
  uint64_t* tfull = bars + 2 * kStages;    // [2] each CTA: accumulator ready
  uint64_t* tempty = tfull + 2;            // [2] even CTA: both CTAs' epilogues done
  uint64_t* drained = tempty + 2;          // even CTA: all MMAs finished
  uint64_t* part = drained + 1;            // wgrad, each CTA: a group's last slice has landed
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_total;
  __shared__ GmTables s_tab;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = blockIdx.x >> 1, nc = gridDim.x >> 1;
  const int ntn = (P.N + P.nt - 1) / P.nt;
  const int b_bytes = P.nt / 2 * 128;          // of one tile of B in a CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kWgrad ? 2 : 1);   // wgrad: each CTA's producer arrives
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
    __syncwarp();
    if (lane == 0) {
      const bool none = P.skip != nullptr && *P.skip != 0;
      s_total = none ? 0 : P.splits * (kWgrad ? P.g.E * ((P.M + 255) / 256) * ntn : s_tab.tstart[P.g.E]);
    }
  }
  if (warp == kGmWarpMma) {
    tmem_alloc_cta2(&s_tmem, 512);
    tmem_relinquish_cta2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int total = s_total;
  volatile int* abort = &s_abort;
  // the slices [k0, k1) of a tile's part of the sum
  auto slices = [&](const GmTile& ti, int tile, int& k0, int& k1) {
    const int nkb = (ti.krows + 63) / 64, sp = tile % P.splits;
    k0 = static_cast<int>(static_cast<int64_t>(nkb) * sp / P.splits);
    k1 = static_cast<int>(static_cast<int64_t>(nkb) * (sp + 1) / P.splits);
  };

  if (warp == kGmWarpProducer) {
    // ------------------------------------------------ TMA (both CTAs)
    int it = 0, parts = 0;
    bool ok = true;
    for (int j = 0; ok && j * nc < total; ++j) {
      const int tile = gm_index<OP>(j, cluster, nc);
      if (tile >= total) continue;               // the last round's missing tiles
      const GmTile ti = gm_tile<OP>(tile / P.splits, P.g.E, P.M, P.K, s_tab, ntn, P.nt, rank);
      const int ncol = ti.n0 + P.nt / 2 * rank;  // this CTA's half of the columns
      int k0, k1;
      slices(ti, tile, k0, k1);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % kStages;
        const uint32_t ph = (it / kStages) & 1;
        ok = lane != 0 || mbar_wait(&empty[s], ph ^ 1, abort, hdr, 111);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
        uint8_t* a = sA + s * kStep;
        uint8_t* b = sB + s * kStep;
        if constexpr (kWgrad) {
          const int krow = ti.k0 + kb * 64, rows = ti.krows - kb * 64;
          if (rows >= 64) {
            if (lane == 0) {
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * PLANES * (kGmTile + b_bytes));
              else mbar_signal_cluster(fb);
#pragma unroll
              for (int p = 0; p < PLANES; ++p) {
                uint8_t *ap = a + p * kGmTile, *bp = b + p * kGmTile;
                const int ar = krow + p * P.a_plane, br = krow + p * P.b_plane;
                if (P.a_blocks) {
                  tma_load_3d_cta2(ap, &P.a, fb, 0, ar, ti.m0 / 64);
                } else {
                  tma_load_2d_cta2(ap, &P.a, fb, ti.m0, ar);
                  tma_load_2d_cta2(ap + kGmTile / 2, &P.a, fb, ti.m0 + 64, ar);
                }
                if (P.b_blocks) {
                  tma_load_3d_cta2(bp, &P.b, fb, 0, br, ncol / 64);
                } else {
                  tma_load_2d_cta2(bp, &P.b, fb, ncol, br);
                  if (P.nt == 256) tma_load_2d_cta2(bp + kGmTile / 2, &P.b, fb, ncol + 64, br);
                }
              }
            }
          } else {
            if (lane == 0) {
              mbar_arrive_expect_tx(part, PLANES * (kGmTile + b_bytes));
#pragma unroll
              for (int p = 0; p < PLANES; ++p) {
                uint8_t *ap = a + p * kGmTile, *bp = b + p * kGmTile;
                const int ar = krow + p * P.a_plane, br = krow + p * P.b_plane;
                if (P.a_blocks) {
                  tma_load_3d(ap, &P.a, part, 0, ar, ti.m0 / 64);
                } else {
                  tma_load_2d(ap, &P.a, part, ti.m0, ar);
                  tma_load_2d(ap + kGmTile / 2, &P.a, part, ti.m0 + 64, ar);
                }
                if (P.b_blocks) {
                  tma_load_3d(bp, &P.b, part, 0, br, ncol / 64);
                } else {
                  tma_load_2d(bp, &P.b, part, ncol, br);
                  if (P.nt == 256) tma_load_2d(bp + kGmTile / 2, &P.b, part, ncol + 64, br);
                }
              }
            }
            ok = warp_wait(part, parts & 1, abort, hdr, 117);
            ++parts;
            if (!ok) break;
            // a half tile is 64 rows of 128 bytes: rows [rows, multiple of 16) become zeros
            const int clear = ((rows + 15) / 16 * 16 - rows) * 8;        // 16-byte vectors of a half
            for (int v = lane; v < 4 * PLANES * clear; v += 32) {
              const int h = v / clear;
              uint8_t* half = (h & 1 ? b : a) + (h >> 1) * (kGmTile / 2);
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
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * PLANES * (kGmTile + b_bytes));
#pragma unroll
          for (int p = 0; p < PLANES; ++p) {
            uint8_t *ap = a + p * kGmTile, *bp = b + p * kGmTile;
            const int e = ti.e + p * P.b_plane;
            tma_load_2d_cta2(ap, &P.a, fb, kb * 64, ti.m0 + p * P.a_plane);
            if constexpr (OP == kGroupedForward) {
              tma_load_3d_cta2(bp, &P.b, fb, kb * 64, ncol, e);
            } else if (P.b_blocks) {
              tma_load_4d_cta2(bp, &P.b, fb, 0, kb * 64, ncol / 64, e);
            } else {
              tma_load_3d_cta2(bp, &P.b, fb, ncol, kb * 64, e);
              if (P.nt == 256) tma_load_3d_cta2(bp + kGmTile / 2, &P.b, fb, ncol + 64, kb * 64, e);
            }
          }
        }
      }
    }
    if (!ok && lane == 0 && rank == 0) {
      // a wait gave up: the copies in flight land before the block ends
      for (int j = 0; j < kStages; ++j) {
        const int i2 = it - 1 - j;
        if (i2 < 0) break;
        mbar_wait(&full[i2 % kStages], (i2 / kStages) & 1, nullptr, hdr, 112);
      }
    }
    __syncwarp();
  } else if (warp == kGmWarpMma) {
    // ------------------------------------------------ MMA (even CTA)
    if (rank == 0) {
      constexpr uint32_t kAMn = kWgrad ? 1u : 0u, kBMn = OP == kGroupedForward ? 0u : 1u;
      const uint32_t idesc = idesc_bf16_f32(256, 0) | (static_cast<uint32_t>(P.nt >> 3) << 17) | (kAMn << 15) | (kBMn << 16);
      constexpr uint64_t kAK = kAMn ? 2048 / 16 : 32 / 16, kBK = kBMn ? 2048 / 16 : 32 / 16;   // 16 of the summed index
      const bool leader = elect_one();
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const int tiles = __shfl_sync(0xffffffffu, total, 0);
      const uint64_t da = kAMn ? smem_desc_sw128_mn(smem_u32(sA)) : smem_desc_sw128(smem_u32(sA));
      const uint64_t db = kBMn ? smem_desc_sw128_mn(smem_u32(sB)) : smem_desc_sw128(smem_u32(sB));
      int s = 0, used = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int j = 0; ok && j * nc < tiles; ++j) {
        const int tile = gm_index<OP>(j, cluster, nc);
        if (tile >= tiles) continue;
        const GmTile ti = gm_tile<OP>(tile / P.splits, P.g.E, P.M, P.K, s_tab, ntn, P.nt, 0);
        int k0, k1;
        slices(ti, tile, k0, k1);                  // none: the epilogue writes zeros
        k0 = __shfl_sync(0xffffffffu, k0, 0);
        k1 = __shfl_sync(0xffffffffu, k1, 0);
        const int krows = __shfl_sync(0xffffffffu, ti.krows, 0);
        int acc = 0;
        for (int kb = k0; kb < k1; ++kb) {
          const bool first = (kb - k0) % kGmChunk<F32> == 0;
          if (first) {
            acc = used % kAccs;
            ok = warp_wait<true>(&tempty[acc], ((used / kAccs) & 1) ^ 1, abort, hdr, 113);
            if (!ok) break;
            ++used;
            tc_fence_after();
          }
          ok = warp_wait<kWgrad>(&full[s], ph, abort, hdr, 114);
          if (!ok) break;
          tc_fence_after();
          // wgrad: the steps of 16 rows that hold one of the group's
          const int steps = kWgrad ? min(4, (krows - kb * 64 + 15) / 16) : 4;
          const bool last = kb + 1 == k1 || (kb + 1 - k0) % kGmChunk<F32> == 0;
          if (leader) {
            const uint64_t as = da + static_cast<uint64_t>(s * (kStep / 16)), bs = db + static_cast<uint64_t>(s * (kStep / 16));
            if constexpr (PLANES == 1) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < steps)
                  umma_f16_cta2(base + acc * 256, as + kk * kAK, bs + kk * kBK, idesc, (!first || kk) ? 1u : 0u);
            } else {
              // the products of planes pa and pb: h h' in the first accumulator, the others in the second
              constexpr int kPa[6] = {0, 2, 0, 1, 1, 0}, kPb[6] = {0, 0, 2, 1, 0, 1};
#pragma unroll
              for (int c = 0; c < 6; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  if (kk < steps)
                    umma_f16_cta2(base + (c ? 256 : 0), as + kPa[c] * (kGmTile / 16) + kk * kAK,
                                  bs + kPb[c] * (kGmTile / 16) + kk * kBK, idesc, (!first || kk || c > 1) ? 1u : 0u);
            }
            umma_commit_cta2_mc(&empty[s], 0x3);
            if (last) umma_commit_cta2_mc(&tfull[acc], 0x3);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (leader) umma_commit_cta2_mc(drained, 0x1);
      __syncwarp();
      warp_wait(drained, 0, nullptr, hdr, 115);
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
      const GmTile ti = gm_tile<OP>(tile / P.splits, P.g.E, P.M, P.K, s_tab, ntn, P.nt, rank);
      const int rem = min(32, ti.mrows - quad * 32);            // rows of the group in this warp's 32
      const bool counts = quad * 32 + lane < ti.mvalid;         // this lane's row is not padding
      const int hc = P.nt / 2;                     // columns of this warp's half
      const int col0 = ti.n0 + half * hc;
      const int row = ti.m0 + quad * 32;
      if constexpr (F32) {
        // the sums of all slices, chunk by chunk in registers
        float sum[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) sum[c] = 0.f;
        int k0, k1;
        slices(ti, tile, k0, k1);
        bool ok = true;
        for (int kb = k0; kb < k1; kb += kGmChunk<F32>) {
          const int acc = used % kAccs;
          ok = warp_wait(&tfull[acc], (used / kAccs) & 1, abort, hdr, 116);
          if (!ok) break;
          ++used;
          tc_fence_after();
          const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * hc;
#pragma unroll
          for (int h = 0; h < (PLANES == 1 ? 1 : 2); ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (16 * c >= hc) break;
              uint32_t r[16];
              tmem_ld_32x32b_x16(tb + (PLANES == 1 ? 0 : 256 - 256 * h) + 16 * c, r);    // the small products first
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 16; ++q) sum[16 * c + q] += __uint_as_float(r[q]);
            }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_signal_cluster(acc ? te1 : te0);
        }
        if (!ok) break;
        if (PLANES == 3 && P.splits == 1) {
          bool over = false;
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            over |= !(fabsf(sum[c]) < INFINITY);
            sum[c] *= kSplitUnscale;
          }
          if (over && counts) *P.over = 1;
        }
        const int sp = tile % P.splits;
        const int64_t orow = kWgrad ? (static_cast<int64_t>(ti.e) + static_cast<int64_t>(sp) * P.out_plane) * P.M + row
                                    : row + static_cast<int64_t>(sp) * P.out_plane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = col0 + 32 * c;
          if (rem <= 0 || 32 * c >= hc || col >= P.N) continue;    // warp-uniform
          if (lane == 0) bulk_wait_read();         // the previous piece's store has read the stage
          __syncwarp();
          // 128-byte rows, 16-byte chunk q of row i at chunk q ^ (i & 7)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(wstage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                counts ? make_float4(sum[32 * c + 4 * q], sum[32 * c + 4 * q + 1], sum[32 * c + 4 * q + 2], sum[32 * c + 4 * q + 3])
                       : make_float4(0.f, 0.f, 0.f, 0.f);
          if (P.out_aligned && (kWgrad || rem == 32)) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if constexpr (kWgrad) tma_store_3d(&P.out, wstage, col, row, ti.e + sp * P.out_plane);
              else tma_store_2d(&P.out, wstage, col, static_cast<int>(orow));
              bulk_commit();
            }
            continue;
          }
          __syncwarp();
          float* o = static_cast<float*>(P.outp) + orow * P.ldo + col;
          if (P.out_aligned) {
            // a group's ragged end: 16 bytes a lane, four rows at once
            if (col + 4 * (lane & 7) < P.N)
              for (int i = lane >> 3; i < rem; i += 4)
                *reinterpret_cast<float4*>(o + i * P.ldo + 4 * (lane & 7)) =
                    *reinterpret_cast<const float4*>(wstage + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
          } else if (col + lane < P.N) {
            // rows that start anywhere: element by element
            for (int i = 0; i < rem; ++i)
              o[i * P.ldo + lane] = *reinterpret_cast<const float*>(wstage + i * 128 + ((((lane >> 2) ^ (i & 7)) << 4) | ((lane & 3) << 2)));
          }
        }
      } else {
        const int acc = used & 1;
        const uint32_t aph = (used >> 1) & 1;
        ++used;
        if (!warp_wait(&tfull[acc], aph, abort, hdr, 116)) break;
        tc_fence_after();
        const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * hc;
#pragma unroll 1
        for (int c = 0; c < hc; c += 64) {
          uint32_t lo[32], hi[32];
          tmem_ld_32x32b_x32(tb + c, lo);          // every lane (warp-collective)
          tmem_ld_32x32b_x32(tb + c + 32, hi);
          tmem_ld_wait();
          if (c + 64 == hc) {                      // the accumulator is read: the next tile may have it
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

// Whether row r holds an assignment (1), is padding of a group (0) or lies
// outside every group (-1).  Called by a full warp.
__device__ __forceinline__ int row_kind(const GroupTables& g, int64_t r) {
  if (g.offsets == nullptr) return 1;
  const int lane = threadIdx.x & 31;
  int kind = -1;
  for (int e = lane; e < g.E; e += 32) {
    const GroupSpan s = group_span(g, e);
    if (r >= s.r0 && r < s.r1) kind = r < s.r0 + s.n ? 1 : 0;
  }
  const uint32_t valid = __ballot_sync(0xffffffffu, kind == 1), pad = __ballot_sync(0xffffffffu, kind == 0);
  return valid ? 1 : pad ? 0 : -1;
}

// fp32 rows times 2^24 as three planes of bf16, [3, rows, pitch8(cols)]; rows that hold no
// assignment as zeros.  *flag is set where a value has no such planes.  A warp
// a row, the tensors' rows one after the other.
__global__ void __launch_bounds__(256)
split_kernel(const SplitTensors S, const GroupTables g, int* flag) {
  pdl_enter();
  int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  int i = 0;
  while (i < S.n && r >= S.t[i].rows) r -= S.t[i++].rows;
  if (i == S.n) return;
  const SplitTensor T = S.t[i];
  if (T.per_group && g.offsets != nullptr && group_span(g, static_cast<int>(r / T.per_group)).n == 0) return;
  const bool valid = T.per_group || row_kind(g, r) == 1;
  const int per = (T.cols + 7) / 8, lane = threadIdx.x & 31;
  const float* s = static_cast<const float*>(T.src) + r * T.cols;
  uint4* dst = static_cast<uint4*>(T.dst) + r * per;
  const bool vec = T.cols % 4 == 0;            // rows start on 16 bytes
  bool bad = false;
  for (int v0 = lane; v0 < per; v0 += 64) {    // two vectors of eight columns a lane
    float x[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const int c = 8 * (v0 + 32 * h) + j;
        if (vec) {
          const float4 f = valid && c < T.cols ? __ldg(reinterpret_cast<const float4*>(s + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[h][j] = f.x; x[h][j + 1] = f.y; x[h][j + 2] = f.z; x[h][j + 3] = f.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[h][j + e] = valid && c + e < T.cols ? __ldg(s + c + e) : 0.f;
        }
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 p[3];
      split_vector(x[h], p);
#pragma unroll
      for (int e = 0; e < 8; ++e) bad |= !(fabsf(x[h][e]) < kSplitMost);
      if (v0 + 32 * h < per)
#pragma unroll
        for (int q = 0; q < 3; ++q) dst[q * T.rows * per + v0 + 32 * h] = p[q];
    }
  }
  if (bad) *flag = 1;
}

// out[r, c] = the sum over the parts, in order, times `scale`, in T; padding rows
// zero, rows outside the groups left alone; *over (or null) is set where a sum is
// not finite.  A warp a row.
template <typename T>
__global__ void __launch_bounds__(256)
join_kernel(const float* __restrict__ parts, T* __restrict__ out, const GroupTables g, const int64_t rows, const int cols,
            const int pitch, const int splits, const float scale, const int* skip, int* over) {
  pdl_enter();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (r >= rows || (skip != nullptr && *skip != 0)) return;
  const int kind = row_kind(g, r);
  if (kind < 0) return;
  const bool vec = cols % 4 == 0;
  for (int c = 4 * (threadIdx.x & 31); c < cols; c += 128) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kind == 1)
      for (int s = 0; s < splits; ++s) {
        const float4 v = *reinterpret_cast<const float4*>(parts + (s * rows + r) * pitch + c);
        sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
      }
    T* o = out + r * cols + c;
    float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (over != nullptr && c + i < cols && !(fabsf(v[i]) < INFINITY)) *over = 1;
      v[i] *= scale;
    }
    if (vec) {
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      else *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < cols) o[i] = static_cast<T>(v[i]);
    }
  }
}

// Rows of 2-byte elements that start anywhere -> rows of pitch8(cols), zeros
// behind the row; a 16-byte vector a thread, from the two aligned vectors that
// hold it.  per_group: rows of a group's matrix, left out where the group has
// no rows; 0: every row.
__global__ void __launch_bounds__(256)
repitch_kernel(const uint16_t* __restrict__ src, uint4* __restrict__ dst, const int64_t vectors, const int64_t elements,
               const int cols, const int per_row, const GroupTables g, const int per_group) {
  pdl_enter();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= vectors) return;
  const int64_t row = vectors <= 0xffffffffll ? static_cast<uint32_t>(v) / static_cast<uint32_t>(per_row) : v / per_row;
  if (per_group && group_span(g, static_cast<int>(row / per_group)).n == 0) return;
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
cudaError_t launch_repitch(const void* src, void* dst, int64_t rows, int cols, const GroupTables& g, int per_group,
                           cudaStream_t st) {
  const int per_row = pitch8(cols) / 8;
  const int64_t vectors = rows * per_row, blocks = (vectors + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(repitch_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                                 static_cast<const uint16_t*>(src), static_cast<uint4*>(dst), vectors, rows * cols, cols, per_row, g,
                                 g.offsets ? per_group : 0);
}

static const CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
static const CUtensorMapSwizzle kSw = CU_TENSOR_MAP_SWIZZLE_128B;

// [rows, cols] K-major, rows of `pitch` elements: box 64 x 128.
static bool map_kmajor(CUtensorMap* m, const void* p, int cols, int64_t rows, int64_t pitch) {
  const uint64_t d[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, s[1] = {static_cast<uint64_t>(pitch) * 2};
  const uint32_t b[2] = {64, 128};
  return make_map(m, kBf, 2, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [E, N, K] K-major: box 64 x `rows` x 1.
static bool map_weights(CUtensorMap* m, const void* p, int K, int64_t pitch, int N, int E, int rows) {
  const uint64_t d[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t s[2] = {static_cast<uint64_t>(pitch) * 2, static_cast<uint64_t>(pitch) * 2 * N};
  const uint32_t b[3] = {64, static_cast<uint32_t>(rows), 1};
  return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [E, N, K] with K as the operand's M / N index: boxes of 64 columns x 64 rows,
// `blocks` of them at once where the columns are whole blocks of 64 (else 0).
static bool map_weights_mn(CUtensorMap* m, const void* p, int K, int64_t pitch, int N, int E, int blocks) {
  const uint64_t row = static_cast<uint64_t>(pitch) * 2;
  if (blocks) {
    const uint64_t d[4] = {64, static_cast<uint64_t>(N), static_cast<uint64_t>(K / 64), static_cast<uint64_t>(E)};
    const uint64_t s[3] = {row, 128, row * N};
    const uint32_t b[4] = {64, 64, static_cast<uint32_t>(blocks), 1};
    return make_map(m, kBf, 4, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
  }
  const uint64_t d[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t s[2] = {row, row * N};
  const uint32_t b[3] = {64, 64, 1};
  return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// [rows, cols] with the rows as the summed index: boxes of 64 columns x 64
// rows, `blocks` of them at once where the columns are whole blocks of 64 (else 0).
static bool map_rows_mn(CUtensorMap* m, const void* p, int cols, int64_t rows, int64_t pitch, int blocks) {
  const uint64_t row = static_cast<uint64_t>(pitch) * 2;
  if (blocks) {
    const uint64_t d[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols / 64)};
    const uint64_t s[2] = {row, 128};
    const uint32_t b[3] = {64, 64, static_cast<uint32_t>(blocks)};
    return make_map(m, kBf, 3, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
  }
  const uint64_t d[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, s[1] = {row};
  const uint32_t b[2] = {64, 64};
  return make_map(m, kBf, 2, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}
// fp32 [planes, rows, cols], rows of `pitch` elements: store boxes of 32 x 32.
static bool map_out_f32(CUtensorMap* m, void* p, int cols, int64_t pitch, int64_t rows, int64_t planes) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(planes)};
  const uint64_t s[2] = {static_cast<uint64_t>(pitch) * 4, static_cast<uint64_t>(pitch) * 4 * rows};
  const uint32_t b[3] = {32, 32, 1};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, planes ? 3 : 2, reinterpret_cast<uint64_t>(p), d, s, b, kSw);
}

template <int OP, int PLANES, bool F32>
static cudaError_t gm_launch(const GmParams& p, int64_t tiles, WsHeader* hdr, cudaStream_t st) {
  auto fn = grouped_tc_kernel<OP, PLANES, F32>;
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), kGmSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms() / 2));
  return launch_dependent_kernel(fn, dim3(static_cast<unsigned>(2 * pairs)), dim3(kGmThreads), kGmSmem, st, p, hdr);
}

// Tiles of a call, and the parts that its sums are cut into: as many as the
// pairs of SMs have room for, where that saves more slices in a row than the
// second launch costs.  A slice takes 0.3 us, of three planes six times that;
// a part has 2.4 us of them at least (K = 8192, N = 512, 300 rows 47 -> 17 us;
// wgrad 768 x 768 over 16384 rows 107 -> 29 us; with 12 slices saved, 10 us
// became 15).
static int64_t gm_row_tiles(int op, const GroupTables& g, int N) {
  return op == kGroupedWgrad ? g.E * static_cast<int64_t>((N + 255) / 256) : row_tiles256(g);
}
static int64_t gm_tiles(int op, const GroupTables& g, int K, int N, int nt) {
  return gm_row_tiles(op, g, N) * (((op == kGroupedForward ? N : K) + nt - 1) / nt);
}
static int gm_columns(int op, const GroupTables& g, int K, int N) {
  return gm_columns(gm_row_tiles(op, g, N), op == kGroupedForward ? N : K);
}
int grouped_splits(int op, const GroupTables& g, int K, int N, int planes) {
  const int64_t slices = op == kGroupedWgrad ? g.rows / (64 * static_cast<int64_t>(g.E))
                                             : ((op == kGroupedForward ? K : N) + 63) / 64;
  const int64_t room = (num_sms() / 2) / std::max<int64_t>(1, gm_tiles(op, g, K, N, gm_columns(op, g, K, N)));
  const int64_t weight = planes == 3 ? 6 : 1;
  const int64_t parts = std::min(room, std::min(slices, slices * weight / 8));
  return parts > 1 && (slices - slices / parts) * weight >= 24 ? static_cast<int>(parts) : 1;
}
static int pitch4(int n) { return (n + 3) / 4 * 4; }
size_t grouped_parts_bytes(int op, const GroupTables& g, int K, int N, int splits) {
  if (splits < 2) return 0;
  const int64_t rows = op == kGroupedWgrad ? static_cast<int64_t>(g.E) * N : g.rows;
  return 4 * static_cast<size_t>(splits) * rows * pitch4(op == kGroupedForward ? N : K);
}

// One operand set: bf16 as given (planes 1), or three planes of bf16.
template <int PLANES>
static cudaError_t gm_run(int op, const GroupedArgs& a, const GroupedTcExtras& x, WsHeader* hdr, cudaStream_t st) {
  GmParams p;
  memset(&p, 0, sizeof(p));
  const bool fwd = op == kGroupedForward, wgrad = op == kGroupedWgrad, parts = x.splits > 1;
  const int64_t kp = pitch8(a.K), np = pitch8(a.N), R = a.g.rows;
  const int E = a.g.E;
  p.g = a.g;
  p.M = wgrad ? a.N : 0;
  p.N = fwd ? a.N : a.K;
  p.nt = gm_columns(op, a.g, a.K, a.N);
  p.K = fwd ? a.K : a.N;
  p.splits = x.splits;
  p.skip = x.skip;
  p.over = x.over;
  p.a_plane = static_cast<int>(R);
  p.b_plane = wgrad ? static_cast<int>(R) : E;
  const bool f32 = wgrad || PLANES == 3 || parts;
  p.outp = parts ? x.parts : a.out;
  p.ldo = parts ? pitch4(p.N) : p.N;
  p.out_plane = wgrad ? E : static_cast<int>(R);
  p.out_aligned = p.ldo % (f32 ? 4 : 8) == 0;
  bool ok;
  if (wgrad) {
    p.a_blocks = a.N % 64 == 0 ? 2 : 0;
    p.b_blocks = a.K % 64 == 0 ? p.nt / 128 : 0;
    ok = map_rows_mn(&p.a, a.dys, a.N, PLANES * R, np, p.a_blocks) && map_rows_mn(&p.b, a.xs, a.K, PLANES * R, kp, p.b_blocks);
  } else if (fwd) {
    ok = map_kmajor(&p.a, a.xs, a.K, PLANES * R, kp) && map_weights(&p.b, a.w, a.K, kp, a.N, PLANES * E, p.nt / 2);
  } else {
    p.b_blocks = a.K % 64 == 0 ? p.nt / 128 : 0;
    ok = map_kmajor(&p.a, a.dys, a.N, PLANES * R, np) && map_weights_mn(&p.b, a.w, a.K, kp, a.N, PLANES * E, p.b_blocks);
  }
  if (ok && p.out_aligned)
    ok = !f32 ? map_out_rows(&p.out, p.outp, p.N, R, 64)
         : wgrad ? map_out_f32(&p.out, p.outp, p.N, p.ldo, a.N, static_cast<int64_t>(p.splits) * E)
                 : map_out_f32(&p.out, p.outp, p.N, p.ldo, p.splits * R, 0);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = gm_tiles(op, a.g, a.K, a.N, p.nt) * p.splits;
  if (wgrad) return gm_launch<kGroupedWgrad, PLANES, true>(p, tiles, hdr, st);
  if constexpr (PLANES == 1)
    if (!parts)
      return fwd ? gm_launch<kGroupedForward, 1, false>(p, tiles, hdr, st) : gm_launch<kGroupedDgrad, 1, false>(p, tiles, hdr, st);
  return fwd ? gm_launch<kGroupedForward, PLANES, true>(p, tiles, hdr, st) : gm_launch<kGroupedDgrad, PLANES, true>(p, tiles, hdr, st);
}

cudaError_t launch_grouped_tc(int op, const GroupedArgs& a, const GroupedTcExtras& x, WsHeader* hdr, cudaStream_t st) {
  return x.planes == 3 ? gm_run<3>(op, a, x, hdr, st) : gm_run<1>(op, a, x, hdr, st);
}

cudaError_t launch_grouped_split(const SplitTensors& t, const GroupTables& g, int* flag, cudaStream_t st) {
  int64_t rows = 0;
  for (int i = 0; i < t.n; ++i) rows += t.t[i].rows;
  const int64_t blocks = (rows + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(split_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, t, g, flag);
}

cudaError_t launch_grouped_join(int op, int dtype, const GroupedArgs& a, const GroupedTcExtras& x, cudaStream_t st) {
  const bool wgrad = op == kGroupedWgrad;
  const int64_t rows = wgrad ? static_cast<int64_t>(a.g.E) * a.N : a.g.rows;
  const int cols = op == kGroupedForward ? a.N : a.K;
  const GroupTables g = wgrad ? GroupTables{nullptr, nullptr, rows, 1} : a.g;
  const int64_t blocks = (rows + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const float* parts = static_cast<const float*>(x.parts);
  const float scale = x.planes == 3 ? kSplitUnscale : 1.f;
  if (wgrad || dtype == kDtypeF32)
    return launch_dependent_kernel(join_kernel<float>, grid, dim3(256), 0, st, parts, static_cast<float*>(a.out), g, rows,
                                   cols, pitch4(cols), x.splits, scale, x.skip, x.over);
  return launch_dependent_kernel(join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, parts, static_cast<__nv_bfloat16*>(a.out),
                                 g, rows, cols, pitch4(cols), x.splits, scale, x.skip, x.over);
}

}  // namespace mm
