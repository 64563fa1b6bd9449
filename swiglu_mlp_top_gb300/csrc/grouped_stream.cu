// Experts' products for few rows: ys[r, n] = sum_k x[r, k] w[e, n, k] with bf16
// rows and weights in bf16 or in 4 bits, or both in fp32.  Bound by reading each needed weight
// row once, and below some ten MB by the latency of doing so.
//
// A block takes 16 rows of w (output columns) of one expert and up to 32 of
// its rows of x; an expert with more rows has them shared out over blocks (64
// tokens of a skewed routing, E = 8, k = 2, K = 2432, N = 768, 4 bits: 16 us
// one after the other, 12).  The block's four or eight warps share out the
// summed index in steps of 32 (4 bits: 128) columns.  A warp multiplies with
// mma.sync m16n8k16, the weights as the M operand straight from global memory:
// the order of the summed index is free as long as both operands use the same,
// so a lane takes 16 contiguous bytes of a weight row, which are 8 values (4
// bits: a whole group of 32 and its scale), and the same columns of x.  All
// loads of a few steps are in flight before the first product.  (The tensor
// cores of tcgen05 want their operands in shared memory and tiles of 128 rows:
// for these shapes a longer way to the same bytes.)
//
// fp32 values are split into three bf16 parts in registers, of whose nine
// products six are made (grouped_tc.cu); every 32 columns' sum is added in
// fp32.  A block whose sums are not finite (a value without such parts, or a sum
// of 2^80 and more) makes its results with multiply-adds.  (Four rows of one
// matrix, K = N = 2048: 8.6 us, 31 with multiply-adds alone.  From some 16 rows of
// an expert on, splitting bounds it: with a test of each value in it, a quarter
// of its instructions, 60 rows at E = 8 took 59 us for 45.)
#include "grouped.cuh"
#include "mx4.cuh"

namespace mm {

constexpr int kGsRows = 16;                  // rows of w per block
constexpr int kGsMost = 32;                  // rows of x

enum GsKind { kGsBf16, kGsMx4, kGsF32 };

struct GsParams {
  const void* x;            // [rows, K], K a multiple of 8
  const uint8_t* w;         // [E, N, K], or codes [E * N, 16 G]
  const uint32_t* sc;       // scale words [words, E * N]
  void* out;                // [rows, N], as x
  GroupTables g;
  int K, N;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <GsKind KIND> struct GsKindTraits { typedef __nv_bfloat16 Row; };
template <> struct GsKindTraits<kGsF32> { typedef float Row; };

template <bool MX4, int NT>
struct GsTraits {
  static constexpr int kParts = MX4 ? 4 : 1;                 // 8-column pieces of a lane's step
  static constexpr int kCols = 32 * kParts;                  // columns of a step
  // steps in flight: as many as registers hold beside the pieces of x
  static constexpr int kUnroll = MX4 ? (NT == 1 ? 2 : 1) : (NT == 1 ? 6 : NT == 2 ? 4 : 2);
};

// A warp's share of 16 rows of w times NT * 8 rows of x.
template <bool MX4, int WARPS, int NT>
__device__ __forceinline__ void gs_sum(const GsParams& P, int64_t wrow, int wlast, const __nv_bfloat16* x, int rows,
                                       float (&acc)[NT][4]) {
  typedef GsTraits<MX4, NT> Tr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int steps = (P.K + Tr::kCols - 1) / Tr::kCols;
  const int groups = (P.K + 31) / 32;
  const int64_t pitch = MX4 ? 16 * static_cast<int64_t>(groups) : 2 * static_cast<int64_t>(P.K);     // bytes of a weight row
  // rows of w behind the last one are read as the last one, and not stored
  const int64_t r0 = wrow + min(g, wlast), r1 = wrow + min(g + 8, wlast);
  const uint8_t *w0 = P.w + r0 * pitch + 16 * t, *w1 = P.w + r1 * pitch + 16 * t;
  const int64_t srows = static_cast<int64_t>(P.g.E) * P.N;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s0 = warp; s0 < steps; s0 += WARPS * Tr::kUnroll) {
    uint4 a[Tr::kUnroll][2], b[Tr::kUnroll][Tr::kParts][NT];
    uint32_t sw[Tr::kUnroll][2];
#pragma unroll
    for (int u = 0; u < Tr::kUnroll; ++u) {
      const int s = s0 + u * WARPS;
      const int k = s * Tr::kCols + 8 * Tr::kParts * t;      // this lane's first column
      const bool in = s < steps && k < P.K;
      a[u][0] = in ? __ldg(reinterpret_cast<const uint4*>(w0 + 64 * static_cast<int64_t>(s))) : zero;
      a[u][1] = in ? __ldg(reinterpret_cast<const uint4*>(w1 + 64 * static_cast<int64_t>(s))) : zero;
      if constexpr (MX4) {
        sw[u][0] = in ? __ldg(P.sc + s * srows + r0) : 0u;
        sw[u][1] = in ? __ldg(P.sc + s * srows + r1) : 0u;
      }
#pragma unroll
      for (int q = 0; q < Tr::kParts; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[u][q][j] = s < steps && k + 8 * q < P.K && 8 * j + g < rows
                           ? __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(8 * j + g) * P.K + k + 8 * q))
                           : zero;
    }
#pragma unroll
    for (int u = 0; u < Tr::kUnroll; ++u) {
      if (s0 + u * WARPS >= steps) break;                 // warp-uniform
      uint32_t f[2][2];
      bool two = false;
      if constexpr (MX4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t byte = (sw[u][i] >> (8 * t)) & 255u;
          mx4_factors(byte, f[i][0], f[i][1]);
          two |= byte > 128u;
        }
        two = __any_sync(0xffffffffu, two);
      }
#pragma unroll
      for (int q = 0; q < Tr::kParts; ++q) {
        uint4 v0 = a[u][0], v1 = a[u][1];
        if constexpr (MX4) {
          const uint32_t c0 = q == 0 ? a[u][0].x : q == 1 ? a[u][0].y : q == 2 ? a[u][0].z : a[u][0].w;
          const uint32_t c1 = q == 0 ? a[u][1].x : q == 1 ? a[u][1].y : q == 2 ? a[u][1].z : a[u][1].w;
          v0 = two ? e2m1_bf16<true>(c0, f[0][0], f[0][1]) : e2m1_bf16<false>(c0, f[0][0], 0u);
          v1 = two ? e2m1_bf16<true>(c1, f[1][0], f[1][1]) : e2m1_bf16<false>(c1, f[1][0], 0u);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_bf16(acc[j], v0.x, v1.x, v0.y, v1.y, b[u][q][j].x, b[u][q][j].y);
          mma_bf16(acc[j], v0.z, v1.z, v0.w, v1.w, b[u][q][j].z, b[u][q][j].w);
        }
      }
    }
  }
}

// The same in fp32.  Returns whether a sum is not finite: a value has no parts, or the sum is too large.
template <int WARPS, int NT>
__device__ __forceinline__ bool gs_sum_f32(const GsParams& P, int64_t wrow, int wlast, const float* x, int rows, float (&acc)[NT][4]) {
  constexpr int kUnroll = NT == 1 ? 3 : NT == 2 ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int steps = (P.K + 31) / 32;
  const float* w = reinterpret_cast<const float*>(P.w);
  const float *w0 = w + (wrow + min(g, wlast)) * P.K, *w1 = w + (wrow + min(g + 8, wlast)) * P.K;
  auto load = [](float (&v)[8], const float* p, bool in) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = in ? __ldg(reinterpret_cast<const float4*>(p)) : zero, b = in ? __ldg(reinterpret_cast<const float4*>(p) + 1) : zero;
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  };
  for (int s0 = warp; s0 < steps; s0 += WARPS * kUnroll) {
    float a[kUnroll][2][8], b[kUnroll][NT][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = s0 + u * WARPS, k = 32 * s + 8 * t;      // this lane's first column
      const bool in = s < steps && k < P.K;
      load(a[u][0], w0 + k, in);
      load(a[u][1], w1 + k, in);
#pragma unroll
      for (int j = 0; j < NT; ++j) load(b[u][j], x + static_cast<int64_t>(8 * j + g) * P.K + k, in && 8 * j + g < rows);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (s0 + u * WARPS >= steps) break;                    // warp-uniform
      uint4 v0[3], v1[3];
      split_vector(a[u][0], v0);
      split_vector(a[u][1], v1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 y[3];
        split_vector(b[u][j], y);
        // the small products first
        constexpr int kPa[6] = {2, 0, 1, 1, 0, 0}, kPb[6] = {0, 2, 1, 0, 1, 0};
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const uint4 &p = v0[kPa[i]], &q = v1[kPa[i]], &z = y[kPb[i]];
          mma_bf16(c[0], p.x, q.x, p.y, q.y, z.x, z.y);
          mma_bf16(c[1], p.z, q.z, p.w, q.w, z.z, z.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += c[0][i] + c[1][i];
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad |= !(fabsf(acc[j][i]) < INFINITY);
      acc[j][i] *= kSplitUnscale;
    }
  return bad;
}

// Two neighbouring results (the second one may lie behind the last column).
__device__ __forceinline__ void gs_store(__nv_bfloat16* o, float a, float b, int left, bool even) {
  if (even) {
    if (left > 0) *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(a, b);
  } else {
    if (left > 0) o[0] = __float2bfloat16_rn(a);
    if (left > 1) o[1] = __float2bfloat16_rn(b);
  }
}
__device__ __forceinline__ void gs_store(float* o, float a, float b, int left, bool even) {
  if (even) {
    if (left > 0) *reinterpret_cast<float2*>(o) = make_float2(a, b);
  } else {
    if (left > 0) o[0] = a;
    if (left > 1) o[1] = b;
  }
}

// 16 columns of `rows` rows (at most 8 NT): the warps' sums joined in warp order.
template <GsKind KIND, int WARPS, int NT>
__device__ __forceinline__ void gs_rows(const GsParams& P, int e, int n0, int64_t row0, int rows, float* s_part) {
  typedef typename GsKindTraits<KIND>::Row Row;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  const Row* x = static_cast<const Row*>(P.x) + row0 * P.K;
  Row* out = static_cast<Row*>(P.out) + row0 * P.N + n0;
  const int64_t wrow = static_cast<int64_t>(e) * P.N + n0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  if constexpr (KIND == kGsF32) {
    const bool bad = gs_sum_f32<WARPS, NT>(P, wrow, P.N - 1 - n0, x, rows, acc);
    if (__syncthreads_or(bad)) {               // and the last use of s_part is over
      const float* w = reinterpret_cast<const float*>(P.w) + wrow * P.K;
      for (int v = warp; v < rows * kGsRows; v += WARPS) {
        const int r = v / kGsRows, c = v % kGsRows;
        if (n0 + c >= P.N) continue;
        float sum = 0.f;
        for (int k = lane; k < P.K; k += 32)
          sum = fmaf(__ldg(w + static_cast<int64_t>(c) * P.K + k), __ldg(x + static_cast<int64_t>(r) * P.K + k), sum);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) out[static_cast<int64_t>(r) * P.N + c] = sum;
      }
      return;
    }
  } else {
    gs_sum<KIND == kGsMx4, WARPS, NT>(P, wrow, P.N - 1 - n0, x, rows, acc);
    __syncthreads();                           // the last use of s_part is over
  }
  // [warp][row of x][row of w]
  float* mine = s_part + warp * (kGsMost * kGsRows);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(8 * j + 2 * t + (i & 1)) * kGsRows + g + 8 * (i >> 1)] = acc[j][i];
  __syncthreads();
  for (int v = threadIdx.x; v < rows * (kGsRows / 2); v += 32 * WARPS) {
    const int r = v / (kGsRows / 2), c = 2 * (v % (kGsRows / 2));
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 p = *reinterpret_cast<const float2*>(s_part + w * (kGsMost * kGsRows) + r * kGsRows + c);
      sum.x += p.x;
      sum.y += p.y;
    }
    gs_store(out + static_cast<int64_t>(r) * P.N + c, sum.x, sum.y, P.N - n0 - c, P.N % 2 == 0);
  }
}

template <GsKind KIND, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
grouped_stream_kernel(const GsParams P) {
  __shared__ __align__(16) float s_part[WARPS * kGsMost * kGsRows];
  __shared__ GroupChunks s_chunks;
  typedef typename GsKindTraits<KIND>::Row Row;
  pdl_enter();
  group_chunks<kGsMost, false>(P.g, &s_chunks);
  __syncthreads();
  const int tiles = (P.N + kGsRows - 1) / kGsRows;
  const int64_t units = static_cast<int64_t>(s_chunks.count) * tiles;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int chunk = static_cast<int>(u / tiles), n0 = static_cast<int>(u % tiles) * kGsRows;
    const int e = chunk_group(s_chunks, chunk);
    const GroupSpan s = s_chunks.span[e];
    const int c = chunk - s_chunks.first[e], of = (s.n + kGsMost - 1) / kGsMost;
    const int each = of > 1 ? ((s.n + of - 1) / of + 7) / 8 * 8 : kGsMost;
    const int rows = min(each, s.n - c * each);
    const int64_t row0 = static_cast<int64_t>(s.r0) + c * each;
    if (rows <= 0) {
    } else if (rows <= 8) gs_rows<KIND, WARPS, 1>(P, e, n0, row0, rows, s_part);
    else if (rows <= 16) gs_rows<KIND, WARPS, 2>(P, e, n0, row0, rows, s_part);
    else if (rows <= 24) gs_rows<KIND, WARPS, 3>(P, e, n0, row0, rows, s_part);
    else gs_rows<KIND, WARPS, 4>(P, e, n0, row0, rows, s_part);
    if (c > 0) continue;
    // padding rows of the group
    const int cols = min(kGsRows, P.N - n0);
    for (int v = threadIdx.x; v < (s.r1 - s.r0 - s.n) * kGsRows; v += 32 * WARPS)
      if (v % kGsRows < cols)
        static_cast<Row*>(P.out)[(static_cast<int64_t>(s.r0) + s.n + v / kGsRows) * P.N + n0 + v % kGsRows] = Row(0.f);
  }
}

template <GsKind KIND, int WARPS>
static cudaError_t gs_launch(const GsParams& p, int64_t units, cudaStream_t st) {
  auto fn = grouped_stream_kernel<KIND, WARPS>;
  const int64_t most = static_cast<int64_t>(num_sms()) * resident_blocks(reinterpret_cast<const void*>(fn), 32 * WARPS);
  return launch_dependent_kernel(fn, dim3(static_cast<unsigned>(std::min(units, most))), dim3(32 * WARPS), 0, st, p);
}
// Eight warps share out the summed index of a tile where four would leave most
// of an SM's warps without one: K = 4096 and N = 4096 for one expert 10.6 ->
// 8.5 us (4 bits 9.0 -> 6.4), two experts with K = 2432, N = 768 6.6 -> 5.1;
// with a tile for every four warps they are slower by 10 to 30%.
template <GsKind KIND>
static cudaError_t gs_choose(const GsParams& p, cudaStream_t st) {
  const int64_t units = most_chunks(p.g, kGsMost) * ((p.N + kGsRows - 1) / kGsRows);
  const bool wide = units <= 2 * num_sms();
  return wide ? gs_launch<KIND, 8>(p, units, st) : gs_launch<KIND, 4>(p, units, st);
}

cudaError_t launch_grouped_stream(int dtype, const GroupedArgs& a, cudaStream_t st) {
  const GsParams p{a.xs, static_cast<const uint8_t*>(a.w), nullptr, a.out, a.g, a.K, a.N};
  return dtype == kDtypeBF16 ? gs_choose<kGsBf16>(p, st) : gs_choose<kGsF32>(p, st);
}
cudaError_t launch_mx4_stream(const Mx4MatmulArgs& a, cudaStream_t st) {
  return gs_choose<kGsMx4>(GsParams{a.x, static_cast<const uint8_t*>(a.w), reinterpret_cast<const uint32_t*>(a.w_exps), a.out, a.g,
                                    a.K, a.N}, st);
}

}  // namespace mm
