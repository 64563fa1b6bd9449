// Experts' products of fp32 rows on the CUDA cores with fp32 multiply-adds: few
// rows of a forward pass with a width that is no multiple of 8 (others:
// grouped_stream.cu), and the calls whose values cannot be split into
// three bf16 parts for the tensor cores (grouped_tc.cu), or whose results are
// too large for that, told by flags on the device without which the tile kernel
// returns.  The tiles are bound by the
// multiply-adds (T = 1000, E = 4, K = 768, N = 2432: 148 us, of which 52 at 72
// Tflop/s; the tensor cores take 51).
//
//   forward   ys[r, n]  = sum_k xs[r, k] w[e, n, k]       A = xs, B = w[e], both with k contiguous
//   dgrad     dxs[r, k] = sum_n dys[r, n] w[e, n, k]      A = dys, B = w[e] with its output index contiguous
//   wgrad     dw[e, n, k] = sum_r dys[r, n] xs[r, k]      A = dys, B = xs, the summed index is the row
//
// One block makes a tile of 128 (or 64) x 128, a thread 8 x 8 outputs of it as
// packed pairs of fp32 (fma.rn.f32x2: two multiply-adds an issue slot).
// Operands come in slices of 16 of the summed index, transposed into shared
// memory where the index is contiguous; the next slice is in registers while
// this one is multiplied.
//
// Few rows (forward): a warp takes four rows of w times up to eight rows of x,
// with the summed index over its lanes; an expert's next eight rows go to
// another warp (20 rows, K = N = 2048: 126 us one after the other, 53).
#include "grouped.cuh"
#include "pack.cuh"

namespace mm {

constexpr int kSimtN = 128, kSimtK = 16;

// One slice (ROWS x kSimtK) of an operand, spread over THREADS threads.
// KC: the summed index is contiguous; element (i, k) at i * ld + k, else k * ld + i.
// V = 4: rows are 16-byte aligned.
template <bool KC, int V, int ROWS, int THREADS>
struct SimtSlice {
  static constexpr int kMine = ROWS * kSimtK / THREADS;
  static constexpr int kPitch = ROWS + 4;      // a transposing store of 4 rows hits 4 x 4 banks apart
  static constexpr int kAcross = (KC ? kSimtK : ROWS) / V;   // vectors along the contiguous index
  float v[kMine];
  __device__ __forceinline__ void load(const float* p, int64_t ld, int i0, int iend, int k0, int kend) {
#pragma unroll
    for (int q = 0; q < kMine / V; ++q) {
      const int u = threadIdx.x + q * THREADS;               // vector u of the slice
      const int c = (u % kAcross) * V, r = u / kAcross;
      const int i = i0 + (KC ? r : c), k = k0 + (KC ? c : r);
      const float* src = p + (KC ? static_cast<int64_t>(i) * ld + k : static_cast<int64_t>(k) * ld + i);
      if constexpr (V == 4) {
        // a row is a multiple of 4 long, so a vector is inside or outside as a whole
        const float4 f = i < iend && k < kend ? __ldg(reinterpret_cast<const float4*>(src))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
      } else {
        v[q] = i < iend && k < kend ? __ldg(src) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void store(float* s) const {      // s[k][i]
#pragma unroll
    for (int q = 0; q < kMine / V; ++q) {
      const int u = threadIdx.x + q * THREADS;
      const int c = (u % kAcross) * V, r = u / kAcross;
      if constexpr (KC) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[(c + j) * kPitch + r] = v[V * q + j];
      } else if constexpr (V == 4) {
        *reinterpret_cast<float4*>(s + r * kPitch + c) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      } else {
        s[r * kPitch + c] = v[q];
      }
    }
  }
};

// OP: 0 forward, 1 dgrad, 2 wgrad.  TM: rows of a tile.  M: rows of w for
// wgrad; N: columns of the result.
template <int OP, int V, int TM>
__global__ void __launch_bounds__(2 * TM, 512 / (2 * TM))
grouped_simt_kernel(const float* __restrict__ a, const float* __restrict__ b, float* __restrict__ out,
                    const GroupTables g, const int M, const int N, const int K, const int* only_if) {
  constexpr bool kAKc = OP != 2, kBKc = OP == 0;
  typedef SimtSlice<kAKc, V, TM, 2 * TM> SliceA;
  typedef SimtSlice<kBKc, V, kSimtN, 2 * TM> SliceB;
  constexpr int kPitchA = SliceA::kPitch, kPitchB = SliceB::kPitch;
  __shared__ __align__(16) float sA[2][kSimtK * kPitchA], sB[2][kSimtK * kPitchB];
  pdl_enter();
  if (only_if != nullptr && only_if[0] == 0 && only_if[1 + OP] == 0) return;
  const int cols = (N + kSimtN - 1) / kSimtN;
  // this block's tile: rows [m0, mend) of A of which those below mval count, columns from n0
  int m0, mend, mval, n0, k0 = 0, kend = K;
  int64_t out0 = 0;
  if constexpr (OP == 2) {
    const int mt = (M + TM - 1) / TM;
    const int64_t t = blockIdx.x;
    const int e = static_cast<int>(t / (static_cast<int64_t>(mt) * cols));
    const int local = static_cast<int>(t - static_cast<int64_t>(e) * mt * cols);
    m0 = (local / cols) * TM;
    n0 = (local % cols) * kSimtN;
    mend = mval = M;
    const GroupSpan s = group_span(g, e);
    k0 = s.r0;
    kend = s.r0 + s.n;
    out0 = static_cast<int64_t>(e) * M * N;
  } else {
    const GroupTile t = find_group_tile(g, blockIdx.x, TM, cols);
    if (t.e < 0) return;
    m0 = t.s.r0 + t.mb * TM;
    mend = t.s.r1;
    mval = t.s.r0 + t.s.n;
    n0 = t.nb * kSimtN;
    b += static_cast<int64_t>(t.e) * N * K;
  }
  const int64_t lda = OP == 2 ? M : K, ldb = OP == 0 ? K : N;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;      // outputs: rows 4 ty + TM/2 h, columns 4 tx + 64 h
  u64 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;

  SliceA la;
  SliceB lb;
  const int slices = (kend - k0 + kSimtK - 1) / kSimtK;
  // a forward or dgrad tile of padding alone has no slices to add up
  const int todo = OP != 2 && m0 >= mval ? 0 : slices;
  if (todo > 0) {
    la.load(a, lda, m0, mval, k0, kend);
    lb.load(b, ldb, n0, N, k0, kend);
    la.store(sA[0]);
    lb.store(sB[0]);
  }
  __syncthreads();
  for (int s = 0; s < todo; ++s) {
    const bool more = s + 1 < todo;
    if (more) {
      la.load(a, lda, m0, mval, k0 + (s + 1) * kSimtK, kend);
      lb.load(b, ldb, n0, N, k0 + (s + 1) * kSimtK, kend);
    }
    const float* pa = sA[s & 1];
    const float* pb = sB[s & 1];
#pragma unroll
    for (int k = 0; k < kSimtK; ++k) {
      const float4 a0 = *reinterpret_cast<const float4*>(pa + k * kPitchA + 4 * ty);
      const float4 a1 = *reinterpret_cast<const float4*>(pa + k * kPitchA + TM / 2 + 4 * ty);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(pb + k * kPitchB + 4 * tx);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(pb + k * kPitchB + 64 + 4 * tx);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const u64 bv[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u64 aa = pair2(av[i], av[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = ffma2(aa, bv[j], acc[i][j]);
      }
    }
    if (more) {
      la.store(sA[(s + 1) & 1]);
      lb.store(sB[(s + 1) & 1]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i < 4 ? 4 * ty + i : TM / 2 + 4 * ty + i - 4);
    if (m >= mend) continue;
    const bool counts = m < mval;                  // padding rows become zeros, whatever B holds
    float* row = out + out0 + static_cast<int64_t>(m) * N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 64 * h + 4 * tx;
      float v[4] = {lo2(acc[i][2 * h]), hi2(acc[i][2 * h]), lo2(acc[i][2 * h + 1]), hi2(acc[i][2 * h + 1])};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = counts ? v[j] : 0.f;
      if (V == 4 && OP != 0) {                     // N is a multiple of 4
        if (n < N) *reinterpret_cast<float4*>(row + n) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) row[n + j] = v[j];
      }
    }
  }
}

// Few rows: four rows of w (a warp's) times up to eight of the group's rows of
// x.  V = 4: rows start on 16 bytes.
constexpr int kSimtFewW = 4, kSimtFewX = 8;

template <int V>
__global__ void __launch_bounds__(128)
grouped_simt_few_kernel(const float* __restrict__ x, const float* __restrict__ w, float* __restrict__ out,
                        const GroupTables g, const int N, const int K) {
  __shared__ GroupChunks s_chunks;
  pdl_enter();
  group_chunks<kSimtFewX, true>(g, &s_chunks);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int tiles = (N + kSimtFewW - 1) / kSimtFewW;
  const int64_t units = static_cast<int64_t>(s_chunks.count) * tiles;
  for (int64_t u = blockIdx.x * 4ll + (threadIdx.x >> 5); u < units; u += gridDim.x * 4ll) {
    const int chunk = static_cast<int>(u / tiles), n0 = static_cast<int>(u % tiles) * kSimtFewW;
    const int e = chunk_group(s_chunks, chunk);
    const GroupSpan s = s_chunks.span[e];
    const int r = (chunk - s_chunks.first[e]) * kSimtFewX;
    const float* wr[kSimtFewW];
#pragma unroll
    for (int q = 0; q < kSimtFewW; ++q)        // rows of w behind the last one are read as the last one, and not stored
      wr[q] = w + (static_cast<int64_t>(e) * N + min(n0 + q, N - 1)) * K;
    const int rows = min(kSimtFewX, s.n - r);        // <= 0: padding alone
    const float* xr = x + static_cast<int64_t>(s.r0 + r) * K;
    float acc[kSimtFewX * kSimtFewW];              // [row of x][row of w]
#pragma unroll
    for (int q = 0; q < kSimtFewX * kSimtFewW; ++q) acc[q] = 0.f;
    if (rows > 0)
#pragma unroll 2
      for (int k = V * lane; k < K; k += 32 * V) {
        float wv[kSimtFewW][V], xv[V];
#pragma unroll
        for (int q = 0; q < kSimtFewW; ++q) {
          const auto raw = *reinterpret_cast<const typename Pack<float, V>::Raw*>(wr[q] + k);
#pragma unroll
          for (int e = 0; e < V; ++e) wv[q][e] = Pack<float, V>::get(raw, e);
        }
#pragma unroll
        for (int j = 0; j < kSimtFewX; ++j) {
          if (j >= rows) break;
          const auto raw = *reinterpret_cast<const typename Pack<float, V>::Raw*>(xr + static_cast<int64_t>(j) * K + k);
#pragma unroll
          for (int e = 0; e < V; ++e) xv[e] = Pack<float, V>::get(raw, e);
#pragma unroll
          for (int q = 0; q < kSimtFewW; ++q)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[j * kSimtFewW + q] = fmaf(wv[q][e], xv[e], acc[j * kSimtFewW + q]);
        }
      }
    const float sum = reduce_scatter(acc, lane);   // lane: row of x lane / 4, row of w lane % 4
    const int row = r + lane / kSimtFewW, n = n0 + lane % kSimtFewW;
    if (row < s.r1 - s.r0 && n < N) out[static_cast<int64_t>(s.r0 + row) * N + n] = row < s.n ? sum : 0.f;
  }
}

template <int OP, int V, int TM>
static cudaError_t simt_tiles(const void* a, const void* b, void* out, const GroupTables& g, int M, int N, int K,
                              int64_t tiles, const int* only_if, cudaStream_t st) {
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(grouped_simt_kernel<OP, V, TM>, dim3(static_cast<unsigned>(tiles)), dim3(2 * TM), 0, st,
                                 static_cast<const float*>(a), static_cast<const float*>(b), static_cast<float*>(out), g,
                                 M, N, K, only_if);
}

// Tiles of `tm` rows that any grouping of the rows can need (wgrad: that there are).
static int64_t simt_row_tiles(int op, const GroupTables& g, int M, int tm) {
  if (op == kGroupedWgrad) return g.E * static_cast<int64_t>((M + tm - 1) / tm);
  return g.offsets ? std::min<int64_t>(g.rows, g.rows / tm + g.E) : (g.rows + tm - 1) / tm;
}

// Tiles of 64 rows where tiles of 128 would not go round the SMs four times:
// the last round is shorter (T = 1000, E = 4, K = 768, N = 2432: 148 us against
// 153).
template <int OP>
static cudaError_t simt(const void* a, const void* b, void* out, const GroupTables& g, int M, int N, int K, bool vec,
                        const int* only_if, cudaStream_t st) {
  const int64_t cols = (N + kSimtN - 1) / kSimtN;
  const int64_t big = simt_row_tiles(OP, g, M, 128) * cols, small = simt_row_tiles(OP, g, M, 64) * cols;
  if (big >= 4 * num_sms())
    return vec ? simt_tiles<OP, 4, 128>(a, b, out, g, M, N, K, big, only_if, st) : simt_tiles<OP, 1, 128>(a, b, out, g, M, N, K, big, only_if, st);
  return vec ? simt_tiles<OP, 4, 64>(a, b, out, g, M, N, K, small, only_if, st) : simt_tiles<OP, 1, 64>(a, b, out, g, M, N, K, small, only_if, st);
}

cudaError_t launch_grouped_simt(int op, const GroupedArgs& p, const int* only_if, cudaStream_t st) {
  const bool k4 = p.K % 4 == 0, kn4 = k4 && p.N % 4 == 0;
  if (op == kGroupedWgrad) return simt<kGroupedWgrad>(p.dys, p.xs, p.out, p.g, p.N, p.K, 0, kn4, only_if, st);
  if (op == kGroupedDgrad) return simt<kGroupedDgrad>(p.dys, p.w, p.out, p.g, 0, p.K, p.N, kn4, only_if, st);
  // the few rows' kernel knows no only_if
  if (only_if != nullptr || p.g.rows > f32_few_rows(p.g.E))
    return simt<kGroupedForward>(p.xs, p.w, p.out, p.g, 0, p.N, p.K, k4, only_if, st);
  const int64_t units = most_chunks(p.g, kSimtFewX) * ((p.N + kSimtFewW - 1) / kSimtFewW);
  auto fn = k4 ? grouped_simt_few_kernel<4> : grouped_simt_few_kernel<1>;
  const int64_t most = static_cast<int64_t>(num_sms()) * resident_blocks(reinterpret_cast<const void*>(fn), 128);
  return launch_dependent_kernel(fn, dim3(static_cast<unsigned>(std::min((units + 3) / 4, most))), dim3(128), 0, st,
                                 static_cast<const float*>(p.xs), static_cast<const float*>(p.w),
                                 static_cast<float*>(p.out), p.g, p.N, p.K);
}

}  // namespace mm
