// Experts' products on the CUDA cores with fp32 multiply-adds (fp32 rows;
// the tensor cores' TF32 keeps 11 bits of each operand, which misses fp32's
// accuracy by three digits).
//
//   forward   ys[r, n]  = sum_k xs[r, k] w[e, n, k]       A = xs, B = w[e], both with k contiguous
//   dgrad     dxs[r, k] = sum_n dys[r, n] w[e, n, k]      A = dys, B = w[e] with its output index contiguous
//   wgrad     dw[e, n, k] = sum_r dys[r, n] xs[r, k]      A = dys, B = xs, the summed index is the row
//
// One block makes a tile of 128 x 128 with 256 threads, 8 x 8 outputs each
// as packed pairs of fp32 (fma.rn.f32x2: two multiply-adds an issue slot).
// Operands come in slices of 16 of the summed index, transposed into shared
// memory where the index is contiguous; the next slice is in registers while
// this one is multiplied.
#include "grouped.cuh"
#include "pack.cuh"

namespace mm {

constexpr int kSimtTile = 128, kSimtK = 16, kSimtThreads = 256;
constexpr int kSimtPitch = kSimtTile + 4;      // a transposing store of 4 rows hits 4 x 4 banks apart

// One slice (kSimtTile x kSimtK) of an operand, 8 values a thread.
// KC: the summed index is contiguous; element (i, k) at i * ld + k, else k * ld + i.
// V = 4: rows are 16-byte aligned.
template <typename T, bool KC, int V>
struct SimtSlice {
  float v[8];
  __device__ __forceinline__ void load(const T* p, int64_t ld, int i0, int iend, int k0, int kend) {
#pragma unroll
    for (int q = 0; q < 8 / V; ++q) {
      const int u = threadIdx.x + q * kSimtThreads;          // vector u of the slice
      constexpr int kAcross = (KC ? kSimtK : kSimtTile) / V; // vectors along the contiguous index
      const int c = (u % kAcross) * V, r = u / kAcross;
      const int i = i0 + (KC ? r : c), k = k0 + (KC ? c : r);
      const T* src = p + (KC ? static_cast<int64_t>(i) * ld + k : static_cast<int64_t>(k) * ld + i);
      if constexpr (V == 4) {
        // a row is a multiple of 4 long, so a vector is inside or outside as a whole
        const bool in = i < iend && k < kend;
        typename Pack<T, V>::Raw raw;
        if (in) raw = *reinterpret_cast<const typename Pack<T, V>::Raw*>(src);
#pragma unroll
        for (int j = 0; j < V; ++j) v[V * q + j] = in ? Pack<T, V>::get(raw, j) : 0.f;
      } else {
        v[q] = i < iend && k < kend ? static_cast<float>(*src) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void store(float* s) const {      // s[k][i]
#pragma unroll
    for (int q = 0; q < 8 / V; ++q) {
      const int u = threadIdx.x + q * kSimtThreads;
      constexpr int kAcross = (KC ? kSimtK : kSimtTile) / V;
      const int c = (u % kAcross) * V, r = u / kAcross;
      if constexpr (KC) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[(c + j) * kSimtPitch + r] = v[V * q + j];
      } else if constexpr (V == 4) {
        *reinterpret_cast<float4*>(s + r * kSimtPitch + c) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      } else {
        s[r * kSimtPitch + c] = v[q];
      }
    }
  }
};

// OP: 0 forward, 1 dgrad, 2 wgrad.  M: rows of w for wgrad; N: columns of the result.
template <typename T, int OP, int V>
__global__ void __launch_bounds__(kSimtThreads, 2)
grouped_simt_kernel(const T* __restrict__ a, const T* __restrict__ b, void* __restrict__ out,
                    const GroupTables g, const int M, const int N, const int K) {
  constexpr bool kAKc = OP != 2, kBKc = OP == 0;
  __shared__ __align__(16) float sA[2][kSimtK * kSimtPitch], sB[2][kSimtK * kSimtPitch];
  pdl_enter();
  const int cols = (N + kSimtTile - 1) / kSimtTile;
  // this block's tile: rows [m0, mend) of A of which those below mval count, columns from n0
  int m0, mend, mval, n0, k0 = 0, kend = K;
  int64_t out0 = 0;
  if constexpr (OP == 2) {
    const int mt = (M + kSimtTile - 1) / kSimtTile;
    const int64_t t = blockIdx.x;
    const int e = static_cast<int>(t / (static_cast<int64_t>(mt) * cols));
    const int local = static_cast<int>(t - static_cast<int64_t>(e) * mt * cols);
    m0 = (local / cols) * kSimtTile;
    n0 = (local % cols) * kSimtTile;
    mend = mval = M;
    const GroupSpan s = group_span(g, e);
    k0 = s.r0;
    kend = s.r0 + s.n;
    out0 = static_cast<int64_t>(e) * M * N;
  } else {
    const GroupTile t = find_group_tile(g, blockIdx.x, kSimtTile, cols);
    if (t.e < 0) return;
    m0 = t.s.r0 + t.mb * kSimtTile;
    mend = t.s.r1;
    mval = t.s.r0 + t.s.n;
    n0 = t.nb * kSimtTile;
    b += static_cast<int64_t>(t.e) * N * K;
  }
  const int64_t lda = OP == 2 ? M : K, ldb = OP == 0 ? K : N;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;      // outputs: rows 4 ty + 64 h, columns 4 tx + 64 h
  u64 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;

  SimtSlice<T, kAKc, V> la;
  SimtSlice<T, kBKc, V> lb;
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
      const float4 a0 = *reinterpret_cast<const float4*>(pa + k * kSimtPitch + 4 * ty);
      const float4 a1 = *reinterpret_cast<const float4*>(pa + k * kSimtPitch + 64 + 4 * ty);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(pb + k * kSimtPitch + 4 * tx);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(pb + k * kSimtPitch + 64 + 4 * tx);
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
    const int m = m0 + (i < 4 ? 4 * ty + i : 64 + 4 * ty + i - 4);
    if (m >= mend) continue;                       // padding rows hold zeros: their A was left out
    typedef typename std::conditional<OP == 2, float, T>::type TO;     // weight gradients are fp32
    TO* row = static_cast<TO*>(out) + out0 + static_cast<int64_t>(m) * N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 64 * h + 4 * tx;
      const float v[4] = {lo2(acc[i][2 * h]), hi2(acc[i][2 * h]), lo2(acc[i][2 * h + 1]), hi2(acc[i][2 * h + 1])};
      if (V == 4 && OP != 0) {                     // N is a multiple of 4
        if (n < N) row_store<TO, 4>(row, 0, n / 4, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) row[n + j] = static_cast<TO>(v[j]);
      }
    }
  }
}

template <typename T, int OP>
static cudaError_t simt_launch(const void* a, const void* b, void* out, const GroupTables& g, int M, int N,
                               int K, int64_t tiles, bool vec, cudaStream_t st) {
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const T *fa = static_cast<const T*>(a), *fb = static_cast<const T*>(b);
  const dim3 grid(static_cast<unsigned>(tiles)), block(kSimtThreads);
  return vec ? launch_dependent_kernel(grouped_simt_kernel<T, OP, 4>, grid, block, 0, st, fa, fb, out, g, M, N, K)
             : launch_dependent_kernel(grouped_simt_kernel<T, OP, 1>, grid, block, 0, st, fa, fb, out, g, M, N, K);
}

static int64_t tiles_of(int64_t n) { return (n + kSimtTile - 1) / kSimtTile; }
// Tiles of rows that any grouping of the rows can need.
static int64_t row_tiles(const GroupTables& g) {
  return g.offsets ? std::min<int64_t>(g.rows, g.rows / kSimtTile + g.E) : tiles_of(g.rows);
}

template <typename T>
static cudaError_t simt(int op, const GroupedArgs& p, cudaStream_t st) {
  if (op == kGroupedForward)
    return simt_launch<T, 0>(p.xs, p.w, p.out, p.g, 0, p.N, p.K, row_tiles(p.g) * tiles_of(p.N), p.K % 4 == 0, st);
  if (op == kGroupedDgrad)
    return simt_launch<T, 1>(p.dys, p.w, p.out, p.g, 0, p.K, p.N, row_tiles(p.g) * tiles_of(p.K),
                             p.K % 4 == 0 && p.N % 4 == 0, st);
  return simt_launch<T, 2>(p.dys, p.xs, p.out, p.g, p.N, p.K, 0, p.g.E * tiles_of(p.N) * tiles_of(p.K),
                           p.K % 4 == 0 && p.N % 4 == 0, st);
}

cudaError_t launch_grouped_simt(int dtype, int op, const GroupedArgs& p, cudaStream_t st) {
  return dtype == kDtypeBF16 ? cudaErrorInvalidValue : simt<float>(op, p, st);
}

}  // namespace mm
