// Norms before and after a block, fused with its gate and residual scale,
// and the gradient (include/mm.h, mm_block_norm):
//   p = f rho_f w_post,  rho_f = 1 / sqrt(mean_h f^2 + eps)     (w_post absent: p = f)
//   r = round(s x + g p)                                        (g absent: 1)
//   n = r rho_r w_pre,   rho_r of the rounded r
//
// Both directions read every input and write every output once, so DRAM
// bounds them.  A row is held in the registers of one group of `tpr` threads
// (a multiple of a warp; V elements per load, NV loads per array), a block
// holds several groups, and the loads of a row are all in flight together.
// Sums run in fp32 in a fixed order: lane, warp tree, the group's warps.
#include <cstring>

#include "mm_kernels.cuh"
#include "pack.cuh"

namespace mm {

// Sums of N values over a group of tpr threads, the same in all of them.
// `red` holds 2 x N floats per warp of the block; the caller flips `turn`
// between calls, so that a call's slots are not overwritten while a slower
// warp of the group still reads them (every warp passes this call's barrier
// before any writes the slots of the call after next).
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int turn, int group, int tpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (tpr == 32) return;
  const int warps = tpr >> 5, w0 = group * warps, total = blockDim.x >> 5;
  float* slot = red + turn * (N * total);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) slot[(threadIdx.x >> 5) * N + i] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += slot[(w0 + w) * N + i];
    v[i] = s;
  }
}

__device__ __forceinline__ float inv_rms_of(float ss, int H, float eps) {
  return 1.0f / sqrtf(ss / static_cast<float>(H) + eps);
}

// A thread's unit m of a row: V consecutive elements, or (V = 1) two single
// columns tpr apart.  Columns behind the row read as zeros.
template <typename T, int V>
struct Unit {
  static constexpr int kPairs = V / 2;
  static constexpr bool kAsync = true;        // 16-byte cp.async
  typedef typename Pack<T, V>::Raw Raw;
  static __device__ __forceinline__ void copy(uint32_t slot, const void* p, int64_t base, int m, int c0, int tpr,
                                              int nv) {
    if (c0 + m * tpr < nv)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot),
                   "l"(reinterpret_cast<const Raw*>(static_cast<const T*>(p) + base) + c0 + m * tpr)
                   : "memory");
  }
  static __device__ __forceinline__ Raw zero() { return Raw{}; }
  static __device__ __forceinline__ u64 get(const Raw& r, int k) {
    return pair2(Pack<T, V>::get(r, 2 * k), Pack<T, V>::get(r, 2 * k + 1));
  }
  static __device__ __forceinline__ Raw put(const u64 (&v)[kPairs]) {
    float o[V];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      o[2 * k] = lo2(v[k]);
      o[2 * k + 1] = hi2(v[k]);
    }
    return Pack<T, V>::put(o);
  }
  static __device__ __forceinline__ void store_raw(void* p, int64_t base, int m, int c0, int tpr, int nv,
                                                   const Raw& r) {
    if (c0 + m * tpr < nv) reinterpret_cast<Raw*>(static_cast<T*>(p) + base)[c0 + m * tpr] = r;
  }
  static __device__ __forceinline__ void store(void* p, int64_t base, int m, int c0, int tpr, int nv,
                                               const u64 (&v)[kPairs]) {
    store_raw(p, base, m, c0, tpr, nv, put(v));
  }
  // fp32 values by column in shared memory: four of a vector's V side by side
  // for all of the group's threads, then the next four, so that a warp's
  // 16-byte accesses meet every bank once.  place(): where column h is.
  static __device__ __forceinline__ int place(int h, int tpr) {
    const int c = h / V, j = h % V, m = c / tpr;
    return ((m * (V / 4) + j / 4) * tpr + (c - m * tpr)) * 4 + j % 4;
  }
  static __device__ __forceinline__ void cols(const float* s, int m, int c0, int tpr, u64 (&v)[kPairs]) {
    const ulonglong2* q = reinterpret_cast<const ulonglong2*>(s) + m * (V / 4) * tpr + c0;
#pragma unroll
    for (int k = 0; k < kPairs / 2; ++k) {
      const ulonglong2 w = q[k * tpr];
      v[2 * k] = w.x;
      v[2 * k + 1] = w.y;
    }
  }
  static __device__ __forceinline__ void keep(float* s, int m, int c0, int tpr, int nv, const u64 (&v)[kPairs]) {
    if (c0 + m * tpr >= nv) return;
    ulonglong2* q = reinterpret_cast<ulonglong2*>(s) + m * (V / 4) * tpr + c0;
#pragma unroll
    for (int k = 0; k < kPairs / 2; ++k) q[k * tpr] = make_ulonglong2(v[2 * k], v[2 * k + 1]);
  }
};
template <typename T>
struct Unit<T, 1> {
  static constexpr int kPairs = 1;
  static constexpr bool kAsync = false;       // cp.async of 4 bytes is slower than plain loads
  struct __align__(2 * sizeof(T)) Raw {
    T a, b;
  };
  static __device__ __forceinline__ Raw zero() { return Raw{T(0.f), T(0.f)}; }
  static __device__ __forceinline__ Raw load(const void* p, int64_t base, int m, int c0, int tpr, int nv) {
    const T* row = static_cast<const T*>(p) + base;
    const int c = c0 + 2 * m * tpr;
    return Raw{c < nv ? row[c] : T(0.f), c + tpr < nv ? row[c + tpr] : T(0.f)};
  }
  static __device__ __forceinline__ u64 get(const Raw& r, int) {
    return pair2(static_cast<float>(r.a), static_cast<float>(r.b));
  }
  static __device__ __forceinline__ Raw put(const u64 (&v)[1]) { return Raw{T(lo2(v[0])), T(hi2(v[0]))}; }
  static __device__ __forceinline__ void store_raw(void* p, int64_t base, int m, int c0, int tpr, int nv,
                                                   const Raw& r) {
    T* row = static_cast<T*>(p) + base;
    const int c = c0 + 2 * m * tpr;
    if (c < nv) row[c] = r.a;
    if (c + tpr < nv) row[c + tpr] = r.b;
  }
  static __device__ __forceinline__ void store(void* p, int64_t base, int m, int c0, int tpr, int nv,
                                               const u64 (&v)[1]) {
    store_raw(p, base, m, c0, tpr, nv, put(v));
  }
  static __device__ __forceinline__ int place(int h, int) { return h; }
  static __device__ __forceinline__ void cols(const float* s, int m, int c0, int tpr, u64 (&v)[1]) {
    const int c = c0 + 2 * m * tpr;
    v[0] = pair2(s[c], s[c + tpr]);
  }
  static __device__ __forceinline__ void keep(float* s, int m, int c0, int tpr, int nv, const u64 (&v)[1]) {
    const int c = c0 + 2 * m * tpr;
    if (c < nv) s[c] = lo2(v[0]);
    if (c + tpr < nv) s[c + tpr] = hi2(v[0]);
  }
};


template <typename T>
__device__ __forceinline__ float bn_param(const void* w, int h) {
  return w ? static_cast<float>(static_cast<const T*>(w)[h]) : 1.f;
}

// The V values of vector c to their columns in shared memory.
template <typename U, int V>
__device__ __forceinline__ void columns_put(float* s, int c, int tpr, const float (&v)[V]) {
  if constexpr (V == 1) {
    s[c] = v[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4*>(s + U::place(c * V + j, tpr)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}

// w_pre and w_post g in fp32 by column, zeros behind the row (an absent w_pre
// is zeros too: nothing is made of it; other absent factors are 1).  One
// vector of each parameter a thread, so that their loads are in flight
// together: a block waits for them once.
template <typename T, int V, bool kTokenGate>
__device__ __forceinline__ void stage_params(const void* pre, const void* post, const void* gate, int H, int tpr,
                                             int span, float* w_pre, float* w_mid) {
  using U = Unit<T, V>;
  using P = Pack<T, V>;
  for (int c = threadIdx.x; c < span / V; c += blockDim.x) {
    const bool in = c < H / V;
    typename P::Raw a, b, g;
    if (in && pre) a = row_load<T, V>(pre, 0, c);
    if (in && post) b = row_load<T, V>(post, 0, c);
    if (in && gate && !kTokenGate) g = row_load<T, V>(gate, 0, c);
    float p[V], m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = in && pre ? P::get(a, j) : 0.f;
      m[j] = in ? (post ? P::get(b, j) : 1.f) * (gate && !kTokenGate ? P::get(g, j) : 1.f) : 0.f;
    }
    columns_put<U, V>(w_pre, c, tpr, p);
    columns_put<U, V>(w_mid, c, tpr, m);
  }
}

// ------------------------------------------------------------------ forward
// The rows that the ring below does not take (bn_ring_pick): many that fill a
// block each, and wider ones than its shared memory holds twice.  A group of
// threads per row, everything in registers.
constexpr size_t kBnMostSmem = 224 * 1024;   // dynamic, of 227 KB a block may have
constexpr int kBnFwdThreads = 512;      // most threads of a block (one group of them: H = 16384)

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kBnFwdThreads) block_norm_kernel(const BlockNormFwd a, int tpr) {
  using P = Pack<T, V>;
  pdl_enter();
  __shared__ float red[2 * kBnFwdThreads / 32];
  const int group = threadIdx.x / tpr, c0 = threadIdx.x - group * tpr, nv = a.H / V;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + group;
  if (t >= a.T) return;                       // whole groups: their barriers are their own
  const int64_t base = t * a.H, gbase = a.gate_per_token ? base : 0;
  typename P::Raw x[NV], f[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * tpr;
    if (c < nv) x[i] = row_load<T, V>(a.x, base, c);
  }
  if (a.f) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * tpr;
      if (c < nv) f[i] = row_load<T, V>(a.f, base, c);
    }
    float rho[1] = {1.f};
    if (a.post_w) {
      rho[0] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * tpr < nv)
#pragma unroll
          for (int j = 0; j < V; ++j) rho[0] = fmaf(P::get(f[i], j), P::get(f[i], j), rho[0]);
      group_sum(rho, red, 0, group, tpr);
      rho[0] = inv_rms_of(rho[0], a.H, a.eps);
      if (c0 == 0 && a.rstd_post) a.rstd_post[t] = rho[0];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * tpr;
      if (c < nv) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = P::get(f[i], j);
        if (a.post_w) {
          const auto w = row_load<T, V>(a.post_w, 0, c);
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = v[j] * rho[0] * P::get(w, j);
        }
        if (a.gate) {
          const auto g = row_load<T, V>(a.gate, gbase, c);
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] *= P::get(g, j);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = fmaf(a.residual_scale, P::get(x[i], j), v[j]);
        x[i] = P::put(v);                     // r as stored
        row_store<T, V>(a.r, base, c, v);
      }
    }
  }
  if (a.pre_w == nullptr) return;
  float rho[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (c0 + i * tpr < nv)
#pragma unroll
      for (int j = 0; j < V; ++j) rho[0] = fmaf(P::get(x[i], j), P::get(x[i], j), rho[0]);
  group_sum(rho, red, 1, group, tpr);
  rho[0] = inv_rms_of(rho[0], a.H, a.eps);
  if (c0 == 0 && a.rstd_pre) a.rstd_pre[t] = rho[0];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * tpr;
    if (c < nv) {
      const auto w = row_load<T, V>(a.pre_w, 0, c);
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = P::get(x[i], j) * rho[0] * P::get(w, j);
      row_store<T, V>(a.n, base, c, v);
    }
  }
}

// The rule: a block of groups per SM walks down the rows, the next row's
// inputs on their way to shared memory (each thread copies and reads its own
// slots, so without a barrier), w_post g and w_pre there in fp32, sums and
// products on pairs.  Against one group per row and no loop (above) no last
// wave is left part empty, and the parameters are read once a block instead of
// once a row, by all its threads: bf16, H = 768, T = 16384 21 -> 18 us, T = 1
// 3.6 -> 2.2 us; fp32 with a token gate 48 -> 40 and 4.5 -> 2.4 us; fp32, H =
// 6144, T = 608 21.7 -> 14.3 us.  Unaligned rows have
// the next row in registers; the parameters re-read in single elements were
// what cost them most (T = 16384, H = 461 with a token gate: 57 -> 20 us).
template <typename T, int V, int NU, bool kTokenGate>
__global__ void __launch_bounds__(kBnFwdThreads, 1)
block_norm_ring_kernel(const BlockNormFwd a, int tpr, int span) {
  using U = Unit<T, V>;
  typedef typename U::Raw Raw;
  constexpr int NP = U::kPairs, kIn = kTokenGate ? 3 : 2;
  extern __shared__ __align__(16) float bn_smem[];
  __shared__ float red[2 * kBnFwdThreads / 32];
  float* w_mid = bn_smem;
  float* w_pre = bn_smem + span;
  const int group = threadIdx.x / tpr, c0 = threadIdx.x - group * tpr, nv = a.H / V, groups = blockDim.x / tpr;
  constexpr int kStageBytes = kIn * NU * 32 * static_cast<int>(sizeof(Raw));
  unsigned char* ring = reinterpret_cast<unsigned char*>(bn_smem + 2 * span) + (threadIdx.x >> 5) * (2 * kStageBytes) +
                        (threadIdx.x & 31) * sizeof(Raw);
  auto at = [](int i, int m) { return (i * NU + m) * 32 * static_cast<int>(sizeof(Raw)); };
  const void* src[3] = {a.x, a.f, kTokenGate ? a.gate : nullptr};
  Raw next[U::kAsync ? 1 : kIn][U::kAsync ? 1 : NU], now[U::kAsync ? 1 : kIn][U::kAsync ? 1 : NU];
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.T)
#pragma unroll
      for (int i = 0; i < kIn; ++i)
        if (src[i])
#pragma unroll
          for (int m = 0; m < NU; ++m) {
            if constexpr (U::kAsync)
              U::copy(smem_u32(ring + stage * kStageBytes) + at(i, m), src[i], t * a.H, m, c0, tpr, nv);
            else
              next[i][m] = U::load(src[i], t * a.H, m, c0, tpr, nv);
          }
    if constexpr (U::kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kIn; ++i)               // what no copy will fill stays zero
#pragma unroll
    for (int m = 0; m < NU; ++m) {
      if constexpr (U::kAsync) {
        if (src[i] == nullptr || c0 + m * tpr >= nv)
          for (int st = 0; st < 2; ++st) *reinterpret_cast<Raw*>(ring + st * kStageBytes + at(i, m)) = U::zero();
      } else {
        next[i][m] = U::zero();
      }
    }
  pdl_enter();
  // rows go to blocks first: few of them to an SM each
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(group) * gridDim.x + blockIdx.x;
  fetch(t, 0);
  stage_params<T, V, kTokenGate>(a.pre_w, a.post_w, a.gate, a.H, tpr, span, w_pre, w_mid);
  __syncthreads();
  const u64 scale2 = pair2(a.residual_scale, a.residual_scale);
  int turn = 0;               // flips with every sum: a row may have one or two
  for (int stage = 0; t < a.T; t += step, stage ^= 1) {
    const int64_t base = t * a.H;
    if constexpr (!U::kAsync) {
#pragma unroll
      for (int i = 0; i < kIn; ++i)
#pragma unroll
        for (int m = 0; m < NU; ++m) now[i][m] = next[i][m];
    }
    fetch(t + step, stage ^ 1);
    if constexpr (U::kAsync) asm volatile("cp.async.wait_group 1;" ::: "memory");
    const unsigned char* here = ring + stage * kStageBytes;
    auto value = [&](int i, int m) -> Raw {
      if constexpr (U::kAsync) return *reinterpret_cast<const Raw*>(here + at(i, m));
      else return now[i][m];
    };
    Raw r[NU];
#pragma unroll
    for (int m = 0; m < NU; ++m) r[m] = value(0, m);
    if (a.f) {
      Raw f[NU];
#pragma unroll
      for (int m = 0; m < NU; ++m) f[m] = value(1, m);
      float rho[1] = {1.f};
      if (a.post_w) {
        u64 ss = 0;
#pragma unroll
        for (int m = 0; m < NU; ++m)
#pragma unroll
          for (int k = 0; k < NP; ++k) ss = ffma2(U::get(f[m], k), U::get(f[m], k), ss);
        rho[0] = hsum2(ss);
        group_sum(rho, red, turn, group, tpr);
        turn ^= 1;
        rho[0] = inv_rms_of(rho[0], a.H, a.eps);
        if (c0 == 0 && a.rstd_post) a.rstd_post[t] = rho[0];
      }
      const u64 rho2 = pair2(rho[0], rho[0]);
#pragma unroll
      for (int m = 0; m < NU; ++m) {
        u64 w[NP], v[NP];
        U::cols(w_mid, m, c0, tpr, w);
        Raw g = U::zero();
        if constexpr (kTokenGate) g = value(2, m);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          v[k] = fmul2(fmul2(U::get(f[m], k), rho2), w[k]);
          if constexpr (kTokenGate) v[k] = fmul2(v[k], U::get(g, k));
          v[k] = ffma2(scale2, U::get(r[m], k), v[k]);
        }
        r[m] = U::put(v);                     // r as stored
        U::store_raw(a.r, base, m, c0, tpr, nv, r[m]);
      }
    }
    if (a.pre_w == nullptr) continue;
    u64 ss = 0;
#pragma unroll
    for (int m = 0; m < NU; ++m)
#pragma unroll
      for (int k = 0; k < NP; ++k) ss = ffma2(U::get(r[m], k), U::get(r[m], k), ss);
    float rho[1] = {hsum2(ss)};
    group_sum(rho, red, turn, group, tpr);
    turn ^= 1;
    rho[0] = inv_rms_of(rho[0], a.H, a.eps);
    if (c0 == 0 && a.rstd_pre) a.rstd_pre[t] = rho[0];
    const u64 rho2 = pair2(rho[0], rho[0]);
#pragma unroll
    for (int m = 0; m < NU; ++m) {
      u64 w[NP], v[NP];
      U::cols(w_pre, m, c0, tpr, w);
#pragma unroll
      for (int k = 0; k < NP; ++k) v[k] = fmul2(fmul2(U::get(r[m], k), rho2), w[k]);
      U::store(a.n, base, m, c0, tpr, nv, v);
    }
  }
  if constexpr (U::kAsync) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ----------------------------------------------------------------- backward
// With v = w_pre dn, e = dr + rho_r v, D = e - r rho_r^3 c_r and q = g D, the
// two row means are linear in three sums that one pass over the row gives:
//   c_r = S1 / H,  S1 = sum r v
//   c_f = (S2 - rho_r^3 c_r S3) / H,  S2 = sum (f w_post g) e,
//                                     S3 = sum (f w_post g) r
// so a row costs one reduction.  A channel gate's two column sums are one,
//   M = sum_t D f rho_f:  d_post_w = g M,  d_gate = w_post M
// (a token gate has only d_post_w = sum_t g D f rho_f), so a thread keeps two
// sums per column of its own over all rows of its group; the groups of a block
// are added through shared memory, the blocks by a second kernel.  Products
// and sums run on pairs (fma.rn.f32x2): with plain fp32 instructions the issue
// slots, not DRAM, set the time (1654 instructions a row of 768 columns).
constexpr int kBnBwdThreads = 512;      // 128 registers a thread
constexpr int kBnSums = 2;              // d_pre_w, M

// Column h of sum q, complete: to the gradients that follow from it.
template <typename T>
__device__ __forceinline__ void bn_finish(const BlockNormBwd& a, int q, int h, float s) {
  if (q == 0) {
    if (a.d_pre_w) a.d_pre_w[h] = s;
    return;
  }
  float* d_gate = a.gate && !a.gate_per_token ? static_cast<float*>(a.d_gate) : nullptr;
  if (a.d_post_w) a.d_post_w[h] = d_gate ? s * bn_param<T>(a.gate, h) : s;
  if (d_gate) d_gate[h] = a.post_w ? s * bn_param<T>(a.post_w, h) : s;
}

// No tokens: zeros, whatever the parameters hold.
__device__ __forceinline__ void bn_zero(const BlockNormBwd& a, int q, int h) {
  if (q == 0) {
    if (a.d_pre_w) a.d_pre_w[h] = 0.f;
    return;
  }
  if (a.d_post_w) a.d_post_w[h] = 0.f;
  if (a.gate && !a.gate_per_token) static_cast<float*>(a.d_gate)[h] = 0.f;
}

// NU units a thread.  The next row's inputs are copied to shared memory with
// cp.async while this one is worked on (`stages` 2; 1 where two do not fit):
// each thread copies and reads its own slots only, so the ring needs no
// barrier, and its registers hold only sums and D.  Without it a group's
// loads, reduction and stores follow one another and DRAM idles between them
// (T = 16384, H = 768, bf16: 41 us, with it 31 us, of which the second kernel
// takes 3; the bytes take 22 us at the measured copy rate).  Rows that are not
// 16-byte aligned load into registers: cp.async of 4 bytes took 74 us where
// plain loads take 26 (T = 4097, H = 1001, fp32; 15 us at the copy rate).
// Dynamic shared memory: w_pre and w_post g by column (`span` floats each: the
// columns of every unit, zeros behind the row), then the ring
// [stages][inputs][NU][threads], in whose place [groups][kBnSums][span] stands
// at the end.

// c += a * b where `on`, by a predicate.  (In the norm's backward, T = 16384, H
// = 768, bf16: 31.2 us with a channel gate, 31.5 with a branch around all of a
// unit's sums; with a token gate, whose registers are all taken, 41.9 and 40.7.)
__device__ __forceinline__ void fma2_if(bool on, u64& c, u64 a, u64 b) {
  asm("{\n.reg .pred p;\nsetp.ne.u32 p, %3, 0;\n@p fma.rn.f32x2 %0, %1, %2, %0;\n}"
      : "+l"(c)
      : "l"(a), "l"(b), "r"(static_cast<uint32_t>(on)));
}

enum BnInput { kInR, kInDn, kInDr, kInF, kInGate, kBnInputs };

template <typename T, int V, int NU, bool kTokenGate>
__global__ void __launch_bounds__(kBnBwdThreads, 1)
block_norm_bwd_kernel(const BlockNormBwd a, int tpr, int span, int stages) {
  using U = Unit<T, V>;
  typedef typename U::Raw Raw;
  constexpr int NP = U::kPairs;
  extern __shared__ __align__(16) float bn_smem[];
  __shared__ float red[2 * 3 * kBnBwdThreads / 32];
  float* w_pre = bn_smem;
  float* w_mid = bn_smem + span;
  float* behind = bn_smem + 2 * span;
  const int group = threadIdx.x / tpr, c0 = threadIdx.x - group * tpr, nv = a.H / V;
  const int groups = blockDim.x / tpr;
  constexpr int kIn = kTokenGate ? kBnInputs : kBnInputs - 1;
  const void* src[kBnInputs] = {a.pre_w ? a.r : nullptr, a.pre_w ? a.dn : nullptr, a.dr, a.f,
                                kTokenGate ? a.gate : nullptr};
  // the thread's slots, a warp's side by side: stage, input i, unit m, lane
  constexpr int kStageBytes = kIn * NU * 32 * static_cast<int>(sizeof(Raw));
  unsigned char* ring = reinterpret_cast<unsigned char*>(behind) + (threadIdx.x >> 5) * (stages * kStageBytes) +
                        (threadIdx.x & 31) * sizeof(Raw);
  auto at = [](int i, int m) { return (i * NU + m) * 32 * static_cast<int>(sizeof(Raw)); };
  Raw reg[U::kAsync ? 1 : kIn][U::kAsync ? 1 : NU];
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.T)
#pragma unroll
      for (int i = 0; i < kIn; ++i)
        if (src[i])
#pragma unroll
          for (int m = 0; m < NU; ++m) {
            if constexpr (U::kAsync)
              U::copy(smem_u32(ring + stage * kStageBytes) + at(i, m), src[i], t * a.H, m, c0, tpr, nv);
            else
              reg[i][m] = U::load(src[i], t * a.H, m, c0, tpr, nv);
          }
    if constexpr (U::kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (U::kAsync) {                  // what no copy will fill stays zero
    for (int st = 0; st < stages; ++st)
#pragma unroll
      for (int i = 0; i < kIn; ++i)
#pragma unroll
        for (int m = 0; m < NU; ++m)
          if (src[i] == nullptr || c0 + m * tpr >= nv)
            *reinterpret_cast<Raw*>(ring + st * kStageBytes + at(i, m)) = U::zero();
  } else {
#pragma unroll
    for (int i = 0; i < kIn; ++i)
#pragma unroll
      for (int m = 0; m < NU; ++m) reg[i][m] = U::zero();
  }
  auto value = [&](const unsigned char* here, int i, int m) -> Raw {
    if constexpr (U::kAsync) return *reinterpret_cast<const Raw*>(here + at(i, m));
    else return reg[i][m];
  };
  pdl_enter();
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group;
  float next_r = 0.f, next_f = 1.f;
  auto fetch_rstd = [&](int64_t row) {
    if (row >= a.T) return;
    if (a.pre_w) next_r = a.rstd_pre[row];
    if (a.post_w) next_f = a.rstd_post[row];
  };
  if (U::kAsync && stages == 2) fetch(t, 0);
  fetch_rstd(t);
  stage_params<T, V, kTokenGate>(a.pre_w, a.post_w, a.gate, a.H, tpr, span, w_pre, w_mid);
  __syncthreads();
  u64 s_pre[NU][NP], s_mid[NU][NP];
#pragma unroll
  for (int m = 0; m < NU; ++m)
#pragma unroll
    for (int k = 0; k < NP; ++k) s_pre[m][k] = s_mid[m][k] = 0;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const u64 scale2 = pair2(a.residual_scale, a.residual_scale);
  const bool post = a.post_w != nullptr;
  int turn = 0, stage = 0;
  for (; t < a.T; t += step) {
    const int64_t base = t * a.H;
    const float rho_r = next_r, rho_f = next_f;
    if (U::kAsync && stages == 2) {
      fetch(t + step, stage ^ 1);
      fetch_rstd(t + step);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      fetch(t, 0);
      fetch_rstd(t + step);
      if constexpr (U::kAsync) asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    const unsigned char* here = ring + stage * kStageBytes;
    const u64 rho_r2 = pair2(rho_r, rho_r), rho_f2 = pair2(rho_f, rho_f);
    u64 s1 = 0, s2 = 0, s3 = 0;
    u64 e[NU][NP];
#pragma unroll
    for (int m = 0; m < NU; ++m) {
      u64 wp[NP], wm[NP];
      U::cols(w_pre, m, c0, tpr, wp);
      U::cols(w_mid, m, c0, tpr, wm);
      const Raw r = value(here, kInR, m), dn = value(here, kInDn, m), dr = value(here, kInDr, m);
      const Raw f = value(here, kInF, m), g = kTokenGate ? value(here, kInGate, m) : U::zero();
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const u64 rk = U::get(r, k), nk = U::get(dn, k);
        const u64 v = fmul2(nk, wp[k]);
        s_pre[m][k] = ffma2(nk, fmul2(rk, rho_r2), s_pre[m][k]);
        s1 = ffma2(rk, v, s1);
        e[m][k] = ffma2(rho_r2, v, U::get(dr, k));
        u64 fw = fmul2(U::get(f, k), wm[k]);
        if constexpr (kTokenGate) fw = fmul2(fw, U::get(g, k));
        s2 = ffma2(fw, e[m][k], s2);
        s3 = ffma2(fw, rk, s3);
      }
    }
    float s[3] = {hsum2(s1), hsum2(s2), hsum2(s3)};
    group_sum(s, red, turn, group, tpr);
    turn ^= 1;
    const float k_r = rho_r * rho_r * (s[0] * inv_h) * rho_r;               // rho_r^3 c_r
    const float k_f = post ? rho_f * rho_f * ((s[1] - k_r * s[2]) * inv_h) : 0.f;  // rho_f^2 c_f
    const u64 k_r2 = pair2(-k_r, -k_r), k_f2 = pair2(-k_f * rho_f, -k_f * rho_f);
#pragma unroll
    for (int m = 0; m < NU; ++m) {
      u64 wm[NP], o[NP];
      U::cols(w_mid, m, c0, tpr, wm);
      const Raw r = value(here, kInR, m);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        e[m][k] = ffma2(U::get(r, k), k_r2, e[m][k]);                       // D
        o[k] = fmul2(scale2, e[m][k]);
      }
      U::store(a.dx, base, m, c0, tpr, nv, o);
      if (a.df == nullptr) continue;
      const Raw f = value(here, kInF, m), g = kTokenGate ? value(here, kInGate, m) : U::zero();
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const u64 fk = U::get(f, k);
        u64 d = fmul2(e[m][k], rho_f2);                                     // D rho_f
        if constexpr (kTokenGate) {
          o[k] = fmul2(fmul2(d, fk), wm[k]);                                // wm is w_post here
          d = fmul2(d, U::get(g, k));
        }
        s_mid[m][k] = ffma2(d, fk, s_mid[m][k]);
        // without a post norm df = q whatever f holds: an infinite one times k_f = 0 would be a NaN
        e[m][k] = fmul2(wm[k], d);
        if constexpr (!kTokenGate) fma2_if(post, e[m][k], fk, k_f2);
      }
      if (kTokenGate && post)
#pragma unroll
        for (int k = 0; k < NP; ++k) e[m][k] = ffma2(U::get(f, k), k_f2, e[m][k]);
      if constexpr (kTokenGate) U::store(a.d_gate, base, m, c0, tpr, nv, o);
      U::store(a.df, base, m, c0, tpr, nv, e[m]);
    }
    if (U::kAsync && stages == 2) stage ^= 1;
  }
  // the block's column sums: each group's side by side, then added in order
  if constexpr (U::kAsync) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (gridDim.x > 1 && a.partial == nullptr) return;                          // none asked for
  __syncthreads();
  float* mine = behind + group * kBnSums * span;
#pragma unroll
  for (int m = 0; m < NU; ++m) {
    U::keep(mine, m, c0, tpr, nv, s_pre[m]);
    U::keep(mine + span, m, c0, tpr, nv, s_mid[m]);
  }
  __syncthreads();
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * kBnSums * a.H;   // not used by one block
  using P = Pack<T, V>;
  const bool one = gridDim.x == 1, chan_gate = a.gate != nullptr && !kTokenGate;
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    typename P::Raw gate, post;
    if (one && chan_gate) gate = row_load<T, V>(a.gate, 0, c);
    if (one && a.post_w) post = row_load<T, V>(a.post_w, 0, c);
    float sum[kBnSums][V];
#pragma unroll
    for (int q = 0; q < kBnSums; ++q) {
#pragma unroll
      for (int j = 0; j < V; ++j) sum[q][j] = 0.f;
      for (int gi = 0; gi < groups; ++gi) {
        const float* from = behind + (gi * kBnSums + q) * span;
        if constexpr (V == 1) {
          sum[q][0] += from[c];
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(from + U::place(c * V + j, tpr));
            sum[q][j] += x.x;
            sum[q][j + 1] += x.y;
            sum[q][j + 2] += x.z;
            sum[q][j + 3] += x.w;
          }
        }
      }
    }
    if (!one) {
#pragma unroll
      for (int q = 0; q < kBnSums; ++q)
#pragma unroll
        for (int j = 0; j < V; ++j) part[q * a.H + c * V + j] = sum[q][j];
      continue;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {             // complete: as bn_finish
      const int h = c * V + j;
      if (a.d_pre_w) a.d_pre_w[h] = sum[0][j];
      if (a.d_post_w) a.d_post_w[h] = chan_gate ? sum[1][j] * P::get(gate, j) : sum[1][j];
      if (chan_gate) static_cast<float*>(a.d_gate)[h] = a.post_w ? sum[1][j] * P::get(post, j) : sum[1][j];
    }
  }
}

// Rows too wide for a block's registers: the block walks the row twice (the
// second time from L2), and keeps its column sums in shared memory, each
// column owned by one thread.
template <typename T, int V>
__global__ void __launch_bounds__(kBnFwdThreads, 1) block_norm_bwd_wide_kernel(const BlockNormBwd a) {
  using P = Pack<T, V>;
  pdl_enter();
  __shared__ float red[2 * 3 * kBnFwdThreads / 32];
  extern __shared__ __align__(16) float bn_smem[];   // [2][H]
  float* cols = bn_smem;
  const int nv = a.H / V;
  const bool token_gate = a.gate != nullptr && a.gate_per_token;
  for (int c = threadIdx.x; c < nv; c += kBnFwdThreads)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < kBnSums; ++q) cols[q * a.H + c * V + j] = 0.f;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t base = t * a.H, gbase = a.gate_per_token ? base : 0;
    const float rho_r = a.pre_w ? a.rstd_pre[t] : 0.f;
    const float rho_f = a.post_w ? a.rstd_post[t] : 1.f;
    float s[3] = {0.f, 0.f, 0.f};
    float k_r = 0.f, k_f = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int c = threadIdx.x; c < nv; c += kBnFwdThreads) {
        float d[V], f[V], w[V], g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          d[j] = f[j] = 0.f;
          w[j] = g[j] = 1.f;
        }
        if (a.dr) {
          const auto x = row_load<T, V>(a.dr, base, c);
#pragma unroll
          for (int j = 0; j < V; ++j) d[j] = P::get(x, j);
        }
        if (a.f) {
          const auto x = row_load<T, V>(a.f, base, c);
#pragma unroll
          for (int j = 0; j < V; ++j) f[j] = P::get(x, j);
        }
        if (a.post_w) {
          const auto x = row_load<T, V>(a.post_w, 0, c);
#pragma unroll
          for (int j = 0; j < V; ++j) w[j] = P::get(x, j);
        }
        if (a.gate) {
          const auto x = row_load<T, V>(a.gate, gbase, c);
#pragma unroll
          for (int j = 0; j < V; ++j) g[j] = P::get(x, j);
        }
        if (a.pre_w) {
          const auto xr = row_load<T, V>(a.r, base, c);
          const auto xd = row_load<T, V>(a.dn, base, c);
          const auto xw = row_load<T, V>(a.pre_w, 0, c);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float r = P::get(xr, j), dn = P::get(xd, j), v = dn * P::get(xw, j);
            if (pass == 0) {
              s[0] = fmaf(r, v, s[0]);
              s[2] = fmaf(f[j] * w[j] * g[j], r, s[2]);
              d[j] = fmaf(rho_r, v, d[j]);
            } else {
              d[j] = fmaf(rho_r, fmaf(-r, k_r, v), d[j]);
              cols[c * V + j] = fmaf(dn, r * rho_r, cols[c * V + j]);
            }
          }
        }
        if (pass == 0) {
#pragma unroll
          for (int j = 0; j < V; ++j) s[1] = fmaf(f[j] * w[j] * g[j], d[j], s[1]);
          continue;
        }
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = a.residual_scale * d[j];
        row_store<T, V>(a.dx, base, c, o);
        if (a.df == nullptr) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = d[j] * (f[j] * rho_f * w[j]);
        if (token_gate) row_store<T, V>(a.d_gate, base, c, o);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int h = c * V + j;
          const float q = d[j] * g[j];
          cols[a.H + h] = fmaf(token_gate ? q : d[j], f[j] * rho_f, cols[a.H + h]);
          d[j] = a.post_w ? rho_f * fmaf(-f[j], k_f, w[j] * q) : q;
        }
        row_store<T, V>(a.df, base, c, d);
      }
      if (pass == 0) {
        group_sum(s, red, turn, 0, kBnFwdThreads);
        turn ^= 1;
        const float inv_h = 1.0f / static_cast<float>(a.H);
        k_r = rho_r * rho_r * (s[0] * inv_h);
        k_f = rho_f * rho_f * ((s[1] - rho_r * k_r * s[2]) * inv_h);
      }
    }
  }
  if (gridDim.x > 1 && a.partial == nullptr) return;          // no sums asked for
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * kBnSums * a.H;
  for (int c = threadIdx.x; c < nv; c += kBnFwdThreads)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < kBnSums; ++q) {
        const int h = c * V + j;
        if (gridDim.x == 1) bn_finish<T>(a, q, h, cols[q * a.H + h]);
        else part[q * a.H + h] = cols[q * a.H + h];
      }
}

// Sums over the blocks' partials: 32 columns x 32 slices of the blocks per
// block of threads (five loads a thread, all in flight; 8 slices took 6 us at
// H = 768), slices added in order; grid.y: 0 d_pre_w, 1 what follows from M.
constexpr int kBnSlices = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kBnSlices)
block_norm_bwd_sum_kernel(const BlockNormBwd a, int nblk) {
  pdl_enter();
  __shared__ float red[kBnSlices][32];
  const int h = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5, q = blockIdx.y;
  if (q == 0 ? a.d_pre_w == nullptr : (a.d_post_w == nullptr && (a.gate == nullptr || a.gate_per_token))) return;
  float s = 0.f;
  if (h < a.H)
#pragma unroll 8
    for (int b = slice; b < nblk; b += kBnSlices)
      s += a.partial[(static_cast<int64_t>(b) * kBnSums + q) * a.H + h];
  red[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && h < a.H) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kBnSlices; ++i) s += red[i][threadIdx.x];
    if (nblk > 0) bn_finish<T>(a, q, h, s);
    else bn_zero(a, q, h);
  }
}

// ----------------------------------------------------------------- launches
static inline int bn_vec(int dtype, int H) {
  const int v = dtype == kDtypeBF16 ? 8 : 4;
  return H % v == 0 ? v : 1;
}
// Threads of a row's group with NV vectors each.
static inline int bn_tpr(int nv, int NV) { return (nv + 32 * NV - 1) / (32 * NV) * 32; }

// Backward: a thread takes up to 24 elements of bf16 (three 16-byte vectors
// of each input), 16 of fp32 or 8 of an unaligned width, as its registers
// allow; the most threads with columns decide between the unit counts, two
// units where that is equal (H = 1024, fp32: 38 us, with one 41, with four
// 43).  A row that needs more than a block's threads so is `wide`.
template <int V> struct BnUnits;
template <> struct BnUnits<8> { static constexpr int kMost = 3, kSome = 2, kFew = 1; };
template <> struct BnUnits<4> { static constexpr int kMost = 4, kSome = 2, kFew = 1; };
template <> struct BnUnits<1> { static constexpr int kMost = 4, kSome = 2, kFew = 1; };

struct BnBwdShape {
  int V, NU, tpr, groups, grid, span;
  bool wide;
};
template <int V>
static BnBwdShape bn_bwd_shape_v(int64_t T, int H) {
  using N = BnUnits<V>;
  constexpr int width = V == 1 ? 2 : V;       // elements of a unit
  BnBwdShape s{V, 0, 0, 1, 1, 0, false};
  int best = 0;
  for (int NU : {N::kSome, N::kMost, N::kFew}) {
    const int tpr = (H + 32 * NU * width - 1) / (32 * NU * width) * 32;
    if (tpr > kBnBwdThreads) continue;
    const int busy = kBnBwdThreads / tpr * ((H + NU * width - 1) / (NU * width));   // threads with columns
    if (busy > best) {
      best = busy;
      s.NU = NU;
      s.tpr = tpr;
    }
  }
  const int64_t sms = num_sms();
  if (s.NU == 0) {
    s.wide = true;
    s.tpr = kBnFwdThreads;
    s.grid = static_cast<int>(T < sms ? (T > 0 ? T : 1) : sms);
    return s;
  }
  s.span = s.NU * s.tpr * width;
  // one block an SM: a second wave costs a block's start and its sums again
  // (T = 16384: 31 -> 34 us at H = 768, 124 -> 131 us at H = 4096)
  s.groups = kBnBwdThreads / s.tpr;
  // few rows: one block, which needs no second kernel, where its groups take a
  // row each or, being many, two (T = 10, H = 896, bf16: 7.5 us, of which the
  // second kernel would add 2)
  if (T <= (V > 1 && s.groups >= 8 ? 2 : 1) * s.groups) return s;
  const int64_t want = (T + s.groups - 1) / s.groups;
  s.grid = static_cast<int>(want < sms ? (want > 0 ? want : 1) : sms);
  return s;
}
static BnBwdShape bn_bwd_shape(int64_t T, int H, int dtype) {
  const int v = bn_vec(dtype, H);
  return v == 8 ? bn_bwd_shape_v<8>(T, H) : v == 4 ? bn_bwd_shape_v<4>(T, H) : bn_bwd_shape_v<1>(T, H);
}

size_t block_norm_bwd_bytes(int64_t T, int H, int dtype) {
  if (T == 0) return 0;
  return 4 * static_cast<size_t>(bn_bwd_shape(T, H, dtype).grid) * kBnSums * H;
}

template <typename T, int V, int NV>
static cudaError_t bn_fwd_launch(const BlockNormFwd& a, int tpr, cudaStream_t st) {
  const int groups = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t blocks = (a.T + groups - 1) / groups;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(block_norm_kernel<T, V, NV>, dim3(static_cast<unsigned>(blocks)),
                                 dim3(groups * tpr), 0, st, a, tpr);
}

// The ring, where two rows of every group fit beside the parameters.  Not
// where many rows would go through a block one at a time, each waiting for its
// sums: there one block per row leaves several on an SM (bf16, 30 M elements:
// H = 5120, two groups, 44 us against 50; H = 8192, one group, 50 against 44).
// cudaErrorNotSupported: not here.
// A thread takes up to 24 elements of an aligned row (16 of fp32 with a token
// gate, whose three inputs of 24 never fit), or 16 / 8 of an unaligned one.
template <typename T, int V, bool kTokenGate> struct BnFwdUnits {
  static constexpr int kWidth = V == 1 ? 2 : V;           // elements of a unit
  static constexpr int kMost = V == 1 ? 16 / static_cast<int>(sizeof(T)) : (sizeof(T) == 4 && kTokenGate ? 16 : 24) / V;
  static constexpr int kSome = V > 1 ? 16 / V : kMost / 2, kFew = V > 1 ? 8 / V : kMost / 4;
  // dynamic shared memory of blocks of `groups` groups of tpr threads, NU units each
  static size_t smem(int NU, int tpr, int groups) {
    const size_t span = static_cast<size_t>(NU) * tpr * kWidth;
    return 2 * sizeof(float) * span + (V > 1 ? 2 * (kTokenGate ? 3 : 2) * sizeof(T) * span * groups : 0);
  }
};
template <typename T, int V, int NU, bool kTokenGate>
static cudaError_t bn_ring_launch(const BlockNormFwd& a, int tpr, cudaStream_t st) {
  using N = BnFwdUnits<T, V, kTokenGate>;
  const int span = NU * tpr * N::kWidth, groups = kBnFwdThreads / tpr;
  const size_t smem = N::smem(NU, tpr, groups);
  const int64_t sms = num_sms();
  auto kern = block_norm_ring_kernel<T, V, NU, kTokenGate>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  // Three waves of blocks where an SM's share is above 2 MB, else one: the SMs
  // do not run at one pace, so an even share waits for the slowest, but each
  // block starts with a load it has nothing to run under (1 / 3 waves, us:
  // 268 MB 46.6 / 50.5, 403 MB 68.1 / 63.2, 671 MB 108 / 100).
  const int64_t share = a.T * a.H * static_cast<int64_t>(sizeof(T)) * (2 + kTokenGate + 1 + (a.pre_w != nullptr)) / sms;
  const int64_t most = share > (2 << 20) ? 3 * sms : sms;
  return launch_dependent_kernel(kern, dim3(static_cast<unsigned>(a.T < most ? a.T : most)), dim3(groups * tpr), smem,
                                 st, a, tpr, span);
}
template <typename T, int V, bool kTokenGate>
static cudaError_t bn_ring_pick(const BlockNormFwd& a, cudaStream_t st) {
  using N = BnFwdUnits<T, V, kTokenGate>;
  int best = 0, busy = 0, tpr = 0;
  for (int NU : {N::kSome, N::kMost, N::kFew}) {          // the most threads with columns, of what fits
    const int lanes = (a.H + NU * N::kWidth - 1) / (NU * N::kWidth), t = (lanes + 31) / 32 * 32;
    if (t > kBnFwdThreads || N::smem(NU, t, kBnFwdThreads / t) > kBnMostSmem) continue;
    const int b = kBnFwdThreads / t * lanes;
    if (b > busy) {
      busy = b;
      best = NU;
      tpr = t;
    }
  }
  if (best == 0 || (V > 1 && kBnFwdThreads / tpr == 1 && a.T > 4 * static_cast<int64_t>(num_sms())))
    return cudaErrorNotSupported;
  if (best == N::kMost) return bn_ring_launch<T, V, N::kMost, kTokenGate>(a, tpr, st);
  if (best == N::kSome) return bn_ring_launch<T, V, N::kSome, kTokenGate>(a, tpr, st);
  return bn_ring_launch<T, V, N::kFew, kTokenGate>(a, tpr, st);
}

template <typename T, int V>
static cudaError_t bn_fwd_pick(const BlockNormFwd& a, cudaStream_t st) {
  const bool token_gate = a.gate != nullptr && a.gate_per_token;
  const cudaError_t ring = token_gate ? bn_ring_pick<T, V, true>(a, st) : bn_ring_pick<T, V, false>(a, st);
  if (ring != cudaErrorNotSupported) return ring;
  // 32 or 24 elements a thread, whichever leaves fewer idle
  const int nv = a.H / V;
  constexpr int kMost = 32 / V, kSome = 24 / V;
  const int tpr = bn_tpr(nv, kSome);
  if (tpr <= kBnFwdThreads && kSome * tpr < kMost * bn_tpr(nv, kMost)) return bn_fwd_launch<T, V, kSome>(a, tpr, st);
  return bn_fwd_launch<T, V, kMost>(a, bn_tpr(nv, kMost), st);
}

cudaError_t launch_block_norm(int dtype, const BlockNormFwd& a, cudaStream_t st) {
  if (dtype == kDtypeBF16)
    return a.H % 8 == 0 ? bn_fwd_pick<__nv_bfloat16, 8>(a, st) : bn_fwd_pick<__nv_bfloat16, 1>(a, st);
  return a.H % 4 == 0 ? bn_fwd_pick<float, 4>(a, st) : bn_fwd_pick<float, 1>(a, st);
}

template <typename T, int V, int NU>
static cudaError_t bn_bwd_launch(const BlockNormBwd& a, const BnBwdShape& s, cudaStream_t st) {
  using U = Unit<T, V>;
  const bool token_gate = a.gate != nullptr && a.gate_per_token;
  auto kern = token_gate ? block_norm_bwd_kernel<T, V, NU, true> : block_norm_bwd_kernel<T, V, NU, false>;
  const size_t threads = static_cast<size_t>(s.groups) * s.tpr;
  const size_t cols = 2 * sizeof(float) * s.span, sums = kBnSums * sizeof(float) * s.span * s.groups;
  const size_t stage = U::kAsync ? (kBnInputs - !token_gate) * NU * threads * sizeof(typename U::Raw) : 0;
  const int stages = cols + 2 * stage <= kBnMostSmem ? 2 : 1;
  const size_t smem = cols + (stages * stage > sums ? stages * stage : sums);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_dependent_kernel(kern, dim3(s.grid), dim3(static_cast<unsigned>(threads)), smem, st, a,
                                 s.tpr, s.span, stages);
}

template <typename T, int V>
static cudaError_t bn_bwd_pick(const BlockNormBwd& a, const BnBwdShape& s, cudaStream_t st) {
  if (s.wide) {
    auto kern = block_norm_bwd_wide_kernel<T, V>;
    const size_t smem = sizeof(float) * kBnSums * a.H;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_dependent_kernel(kern, dim3(s.grid), dim3(kBnFwdThreads), smem, st, a);
  }
  using N = BnUnits<V>;
  if (s.NU == N::kMost) return bn_bwd_launch<T, V, N::kMost>(a, s, st);
  if (s.NU == N::kSome) return bn_bwd_launch<T, V, N::kSome>(a, s, st);
  return bn_bwd_launch<T, V, N::kFew>(a, s, st);
}

cudaError_t launch_block_norm_bwd_rows(int dtype, const BlockNormBwd& a, cudaStream_t st) {
  const BnBwdShape s = bn_bwd_shape(a.T, a.H, dtype);
  if (dtype == kDtypeBF16)
    return s.V == 8 ? bn_bwd_pick<__nv_bfloat16, 8>(a, s, st) : bn_bwd_pick<__nv_bfloat16, 1>(a, s, st);
  return s.V == 4 ? bn_bwd_pick<float, 4>(a, s, st) : bn_bwd_pick<float, 1>(a, s, st);
}

bool block_norm_bwd_one_block(int64_t T, int H, int dtype) {
  return T > 0 && bn_bwd_shape(T, H, dtype).grid == 1;
}

cudaError_t launch_block_norm_bwd_cols(int dtype, const BlockNormBwd& a, cudaStream_t st) {
  const int nblk = a.T > 0 ? bn_bwd_shape(a.T, a.H, dtype).grid : 0;
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, dim3((a.H + 31) / 32, kBnSums), dim3(32 * kBnSlices), 0, st, a, nblk);
  };
  return dtype == kDtypeBF16 ? run(block_norm_bwd_sum_kernel<__nv_bfloat16>)
                             : run(block_norm_bwd_sum_kernel<float>);
}

}  // namespace mm
