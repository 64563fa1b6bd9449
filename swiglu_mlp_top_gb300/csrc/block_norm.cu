// Norms before and after a block, fused with its gate and residual scale,
// and the gradient (include/mm.h, mm_block_norm):
//   p = f rho_f w_post,  rho_f = 1 / sqrt(mean_h f^2 + eps)     (w_post absent: p = f)
//   r = round(s x + g p)                                        (g absent: 1)
//   n = r rho_r w_pre,   rho_r of the rounded r
// One block per row, fp32 sums in a fixed order.
#include <cstring>

#include "mm_kernels.cuh"

namespace mm {

constexpr int kBnThreads = 256;

__device__ __forceinline__ float bn_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float bn_load(const float* p) { return *p; }
__device__ __forceinline__ void bn_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void bn_store(float* p, float v) { *p = v; }
template <typename T> __device__ __forceinline__ float bn_round(float v);
template <> __device__ __forceinline__ float bn_round<float>(float v) { return v; }
template <> __device__ __forceinline__ float bn_round<__nv_bfloat16>(float v) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// Sum over the block, the same value and order in every thread.
__device__ __forceinline__ float bn_block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kBnThreads / 32; ++w) s += red[w];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kBnThreads) block_norm_kernel(const BlockNormFwd a) {
  pdl_enter();
  __shared__ float red[kBnThreads / 32];
  extern __shared__ float row[];           // r of the row, fp32
  const int H = a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + t * H;
    const T* f = a.f ? static_cast<const T*>(a.f) + t * H : nullptr;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + (a.gate_per_token ? t * H : 0) : nullptr;
    float rho_f = 1.f;
    if (a.post_w) {
      float ss = 0.f;
      for (int h = threadIdx.x; h < H; h += kBnThreads) {
        const float v = bn_load(f + h);
        ss = fmaf(v, v, ss);
      }
      rho_f = 1.0f / sqrtf(bn_block_sum(ss, red) / static_cast<float>(H) + a.eps);
      if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[t] = rho_f;
    }
    float ss = 0.f;
    for (int h = threadIdx.x; h < H; h += kBnThreads) {
      float v = bn_load(x + h);
      if (f) {
        float p = bn_load(f + h);
        if (a.post_w) p = p * rho_f * bn_load(static_cast<const T*>(a.post_w) + h);
        if (gate) p *= bn_load(gate + h);
        v = bn_round<T>(fmaf(a.residual_scale, v, p));
        bn_store(static_cast<T*>(a.r) + t * H + h, v);
      }
      row[h] = v;
      ss = fmaf(v, v, ss);
    }
    if (a.pre_w) {
      const float rho_r = 1.0f / sqrtf(bn_block_sum(ss, red) / static_cast<float>(H) + a.eps);
      if (threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[t] = rho_r;
      for (int h = threadIdx.x; h < H; h += kBnThreads)
        bn_store(static_cast<T*>(a.n) + t * H + h,
                 row[h] * rho_r * bn_load(static_cast<const T*>(a.pre_w) + h));
    }
  }
}

// D = dr + rho_r (w_pre dn) - r rho_r^3 c_r,  c_r = mean_h(r w_pre dn)
template <typename T>
__device__ __forceinline__ float bn_grad_r(const BlockNormBwd& a, int64_t t, int h, float rho_r,
                                           float c_r) {
  const int64_t i = t * a.H + h;
  float d = a.dr ? bn_load(static_cast<const T*>(a.dr) + i) : 0.f;
  if (a.pre_w) {
    const float v = bn_load(static_cast<const T*>(a.dn) + i) * bn_load(static_cast<const T*>(a.pre_w) + h);
    d += rho_r * (v - bn_load(static_cast<const T*>(a.r) + i) * (rho_r * rho_r * c_r));
  }
  return d;
}

template <typename T>
__global__ void __launch_bounds__(kBnThreads) block_norm_bwd_rows_kernel(const BlockNormBwd a) {
  pdl_enter();
  __shared__ float red[kBnThreads / 32];
  const int H = a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + (a.gate_per_token ? t * H : 0) : nullptr;
    float rho_r = 0.f, c_r = 0.f;
    if (a.pre_w) {
      rho_r = a.rstd_pre[t];
      float s = 0.f;
      for (int h = threadIdx.x; h < H; h += kBnThreads)
        s = fmaf(bn_load(static_cast<const T*>(a.r) + t * H + h) * bn_load(static_cast<const T*>(a.pre_w) + h),
                 bn_load(static_cast<const T*>(a.dn) + t * H + h), s);
      c_r = bn_block_sum(s, red) / static_cast<float>(H);
    }
    if (threadIdx.x == 0) a.partial[t] = c_r;
    float rho_f = 1.f, c_f = 0.f;
    if (a.post_w) {
      rho_f = a.rstd_post[t];
      float s = 0.f;
      for (int h = threadIdx.x; h < H; h += kBnThreads) {
        float q = bn_grad_r<T>(a, t, h, rho_r, c_r);
        if (gate) q *= bn_load(gate + h);
        s = fmaf(bn_load(static_cast<const T*>(a.f) + t * H + h) * bn_load(static_cast<const T*>(a.post_w) + h), q, s);
      }
      c_f = bn_block_sum(s, red) / static_cast<float>(H);
    }
    for (int h = threadIdx.x; h < H; h += kBnThreads) {
      const int64_t i = t * H + h;
      const float d = bn_grad_r<T>(a, t, h, rho_r, c_r);
      bn_store(static_cast<T*>(a.dx) + i, a.residual_scale * d);
      if (a.df == nullptr) continue;
      const float f = a.f ? bn_load(static_cast<const T*>(a.f) + i) : 0.f;
      const float w = a.post_w ? bn_load(static_cast<const T*>(a.post_w) + h) : 1.f;
      const float q = gate ? d * bn_load(gate + h) : d;
      if (gate && a.gate_per_token) bn_store(static_cast<T*>(a.d_gate) + i, d * (f * rho_f * w));
      bn_store(static_cast<T*>(a.df) + i, a.post_w ? rho_f * (w * q - f * (rho_f * rho_f * c_f)) : q);
    }
  }
}

// Column sums over the tokens: one thread per column.
template <typename T>
__global__ void __launch_bounds__(kBnThreads) block_norm_bwd_cols_kernel(const BlockNormBwd a) {
  pdl_enter();
  const int h = blockIdx.x * kBnThreads + threadIdx.x;
  if (h >= a.H) return;
  const float w = a.post_w ? bn_load(static_cast<const T*>(a.post_w) + h) : 1.f;
  float s_pre = 0.f, s_post = 0.f, s_gate = 0.f;
  for (int64_t t = 0; t < a.T; ++t) {
    const int64_t i = t * a.H + h;
    const float rho_r = a.pre_w ? a.rstd_pre[t] : 0.f;
    if (a.pre_w)
      s_pre += bn_load(static_cast<const T*>(a.dn) + i) * (bn_load(static_cast<const T*>(a.r) + i) * rho_r);
    if (a.post_w == nullptr && (a.gate == nullptr || a.gate_per_token)) continue;
    const float d = bn_grad_r<T>(a, t, h, rho_r, a.partial[t]);
    const float u = bn_load(static_cast<const T*>(a.f) + i) * (a.post_w ? a.rstd_post[t] : 1.f);
    const float g = a.gate ? bn_load(static_cast<const T*>(a.gate) + (a.gate_per_token ? i : h)) : 1.f;
    s_post += d * g * u;
    s_gate += d * (u * w);
  }
  if (a.pre_w) a.d_pre_w[h] = s_pre;
  if (a.post_w) a.d_post_w[h] = s_post;
  if (a.gate && !a.gate_per_token) static_cast<float*>(a.d_gate)[h] = s_gate;
}

size_t block_norm_bwd_bytes(int64_t T, int H, int dtype) {
  (void)H;
  (void)dtype;
  return 4 * static_cast<size_t>(T);
}

static dim3 bn_row_grid(int64_t T) {
  const int64_t most = static_cast<int64_t>(num_sms()) * 8;
  return dim3(static_cast<unsigned>(T < most ? (T > 0 ? T : 1) : most));
}

cudaError_t launch_block_norm(int dtype, const BlockNormFwd& a, cudaStream_t st) {
  const size_t smem = 4 * static_cast<size_t>(a.H);
  auto run = [&](auto kern) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_dependent_kernel(kern, bn_row_grid(a.T), dim3(kBnThreads), smem, st, a);
  };
  return dtype == kDtypeBF16 ? run(block_norm_kernel<__nv_bfloat16>) : run(block_norm_kernel<float>);
}

cudaError_t launch_block_norm_bwd_rows(int dtype, const BlockNormBwd& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, bn_row_grid(a.T), dim3(kBnThreads), 0, st, a);
  };
  return dtype == kDtypeBF16 ? run(block_norm_bwd_rows_kernel<__nv_bfloat16>)
                             : run(block_norm_bwd_rows_kernel<float>);
}

cudaError_t launch_block_norm_bwd_cols(int dtype, const BlockNormBwd& a, cudaStream_t st) {
  const dim3 grid((a.H + kBnThreads - 1) / kBnThreads);
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, grid, dim3(kBnThreads), 0, st, a);
  };
  return dtype == kDtypeBF16 ? run(block_norm_bwd_cols_kernel<__nv_bfloat16>)
                             : run(block_norm_bwd_cols_kernel<float>);
}

}  // namespace mm
