// Tokens sorted by expert and back, with the routing weights, and the
// gradient (include/mm.h, mm_moe_permute).  Assignment a = t*k + s goes to
// row pos[a] = offset[e] + (number of assignments to e before a), where
// group e starts at offset[e], a multiple of `align`; an expert index
// outside [0, E) drops the assignment (pos -1).
#include "mm_kernels.cuh"

namespace mm {

constexpr int kPmThreads = 256;

__device__ __forceinline__ float pm_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float pm_load(const float* p) { return *p; }
__device__ __forceinline__ void pm_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void pm_store(float* p, float v) { *p = v; }

// One block: counts, offsets, then the ranks 32 assignments at a time.
__global__ void __launch_bounds__(kPmThreads) permute_sort_kernel(const PermuteArgs a) {
  pdl_enter();
  __shared__ int cnt[MM_MAX_EXPERTS], run[MM_MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t na = a.T * a.k;
  for (int e = tid; e < a.E; e += kPmThreads) cnt[e] = 0;
  __syncthreads();
  for (int64_t i = tid; i < na; i += kPmThreads) {
    const int e = a.topk_idx[i];
    if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid == 0) {
    int off = 0;
    for (int e = 0; e < a.E; ++e) {
      a.offsets[e] = off;
      a.counts[e] = cnt[e];
      run[e] = off;
      off += (cnt[e] + a.align - 1) / a.align * a.align;
    }
    a.offsets[a.E] = off;
  }
  __syncthreads();
  for (int64_t r = tid; r < a.rows; r += kPmThreads) a.perm[r] = -1;
  __syncthreads();
  if (tid < 32) {
    for (int64_t base = 0; base < na; base += 32) {
      const int64_t i = base + lane;
      int e = i < na ? a.topk_idx[i] : -1;
      const bool valid = e >= 0 && e < a.E;
      e = valid ? e : MM_MAX_EXPERTS + lane;
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      const unsigned below = peers & ((1u << lane) - 1u);
      const int prior = valid ? run[e] : 0;
      __syncwarp();
      if (i < na) a.pos[i] = valid ? prior + __popc(below) : -1;
      if (valid) {
        a.perm[prior + __popc(below)] = static_cast<int32_t>(i);
        if (below == 0u) run[e] = prior + __popc(peers);
      }
      __syncwarp();
    }
  }
}

// One block per row of the sorted tensor: a copy of its token's row, zeros
// where the group is padded, nothing behind the last group.
template <typename T>
__global__ void __launch_bounds__(kPmThreads) permute_copy_kernel(const PermuteArgs a) {
  pdl_enter();
  const int64_t end = a.offsets[a.E];
  for (int64_t r = blockIdx.x; r < end; r += gridDim.x) {
    const int src = a.perm[r];
    T* o = static_cast<T*>(a.xs) + r * a.H;
    const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(src < 0 ? 0 : src / a.k) * a.H;
    for (int h = threadIdx.x; h < a.H; h += kPmThreads) o[h] = src < 0 ? T(0.f) : x[h];
  }
}

template <typename T>
__global__ void __launch_bounds__(kPmThreads) unpermute_kernel(const UnpermuteArgs a) {
  pdl_enter();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
    for (int h = threadIdx.x; h < a.H; h += kPmThreads) {
      float acc = 0.f;
      for (int s = 0; s < a.k; ++s) {
        const int64_t p = a.pos[t * a.k + s];
        if (p < 0 || p >= a.rows) continue;
        const float v = pm_load(static_cast<const T*>(a.ys) + p * a.H + h);
        acc = a.w ? fmaf(a.w[t * a.k + s], v, acc) : acc + v;
      }
      pm_store(static_cast<T*>(a.y) + t * a.H + h, acc);
    }
}

// Blocks [0, T): one token each; blocks [T, T + E): one group's padding.
template <typename T>
__global__ void __launch_bounds__(kPmThreads) unpermute_bwd_kernel(const UnpermuteBwdArgs a) {
  pdl_enter();
  __shared__ float red[kPmThreads / 32];
  for (int64_t b = blockIdx.x; b < a.T + a.E; b += gridDim.x) {
    if (b >= a.T) {
      const int e = static_cast<int>(b - a.T);
      int64_t r0 = static_cast<int64_t>(a.offsets[e]) + a.counts[e], r1 = a.offsets[e + 1];
      if (r0 < 0) r0 = 0;
      if (r1 > a.rows) r1 = a.rows;
      for (int64_t i = r0 * a.H + threadIdx.x; i < r1 * a.H; i += kPmThreads)
        static_cast<T*>(a.dys)[i] = T(0.f);
      continue;
    }
    for (int s = 0; s < a.k; ++s) {
      const int64_t i = b * a.k + s, p = a.pos[i];
      const bool kept = p >= 0 && p < a.rows;
      const float w = a.w ? a.w[i] : 1.f;
      float dot = 0.f;
      if (kept)
        for (int h = threadIdx.x; h < a.H; h += kPmThreads) {
          const float g = pm_load(static_cast<const T*>(a.dy) + b * a.H + h);
          if (a.dw) dot = fmaf(g, pm_load(static_cast<const T*>(a.ys) + p * a.H + h), dot);
          pm_store(static_cast<T*>(a.dys) + p * a.H + h, w * g);
        }
      if (a.dw == nullptr) continue;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int q = 0; q < kPmThreads / 32; ++q) sum += red[q];
        a.dw[i] = sum;
      }
    }
  }
}

static dim3 pm_grid(int64_t n) {
  const int64_t most = static_cast<int64_t>(num_sms()) * 8;
  return dim3(static_cast<unsigned>(n < most ? (n > 0 ? n : 1) : most));
}

size_t permute_bytes(int64_t T, int E, int k) {
  (void)T;
  (void)E;
  (void)k;
  return 0;
}

cudaError_t launch_permute_sort(const PermuteArgs& a, cudaStream_t st) {
  return launch_dependent_kernel(permute_sort_kernel, dim3(1), dim3(kPmThreads), 0, st, a);
}
cudaError_t launch_permute_copy(int dtype, const PermuteArgs& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, pm_grid(a.rows), dim3(kPmThreads), 0, st, a);
  };
  return dtype == kDtypeBF16 ? run(permute_copy_kernel<__nv_bfloat16>) : run(permute_copy_kernel<float>);
}
cudaError_t launch_unpermute(int dtype, const UnpermuteArgs& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, pm_grid(a.T), dim3(kPmThreads), 0, st, a);
  };
  return dtype == kDtypeBF16 ? run(unpermute_kernel<__nv_bfloat16>) : run(unpermute_kernel<float>);
}
cudaError_t launch_unpermute_bwd(int dtype, const UnpermuteBwdArgs& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, pm_grid(a.T + a.E), dim3(kPmThreads), 0, st, a);
  };
  return dtype == kDtypeBF16 ? run(unpermute_bwd_kernel<__nv_bfloat16>) : run(unpermute_bwd_kernel<float>);
}

}  // namespace mm
