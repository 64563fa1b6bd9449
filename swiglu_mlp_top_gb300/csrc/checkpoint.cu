// Activations kept in 8 bits, and the SwiGLU activation that writes and
// reads them (include/mm.h, mm_checkpoint_pack).  A group of 32 columns
// shares a power of two: e is the least integer >= -126 with amax <= 448 2^e
// over the group's finite values, code = e4m3(x 2^-e), round to nearest even.
// The scaling is exact, so the codes do not depend on how they are computed.
// One lane per column, one warp per group.
#include "mm_kernels.cuh"

namespace mm {

constexpr int kCkThreads = 256;
constexpr int kCkWarps = kCkThreads / 32;

__device__ __forceinline__ float ck_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ck_load(const float* p) { return *p; }
__device__ __forceinline__ void ck_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void ck_store(float* p, float v) { *p = v; }

// |v| of a finite value, 0 for an infinity or a NaN.
__device__ __forceinline__ float ck_finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.f;
}
// Biased exponent e + 127 of a group with the given finite amax: amax = 1.m 2^p
// and 448 = 1.75 * 2^8.
__device__ __forceinline__ int ck_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (e < -126 ? -126 : e) + 127;
}
__device__ __forceinline__ float ck_scale(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }
__device__ __forceinline__ float ck_inv_scale(int biased) {
  return __uint_as_float(static_cast<uint32_t>(254 - biased) << 23);
}
// Two values to e4m3 (lo in the low byte); an infinity becomes a NaN.
__device__ __forceinline__ uint16_t ck_encode2(float lo, float hi) {
  uint16_t r;
  const float nan = __uint_as_float(0x7fffffffu);
  lo = fabsf(lo) <= 3.402823466e38f ? lo : nan;
  hi = fabsf(hi) <= 3.402823466e38f ? hi : nan;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 ck_decode2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return f16x2_to_f32x2(h);
}

// One group: lane's value to its code; returns the group's biased exponent.
__device__ __forceinline__ int ck_group(float v, uint8_t& code) {
  float amax = ck_finite_abs(v);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = ck_exponent(amax);
  code = static_cast<uint8_t>(ck_encode2(v * ck_inv_scale(e), 0.f) & 0xff);
  return e;
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) checkpoint_pack_kernel(const CheckpointArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t G = (a.C + 31) / 32, n = a.R * G;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kCkWarps) + (threadIdx.x >> 5); i < n;
       i += static_cast<int64_t>(gridDim.x) * kCkWarps) {
    const int64_t row = i / G, c = (i % G) * 32 + lane;
    const float v = c < a.C ? ck_load(static_cast<const T*>(a.x) + row * a.C + c) : 0.f;
    uint8_t code;
    const int e = ck_group(v, code);
    if (c < a.C) a.codes[row * a.C + c] = code;
    if (lane == 0) a.exps[i] = static_cast<uint8_t>(e);
  }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) checkpoint_unpack_kernel(const CheckpointArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t G = (a.C + 31) / 32, n = a.R * G;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kCkWarps) + (threadIdx.x >> 5); i < n;
       i += static_cast<int64_t>(gridDim.x) * kCkWarps) {
    const int64_t row = i / G, c = (i % G) * 32 + lane;
    if (c < a.C)
      ck_store(static_cast<T*>(a.x_out) + row * a.C + c,
               ck_decode2(a.codes[row * a.C + c]).x * ck_scale(a.exps[i]));
  }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_kernel(const SwigluActArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  int64_t R = a.R;
  if (a.n_rows && *a.n_rows < R) R = *a.n_rows;
  const int64_t I = a.I, G = (I + 31) / 32, n = R * G;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kCkWarps) + (threadIdx.x >> 5); i < n;
       i += static_cast<int64_t>(gridDim.x) * kCkWarps) {
    const int64_t row = i / G, q = i % G, c = q * 32 + lane;
    const bool in = c < I;
    const float g = in ? ck_load(static_cast<const T*>(a.gu) + row * 2 * I + c) : 0.f;
    const float u = in ? ck_load(static_cast<const T*>(a.gu) + row * 2 * I + I + c) : 0.f;
    if (in) ck_store(static_cast<T*>(a.h) + row * I + c, silu_f32(g) * u);
    if (a.codes == nullptr) continue;
    uint8_t cg, cu;
    const int eg = ck_group(g, cg), eu = ck_group(u, cu);
    if (in) {
      a.codes[row * 2 * I + c] = cg;
      a.codes[row * 2 * I + I + c] = cu;
    }
    if (lane == 0) {
      a.exps[row * 2 * G + q] = static_cast<uint8_t>(eg);
      a.exps[row * 2 * G + G + q] = static_cast<uint8_t>(eu);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_bwd_kernel(const SwigluActArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  int64_t R = a.R;
  if (a.n_rows && *a.n_rows < R) R = *a.n_rows;
  const int64_t I = a.I, G = (I + 31) / 32, n = R * G;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kCkWarps) + (threadIdx.x >> 5); i < n;
       i += static_cast<int64_t>(gridDim.x) * kCkWarps) {
    const int64_t row = i / G, q = i % G, c = q * 32 + lane;
    if (c >= I) continue;
    const float g = ck_decode2(a.codes[row * 2 * I + c]).x * ck_scale(a.exps[row * 2 * G + q]);
    const float u = ck_decode2(a.codes[row * 2 * I + I + c]).x * ck_scale(a.exps[row * 2 * G + G + q]);
    const float dh = ck_load(static_cast<const T*>(a.dh) + row * I + c);
    const float sig = 1.0f / (1.0f + expf(-g));
    const float silu = g * sig;
    ck_store(static_cast<T*>(a.dgu) + row * 2 * I + c, dh * u * (sig * (1.0f + g * (1.0f - sig))));
    ck_store(static_cast<T*>(a.dgu) + row * 2 * I + I + c, dh * silu);
    if (a.h) ck_store(static_cast<T*>(a.h) + row * I + c, silu * u);
  }
}

static dim3 ck_grid(int64_t groups) {
  const int64_t most = static_cast<int64_t>(num_sms()) * 8, want = (groups + kCkWarps - 1) / kCkWarps;
  return dim3(static_cast<unsigned>(want < most ? (want > 0 ? want : 1) : most));
}

cudaError_t launch_checkpoint(int dtype, bool pack, const CheckpointArgs& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, ck_grid(a.R * ((a.C + 31) / 32)), dim3(kCkThreads), 0, st, a);
  };
  if (dtype == kDtypeBF16)
    return pack ? run(checkpoint_pack_kernel<__nv_bfloat16>) : run(checkpoint_unpack_kernel<__nv_bfloat16>);
  return pack ? run(checkpoint_pack_kernel<float>) : run(checkpoint_unpack_kernel<float>);
}

cudaError_t launch_swiglu_act(int dtype, bool backward, const SwigluActArgs& a, cudaStream_t st) {
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, ck_grid(a.R * ((a.I + 31) / 32)), dim3(kCkThreads), 0, st, a);
  };
  if (dtype == kDtypeBF16)
    return backward ? run(swiglu_act_bwd_kernel<__nv_bfloat16>) : run(swiglu_act_kernel<__nv_bfloat16>);
  return backward ? run(swiglu_act_bwd_kernel<float>) : run(swiglu_act_kernel<float>);
}

}  // namespace mm
