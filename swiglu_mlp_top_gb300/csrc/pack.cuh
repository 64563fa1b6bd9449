// Row elements moved in one access of V of them, and as fp32 values.
#pragma once

#include "mm_device.cuh"

namespace mm {

// V consecutive elements as loaded (one access), and as fp32.
template <typename T, int V> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> {
  typedef uint4 Raw;
  static __device__ __forceinline__ float get(const Raw& r, int j) {
    const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
    return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ Raw put(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Pack<__nv_bfloat16, 4> {
  typedef uint2 Raw;
  static __device__ __forceinline__ float get(const Raw& r, int j) {
    const uint32_t w = j < 2 ? r.x : r.y;
    return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ Raw put(const float (&v)[4]) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
template <> struct Pack<__nv_bfloat16, 2> {
  typedef uint32_t Raw;
  static __device__ __forceinline__ float get(const Raw& r, int j) {
    return __uint_as_float(j ? (r & 0xffff0000u) : (r << 16));
  }
  static __device__ __forceinline__ Raw put(const float (&v)[2]) { return pack_bf16x2(v[0], v[1]); }
};
template <> struct Pack<__nv_bfloat16, 1> {
  typedef __nv_bfloat16 Raw;
  static __device__ __forceinline__ float get(const Raw& r, int) { return __bfloat162float(r); }
  static __device__ __forceinline__ Raw put(const float (&v)[1]) { return __float2bfloat16_rn(v[0]); }
};
template <> struct Pack<float, 4> {
  typedef float4 Raw;
  static __device__ __forceinline__ float get(const Raw& r, int j) {
    return j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
  }
  static __device__ __forceinline__ Raw put(const float (&v)[4]) {
    return make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Pack<float, 2> {
  typedef float2 Raw;
  static __device__ __forceinline__ float get(const Raw& r, int j) { return j ? r.y : r.x; }
  static __device__ __forceinline__ Raw put(const float (&v)[2]) { return make_float2(v[0], v[1]); }
};
template <> struct Pack<float, 1> {
  typedef float Raw;
  static __device__ __forceinline__ float get(const Raw& r, int) { return r; }
  static __device__ __forceinline__ Raw put(const float (&v)[1]) { return v[0]; }
};

// Vector c of a row that starts at element `base` of p.
template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::Raw row_load(const void* p, int64_t base, int c) {
  return reinterpret_cast<const typename Pack<T, V>::Raw*>(static_cast<const T*>(p) + base)[c];
}
template <typename T, int V>
__device__ __forceinline__ void row_store(void* p, int64_t base, int c, const float (&v)[V]) {
  reinterpret_cast<typename Pack<T, V>::Raw*>(static_cast<T*>(p) + base)[c] = Pack<T, V>::put(v);
}

}  // namespace mm
