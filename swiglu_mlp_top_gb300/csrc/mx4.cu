// Microscaled 4-bit floating point: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives) that share a power of two per 32 columns.
//
//   e     the least integer >= -126 with amax <= 6 * 2^e over the group
//   code  x * 2^-e rounded to the nearest e2m1, ties to the even code
//
// With amax = 1.f * 2^q, amax <= 1.5 * 2^(e+2) gives e = q - 2, or q - 1 where
// 1.f > 1.5: the exponent byte follows from amax's bits, and scaling by a
// power of two is exact, so the codes do not depend on the order of anything.
// The maximum is taken over magnitudes as integers, in which an infinity or a
// NaN is above every number: it gives the byte 255 and a group of NaN.
//
// per_group: the rows are matrices of so many rows, one a group, and those of
// groups without rows are left out.
//
// Bound by memory (2 + 0.53 bytes a value in bf16) where few enough
// instructions go into a value.  Rows of whole 32-byte pieces: a lane takes 16
// columns in 32-byte loads, magnitudes and products stay packed in bf16 (a
// product that bf16 cannot hold is below 2^-126 and becomes zero either way),
// 6 instructions a value.  Other rows: 8 columns a lane, as wide as the rows'
// alignment allows; narrow rows are written element by element, neighbouring
// lanes next to each other.
#include "grouped.cuh"
#include "mx4.cuh"
#include "pack.cuh"

namespace mm {

constexpr int kMxThreads = 256;
constexpr int kMxLanes = 16;                 // lanes of a word of 128 columns
constexpr int kMxUnits = 4;                  // words a lane takes, one after the other

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The eight values of a word of codes, as fp32.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f16x2_to_f32x2(h[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

struct MxUnit {
  int64_t row;
  int word;
};
// Unit u (row by row) and the ones after it.
__device__ __forceinline__ MxUnit mx_unit(int64_t u, int words) {
  if (u < 0xffffffffll) {
    const uint32_t r = static_cast<uint32_t>(u) / static_cast<uint32_t>(words);
    return MxUnit{r, static_cast<int>(static_cast<uint32_t>(u) - r * words)};
  }
  return MxUnit{u / words, static_cast<int>(u % words)};
}

// Eight columns of a row from column c on; those from C on count as 0.
template <typename T, int V>
__device__ __forceinline__ void mx_load(const T* row, int c, int C, typename Pack<T, V>::Raw (&raw)[8 / V]) {
#pragma unroll
  for (int j = 0; j < 8 / V; ++j) {            // C is a multiple of V: a vector is inside or outside
    if (c + j * V < C) {
      raw[j] = *reinterpret_cast<const typename Pack<T, V>::Raw*>(row + c + j * V);
    } else {
      float z[V] = {};
      raw[j] = Pack<T, V>::put(z);
    }
  }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 32 bytes in one access, from a 32-byte boundary.
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
// The scale byte of a group whose largest magnitude has these fp32 bits.
__device__ __forceinline__ uint32_t mx4_byte(uint32_t top) {
  const int q = static_cast<int>(top >> 23);
  return q == 255 ? 255u : static_cast<uint32_t>(max(q - 2 + ((top & 0x7fffffu) > 0x400000u), 1));
}

constexpr int kMxWideLanes = 8;              // lanes of a word, 16 columns each

// Rows of C columns that are whole pieces of 16 (32 bytes aligned).
template <typename T>
__global__ void __launch_bounds__(kMxThreads)
mx4_quantize_wide_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                         const int32_t* n_rows, const int64_t R, const int C) {
  constexpr bool kBf = sizeof(T) == 2;
  constexpr int kUnits = kBf ? 4 : 2, kLoads = kBf ? 1 : 2;
  pdl_enter();
  const int groups = (C + 31) / 32, words = (groups + 3) / 4;
  const int64_t rows = n_rows ? min(static_cast<int64_t>(max(*n_rows, 0)), R) : R;
  const int l = threadIdx.x % kMxWideLanes;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kMxThreads / kMxWideLanes) + threadIdx.x / kMxWideLanes) * kUnits;
  MxUnit at = mx_unit(first, words);
  MxUnit units[kUnits];
  uint32_t raw[kUnits][8 * kLoads];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    units[q] = at;
    const int c = at.word * 128 + 16 * l;
    if (at.row < rows && c < C) {
      const T* from = x + at.row * C + c;
#pragma unroll
      for (int h = 0; h < kLoads; ++h) load32(from + 8 * h, *reinterpret_cast<uint32_t(*)[8]>(&raw[q][8 * h]));
    } else {
#pragma unroll
      for (int h = 0; h < 8 * kLoads; ++h) raw[q][h] = 0u;
    }
    if (++at.word == words) {
      at.word = 0;
      ++at.row;
    }
  }
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    if (units[q].row >= rows) break;           // the 8 lanes of a unit agree
    uint32_t top;
    if constexpr (kBf) {
      uint32_t m = raw[q][0] & 0x7fff7fffu;
#pragma unroll
      for (int h = 1; h < 8; ++h) m = max_u16x2(m, raw[q][h] & 0x7fff7fffu);
      top = max(m & 0xffff0000u, m << 16);
    } else {
      top = raw[q][0] & 0x7fffffffu;
#pragma unroll
      for (int h = 1; h < 16; ++h) top = max(top, raw[q][h] & 0x7fffffffu);
    }
    top = max(top, __shfl_xor_sync(mask, top, 1));
    uint32_t byte = mx4_byte(top);
    const uint32_t scale = (254u - min(byte, 253u)) << 23;       // 2^-e
    float v[16];
    if constexpr (kBf) {
      const uint32_t s2 = (scale >> 16) | scale;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const uint32_t w = bf16x2_mul(raw[q][h], s2);
        v[2 * h] = __uint_as_float(w << 16);
        v[2 * h + 1] = __uint_as_float(w & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 16; ++h) v[h] = __uint_as_float(raw[q][h]) * __uint_as_float(scale);
    }
    const int group = units[q].word * 4 + l / 2;
    if (group < groups) {
      // a lane behind the last column of its group has zeros there
      uint2 c = make_uint2(e2m1x8(*reinterpret_cast<const float(*)[8]>(v)), e2m1x8(*reinterpret_cast<const float(*)[8]>(v + 8)));
      if (byte == 255u) c = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(codes + units[q].row * (16 * static_cast<int64_t>(groups)) + group * 16 + (l & 1) * 8) = c;
    } else {
      byte = 127;
    }
    byte <<= 8 * (l / 2);
    byte |= __shfl_xor_sync(mask, byte, 2);
    byte |= __shfl_xor_sync(mask, byte, 4);
    if (l == 0) reinterpret_cast<uint32_t*>(exps)[units[q].word * R + units[q].row] = byte;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kMxThreads)
mx4_quantize_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                    const int32_t* n_rows, const int64_t R, const int C) {
  pdl_enter();
  const int groups = (C + 31) / 32, words = (groups + 3) / 4;
  const int64_t rows = n_rows ? min(static_cast<int64_t>(max(*n_rows, 0)), R) : R;
  const int l = threadIdx.x % kMxLanes;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kMxThreads / kMxLanes) + threadIdx.x / kMxLanes) * kMxUnits;
  MxUnit at = mx_unit(first, words);
  MxUnit units[kMxUnits];
  typename Pack<T, V>::Raw raw[kMxUnits][8 / V];
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    units[q] = at;
    if (at.row < rows) mx_load<T, V>(x + at.row * C, at.word * 128 + 8 * l, C, raw[q]);
    if (++at.word == words) {
      at.word = 0;
      ++at.row;
    }
  }
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    if (units[q].row >= rows) break;           // the 16 lanes of a unit agree
    const uint32_t mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = Pack<T, V>::get(raw[q][j / V], j % V);
      top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    top = max(top, __shfl_xor_sync(mask, top, 1));
    top = max(top, __shfl_xor_sync(mask, top, 2));
    uint32_t byte = mx4_byte(top);
    const float scale = __uint_as_float((254u - min(byte, 253u)) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    const int group = units[q].word * 4 + l / 4;
    if (group < groups)
      *reinterpret_cast<uint32_t*>(codes + units[q].row * (16 * static_cast<int64_t>(groups)) + group * 16 + (l & 3) * 4) =
          byte == 255u ? 0u : e2m1x8(v);
    else
      byte = 127;
    byte <<= 8 * (l / 4);
    byte |= __shfl_xor_sync(mask, byte, 4);
    byte |= __shfl_xor_sync(mask, byte, 8);
    if (l == 0) reinterpret_cast<uint32_t*>(exps)[units[q].word * R + units[q].row] = byte;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kMxThreads)
mx4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, T* __restrict__ x,
                      const GroupTables g, const int per_group, const int32_t* n_rows, const int64_t R, const int C) {
  pdl_enter();
  const int groups = (C + 31) / 32, words = (groups + 3) / 4;
  const int64_t rows = n_rows ? min(static_cast<int64_t>(max(*n_rows, 0)), R) : R;
  const int l = threadIdx.x % kMxLanes;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kMxThreads / kMxLanes) + threadIdx.x / kMxLanes) * kMxUnits;
  MxUnit at = mx_unit(first, words);
  MxUnit units[kMxUnits];
  uint32_t code[kMxUnits], word[kMxUnits];
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    units[q] = at;
    const int group = at.word * 4 + l / 4;
    if (per_group && at.row < rows && group_span(g, static_cast<int>(at.row / per_group)).n == 0) units[q].row = R;
    if (units[q].row < rows && group < groups) {
      code[q] = *reinterpret_cast<const uint32_t*>(codes + at.row * (16 * static_cast<int64_t>(groups)) + group * 16 + (l & 3) * 4);
      word[q] = reinterpret_cast<const uint32_t*>(exps)[at.word * R + at.row];
    }
    if (++at.word == words) {
      at.word = 0;
      ++at.row;
    }
  }
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    if (units[q].row >= rows || units[q].word * 4 + l / 4 >= groups) continue;
    const uint32_t byte = (word[q] >> (8 * (l / 4))) & 255u;
    // 2^(byte - 127): subnormal for byte 0, NaN for 255
    const float scale = byte == 255u ? __uint_as_float(0x7fffffffu)
                                     : __uint_as_float(byte ? byte << 23 : 0x400000u);
    float v[8];
    e2m1x8_values(code[q], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    T* row = x + units[q].row * C;
    const int c = units[q].word * 128 + 8 * l;
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
      float part[V];
#pragma unroll
      for (int i = 0; i < V; ++i) part[i] = v[j * V + i];
      if (c + j * V < C) *reinterpret_cast<typename Pack<T, V>::Raw*>(row + c + j * V) = Pack<T, V>::put(part);
    }
  }
}

// bf16 rows of whole 32-byte pieces: 16 columns a lane.
__global__ void __launch_bounds__(kMxThreads)
mx4_dequantize_wide_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, __nv_bfloat16* __restrict__ x,
                           const GroupTables g, const int per_group, const int32_t* n_rows, const int64_t R, const int C) {
  pdl_enter();
  const int groups = (C + 31) / 32, words = (groups + 3) / 4;
  const int64_t rows = n_rows ? min(static_cast<int64_t>(max(*n_rows, 0)), R) : R;
  const int l = threadIdx.x % kMxWideLanes;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kMxThreads / kMxWideLanes) + threadIdx.x / kMxWideLanes) * kMxUnits;
  MxUnit at = mx_unit(first, words);
  int64_t to[kMxUnits];                        // first element, -1: nothing to write
  uint2 code[kMxUnits];
  uint32_t word[kMxUnits];
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    const int c = at.word * 128 + 16 * l;
    to[q] = at.row < rows && c < C ? at.row * C + c : -1;
    if (per_group && to[q] >= 0 && group_span(g, static_cast<int>(at.row / per_group)).n == 0) to[q] = -1;
    if (to[q] >= 0) {
      code[q] = *reinterpret_cast<const uint2*>(codes + at.row * (16 * static_cast<int64_t>(groups)) + at.word * 64 + 8 * l);
      word[q] = reinterpret_cast<const uint32_t*>(exps)[at.word * R + at.row];
    }
    if (++at.word == words) {
      at.word = 0;
      ++at.row;
    }
  }
#pragma unroll
  for (int q = 0; q < kMxUnits; ++q) {
    if (to[q] < 0) continue;
    const uint32_t byte = (word[q] >> (8 * (l / 2))) & 255u;
    uint32_t f1, f2;
    mx4_factors(byte, f1, f2);
    const bool two = byte > 128u;
    const uint4 a = two ? e2m1_bf16<true>(code[q].x, f1, f2) : e2m1_bf16<false>(code[q].x, f1, 0u);
    const uint4 b = two ? e2m1_bf16<true>(code[q].y, f1, f2) : e2m1_bf16<false>(code[q].y, f1, 0u);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(x + to[q]), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  }
}

// Rows that start anywhere: neighbouring lanes write neighbouring elements.
template <typename T>
__global__ void __launch_bounds__(kMxThreads)
mx4_dequantize_narrow_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, T* __restrict__ x,
                             const GroupTables g, const int per_group, const int32_t* n_rows, const int64_t R, const int C) {
  pdl_enter();
  const int groups = (C + 31) / 32, words = (groups + 3) / 4;
  const int64_t rows = n_rows ? min(static_cast<int64_t>(max(*n_rows, 0)), R) : R;
  const int lane = threadIdx.x & 31;
  const MxUnit u = mx_unit(static_cast<int64_t>(blockIdx.x) * (kMxThreads / 32) + (threadIdx.x >> 5), words);
  if (u.row >= rows) return;                   // a warp's word of 128 columns
  if (per_group && group_span(g, static_cast<int>(u.row / per_group)).n == 0) return;
  const uint32_t word = reinterpret_cast<const uint32_t*>(exps)[u.word * R + u.row];
  const uint8_t* from = codes + u.row * (16 * static_cast<int64_t>(groups));
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int c = u.word * 128 + 32 * g + lane;
    if (c >= C) break;
    const uint32_t code = (from[c >> 1] >> (4 * (c & 1))) & 15u;
    const uint32_t byte = (word >> (8 * g)) & 255u;
    // 2^(byte - 127): subnormal for byte 0, NaN for 255
    const float scale = byte == 255u ? __uint_as_float(0x7fffffffu)
                                     : __uint_as_float(byte ? byte << 23 : 0x400000u);
    // sign at bit 31, exponent and fraction at 24..22: the value times 2^-126
    const float v = __uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f;
    x[u.row * C + c] = static_cast<T>(v * scale);
  }
}

// A grid of `per` words of 128 columns a block.
template <typename Kern, typename... Args>
static cudaError_t mx4_launch(Kern fn, int per, const Mx4Args& a, cudaStream_t st, Args... args) {
  const int64_t blocks = (a.R * ((a.C + 127) / 128) + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent_kernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kMxThreads), 0, st, args..., a.n_rows, a.R, a.C);
}

template <typename T>
static cudaError_t mx4_quantize(const Mx4Args& a, cudaStream_t st) {
  const T* x = static_cast<const T*>(a.x);
  constexpr int kPer = kMxThreads / kMxLanes * kMxUnits;
  if (a.C % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 32 == 0)
    return mx4_launch(mx4_quantize_wide_kernel<T>, kMxThreads / kMxWideLanes * (sizeof(T) == 2 ? 4 : 2), a, st, x, a.codes, a.exps);
  if constexpr (sizeof(T) == 2)
    if (a.C % 8 == 0) return mx4_launch(mx4_quantize_kernel<T, 8>, kPer, a, st, x, a.codes, a.exps);
  if (a.C % 4 == 0) return mx4_launch(mx4_quantize_kernel<T, 4>, kPer, a, st, x, a.codes, a.exps);
  if (a.C % 2 == 0) return mx4_launch(mx4_quantize_kernel<T, 2>, kPer, a, st, x, a.codes, a.exps);
  return mx4_launch(mx4_quantize_kernel<T, 1>, kPer, a, st, x, a.codes, a.exps);
}

template <typename T>
static cudaError_t mx4_dequantize(const Mx4Args& a, cudaStream_t st) {
  const uint8_t *codes = a.codes, *exps = a.exps;
  T* x = static_cast<T*>(a.x_out);
  constexpr int kWide = 16 / sizeof(T), kPer = kMxThreads / kMxLanes * kMxUnits;
  if constexpr (sizeof(T) == 2)
    if (a.C % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 32 == 0)
      return mx4_launch(mx4_dequantize_wide_kernel, kMxThreads / kMxWideLanes * kMxUnits, a, st, codes, exps, x, a.g, a.per_group);
  if (a.C % kWide == 0) return mx4_launch(mx4_dequantize_kernel<T, kWide>, kPer, a, st, codes, exps, x, a.g, a.per_group);
  if constexpr (sizeof(T) == 2)
    if (a.C % 4 == 0) return mx4_launch(mx4_dequantize_kernel<T, 4>, kPer, a, st, codes, exps, x, a.g, a.per_group);
  return mx4_launch(mx4_dequantize_narrow_kernel<T>, kMxThreads / 32, a, st, codes, exps, x, a.g, a.per_group);
}

cudaError_t launch_mx4(int dtype, bool quantise, const Mx4Args& a, cudaStream_t st) {
  if (dtype == kDtypeBF16) return quantise ? mx4_quantize<__nv_bfloat16>(a, st) : mx4_dequantize<__nv_bfloat16>(a, st);
  return quantise ? mx4_quantize<float>(a, st) : mx4_dequantize<float>(a, st);
}

}  // namespace mm
