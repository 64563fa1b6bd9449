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
// Bound by memory: 2 + 0.53 bytes a value in bf16.  16 lanes take a word of
// four groups (128 columns), 8 columns a lane: 16-byte loads and 4-byte
// stores without gaps, the group's maximum in two exchanges.
#include "pack.cuh"
#include "mm_kernels.cuh"

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
    const int q2 = static_cast<int>(top >> 23);
    uint32_t byte = q2 == 255 ? 255u : static_cast<uint32_t>(max(q2 - 2 + ((top & 0x7fffffu) > 0x400000u), 1));
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
                      const int32_t* n_rows, const int64_t R, const int C) {
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
    if (at.row < rows && group < groups) {
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

template <typename T, int V>
static cudaError_t mx4_launch(bool quantise, const Mx4Args& a, cudaStream_t st) {
  const int64_t units = a.R * ((a.C + 127) / 128);
  constexpr int kPer = kMxThreads / kMxLanes * kMxUnits;
  const int64_t blocks = (units + kPer - 1) / kPer;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (quantise)
    return launch_dependent_kernel(mx4_quantize_kernel<T, V>, grid, dim3(kMxThreads), 0, st,
                                   static_cast<const T*>(a.x), a.codes, a.exps, a.n_rows, a.R, a.C);
  return launch_dependent_kernel(mx4_dequantize_kernel<T, V>, grid, dim3(kMxThreads), 0, st,
                                 static_cast<const uint8_t*>(a.codes), static_cast<const uint8_t*>(a.exps),
                                 static_cast<T*>(a.x_out), a.n_rows, a.R, a.C);
}

// Accesses as wide as every row's alignment allows.
cudaError_t launch_mx4(int dtype, bool quantise, const Mx4Args& a, cudaStream_t st) {
  if (dtype == kDtypeBF16) {
    if (a.C % 8 == 0) return mx4_launch<__nv_bfloat16, 8>(quantise, a, st);
    if (a.C % 4 == 0) return mx4_launch<__nv_bfloat16, 4>(quantise, a, st);
    if (a.C % 2 == 0) return mx4_launch<__nv_bfloat16, 2>(quantise, a, st);
    return mx4_launch<__nv_bfloat16, 1>(quantise, a, st);
  }
  if (a.C % 4 == 0) return mx4_launch<float, 4>(quantise, a, st);
  if (a.C % 2 == 0) return mx4_launch<float, 2>(quantise, a, st);
  return mx4_launch<float, 1>(quantise, a, st);
}

}  // namespace mm
