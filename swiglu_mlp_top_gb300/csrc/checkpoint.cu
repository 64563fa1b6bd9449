// Activations kept in 8 bits, and the SwiGLU activation that writes and
// reads them (include/mm.h, mm_checkpoint_pack).  A group of 32 columns
// shares a power of two: e is the least integer >= -126 with amax <= 448 2^e
// over the group's finite values, code = e4m3(x 2^-e), round to nearest even.
// The scaling is exact, so the codes do not depend on how they are computed.
//
// All kernels stream: each input is read and each output written once.  A
// thread owns V consecutive columns (V / 32 of a group), always the same ones
// of a row, and walks down the rows; V is the widest of 16, 8 and 4 that
// divides the width (within what ck_vec allows the type), so that values and
// codes move in whole aligned accesses.
// Rows of other widths go in strips of 128 columns, a warp each: a lane has
// one column of each of the strip's four groups, and single accesses.
#include "mm_kernels.cuh"

namespace mm {

constexpr int kCkThreads = 512;         // most threads of a block

// V elements of T (4, 8 or 16) as 32-bit words.
template <typename T, int V>
struct Words {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  static constexpr int kN = kBytes / 4;
  uint32_t w[kN];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = static_cast<const uint4*>(p)[i];
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = *static_cast<const uint2*>(p);
      w[0] = q.x; w[1] = q.y;
    } else {
      w[0] = *static_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
      *static_cast<uint32_t*>(p) = w[0];
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    return __uint_as_float((j & 1) ? (w[j / 2] & 0xffff0000u) : (w[j / 2] << 16));
  }
  __device__ __forceinline__ void put(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = __float_as_uint(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) w[j / 2] = pack_bf16x2(v[j], v[j + 1]);
    }
  }
  // Elements 2k and 2k + 1.
  __device__ __forceinline__ u64 get2(int k) const { return pair2(get(2 * k), get(2 * k + 1)); }
  __device__ __forceinline__ void put2(int k, u64 v) {
    if constexpr (sizeof(T) == 2) {
      w[k] = pack_bf16x2(lo2(v), hi2(v));
    } else {
      w[2 * k] = __float_as_uint(lo2(v));
      w[2 * k + 1] = __float_as_uint(hi2(v));
    }
  }
  // The largest |value| as the bits of an fp32; infinities and NaN order above.
  __device__ __forceinline__ uint32_t abs_max_bits() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i] & 0x7fff7fffu));
      return max(m << 16, m & 0xffff0000u);
    }
  }
};
typedef uint8_t Code;

__device__ __forceinline__ float ck_scale(uint32_t biased) { return __uint_as_float(biased << 23); }

// Biased exponent e + 127 of a group with the given finite amax (fp32 bits):
// amax = 1.m 2^p and 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t ck_exponent(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1u : static_cast<uint32_t>(e);
}

template <int V>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
  for (int o = 1; o < 32 / V; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Codes of the thread's V values and its group's biased exponent.  The whole
// warp calls.  An infinity or a NaN gets a NaN code and no say in the scale.
template <typename T, int V>
__device__ __forceinline__ uint32_t ck_encode(Words<T, V> x, Words<Code, V>& codes) {
  uint32_t amax = group_max<V>(x.abs_max_bits());
  if (__any_sync(0xffffffffu, amax >= 0x7f800000u)) {
    uint32_t m = 0;
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t b = __float_as_uint(x.get(j)) & 0x7fffffffu;
      m = max(m, b < 0x7f800000u ? b : 0u);
      v[j] = b < 0x7f800000u ? x.get(j) : __uint_as_float(0x7fffffffu);
    }
    amax = group_max<V>(m);
    x.put(v);
  }
  const uint32_t e = ck_exponent(amax);
  const float inv = ck_scale(254u - e);
  uint16_t c[V / 2];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const u64 v = fmul2(x.get2(k), pair2(inv, inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[k]) : "f"(hi2(v)), "f"(lo2(v)));
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) codes.w[i] = c[2 * i] | (static_cast<uint32_t>(c[2 * i + 1]) << 16);
  return e;
}

// Values of codes 2k and 2k + 1.
template <int V>
__device__ __forceinline__ u64 ck_decode2(const Words<Code, V>& codes, int k, float scale) {
  const uint16_t c = static_cast<uint16_t>(codes.w[k / 2] >> (16 * (k % 2)));
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  const float2 f = f16x2_to_f32x2(h);
  return fmul2(pair2(f.x, f.y), pair2(scale, scale));
}

// sigma(g) and 1 - sigma(g) of two values: with t = exp(-|g|), 1 / (1 + t) and
// t / (1 + t), without cancellation for either sign.  fp32 rows take expf and
// a division.  For bf16 rows these are what a streaming kernel has no issue
// slots for (79% of them were taken, at 41 instructions an element), so
//   t = (2^q)^2,  q = -|g| log2(e) / 2
// with the product in two parts (Cody and Waite: head q, tail r, 2^(q + r) =
// 2^q (1 + r ln 2)) and the hardware's 2^x: half the argument keeps 2^q above
// fp32's smallest normal wherever t is above its smallest subnormal.  Relative
// error of t below 2^-20.5 (twice the instruction's 2 ulp, and four roundings).
template <typename T>
__device__ __forceinline__ void sigmoid2(u64 g, u64& sig, u64& rest) {
  const float g0 = lo2(g), g1 = hi2(g);
  u64 t, s;
  if constexpr (sizeof(T) == 4) {
    t = pair2(expf(-fabsf(g0)), expf(-fabsf(g1)));
    s = pair2(1.0f / (1.0f + lo2(t)), 1.0f / (1.0f + hi2(t)));
  } else {
    constexpr double kC = 0.72134752044448170368;               // log2(e) / 2
    constexpr float kHead = static_cast<float>(kC), kTail = static_cast<float>(kC - static_cast<double>(kHead));
    constexpr float kLn2 = 0.693147180559945f;
    // -|g|, but no infinity, whose tail would be a NaN (t is 0 from 104 on)
    const u64 a = pair2(fmaxf(-fabsf(g0), -256.0f), fmaxf(-fabsf(g1), -256.0f));
    const u64 q = fmul2(a, pair2(kHead, kHead));
    const u64 r = ffma2(a, pair2(kTail, kTail), ffma2(a, pair2(kHead, kHead), q ^ 0x8000000080000000ull));
    float e0, e1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(lo2(q)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(hi2(q)));
    const u64 e = pair2(e0, e1), root = ffma2(e, fmul2(r, pair2(kLn2, kLn2)), e);
    t = fmul2(root, root);
    const u64 d = ffma2(root, root, pair2(1.0f, 1.0f));
    float s0, s1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(lo2(d)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(hi2(d)));
    s = pair2(s0, s1);
  }
  const u64 ts = fmul2(t, s);
  const bool p0 = g0 >= 0.f, p1 = g1 >= 0.f;                    // a NaN g is left to the caller's product with g
  sig = pair2(p0 ? lo2(s) : lo2(ts), p1 ? hi2(s) : hi2(ts));
  rest = pair2(p0 ? lo2(ts) : lo2(s), p1 ? hi2(ts) : hi2(s));
}

// A block's threads cover `rpb` rows of `upr` units (of V columns, whole
// groups), or a part of one row at a time.
struct CkShape {
  int upr;                    // units of a row: 32 / V for each group
  int rpb;                    // rows of a block and step
};

// One step of a thread: V columns of a row.
struct CkUnit {
  int64_t row, c;             // row, first column
  int g;                      // its group's place in the row
  bool in;                    // the columns are inside the tensor
  bool lead;                  // the thread writes the group's exponent
};

// Runs load(unit) and body(unit, what load gave) over the thread's units; the
// whole block goes through the same number of steps.  The next unit's loads
// are issued before this one's body, so that a block's arithmetic runs under
// its loads (R = 32768, I = 2432, bf16: SwiGLU with checkpoint 124 us without).
template <int V, bool kStrip = false, typename L, typename F>
__device__ __forceinline__ void each_unit(const CkShape& s, int64_t R, int64_t cols, L&& load, F&& body) {
  const int lrow = s.rpb > 1 ? static_cast<int>(threadIdx.x) / s.upr : 0;
  const int u0 = static_cast<int>(threadIdx.x) - lrow * s.upr;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.rpb;
  int base = 0;               // first unit of the block's part of the row
  auto unit = [&](int64_t r, int part) {
    const int u = part + u0;
    CkUnit q;
    q.row = r + lrow;
    const bool own = lrow < s.rpb && u < s.upr && q.row < R;
    if constexpr (kStrip) {                   // the lane's column of the first group
      q.c = (u >> 5) * 128 + (u & 31);
      q.g = (u >> 5) * 4;
      q.in = own;
      q.lead = own && (u & 31) == 0;
    } else {
      q.c = static_cast<int64_t>(u) * V;
      q.g = u / (32 / V);
      q.in = own && q.c < cols;
      q.lead = own && u % (32 / V) == 0;
    }
    return q;
  };
  if (r0 >= R) return;
  CkUnit now = unit(r0, base);
  auto data = load(now);
  for (;;) {
    base += blockDim.x;
    if (base >= s.upr) {
      base = 0;
      r0 += static_cast<int64_t>(gridDim.x) * s.rpb;
    }
    if (r0 >= R) break;
    const CkUnit next = unit(r0, base);
    const auto ahead = load(next);
    body(now, data);
    now = next;
    data = ahead;
  }
  body(now, data);
}

template <typename T, int V>
__global__ void __launch_bounds__(kCkThreads) checkpoint_pack_kernel(const CheckpointArgs a, const CkShape s) {
  pdl_enter();
  const int64_t G = (a.C + 31) / 32;
  each_unit<V>(
      s, a.R, a.C,
      [&](const CkUnit& q) {
        Words<T, V> x;
        x.clear();
        if (q.in) x.load(static_cast<const T*>(a.x) + q.row * a.C + q.c);
        return x;
      },
      [&](const CkUnit& q, const Words<T, V>& x) {
        Words<Code, V> codes;
        const uint32_t e = ck_encode<T, V>(x, codes);
        if (q.in) codes.store(a.codes + q.row * a.C + q.c);
        if (q.lead) a.exps[q.row * G + q.g] = static_cast<uint8_t>(e);
      });
}

template <typename T, int V>
__global__ void __launch_bounds__(kCkThreads) checkpoint_unpack_kernel(const CheckpointArgs a, const CkShape s) {
  pdl_enter();
  const int64_t G = (a.C + 31) / 32;
  struct In {
    Words<Code, V> codes;
    uint32_t e;
  };
  each_unit<V>(
      s, a.R, a.C,
      [&](const CkUnit& q) {
        In in;
        if (q.in) {
          in.codes.load(a.codes + q.row * a.C + q.c);
          in.e = a.exps[q.row * G + q.g];
        }
        return in;
      },
      [&](const CkUnit& q, const In& in) {
        if (!q.in) return;
        Words<T, V> x;
#pragma unroll
        for (int k = 0; k < V / 2; ++k) x.put2(k, ck_decode2<V>(in.codes, k, ck_scale(in.e)));
        x.store(static_cast<T*>(a.x_out) + q.row * a.C + q.c);
      });
}

__device__ __forceinline__ int64_t act_rows(const SwigluActArgs& a) {
  return a.n_rows && *a.n_rows < a.R ? *a.n_rows : a.R;
}

template <typename T, int V>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_kernel(const SwigluActArgs a, const CkShape s) {
  pdl_enter();
  const int64_t I = a.I, G = (I + 31) / 32;
  struct In {
    Words<T, V> g, u;
  };
  each_unit<V>(
      s, act_rows(a), I,
      [&](const CkUnit& q) {
        In in;
        in.g.clear();
        in.u.clear();
        if (q.in) {
          const T* src = static_cast<const T*>(a.gu) + q.row * 2 * I + q.c;
          in.g.load(src);
          in.u.load(src + I);
        }
        return in;
      },
      [&](const CkUnit& q, const In& in) {
        if (q.in) {
          Words<T, V> out;
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            u64 sig, rest;
            sigmoid2<T>(in.g.get2(k), sig, rest);
            out.put2(k, fmul2(fmul2(in.g.get2(k), sig), in.u.get2(k)));
          }
          out.store(static_cast<T*>(a.h) + q.row * I + q.c);
        }
        if (a.codes == nullptr) return;
        Words<Code, V> cg, cu;
        const uint32_t eg = ck_encode<T, V>(in.g, cg), eu = ck_encode<T, V>(in.u, cu);
        if (q.in) {
          cg.store(a.codes + q.row * 2 * I + q.c);
          cu.store(a.codes + q.row * 2 * I + I + q.c);
        }
        if (q.lead) {
          a.exps[q.row * 2 * G + q.g] = static_cast<uint8_t>(eg);
          a.exps[q.row * 2 * G + G + q.g] = static_cast<uint8_t>(eu);
        }
      });
}

template <typename T, int V>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_bwd_kernel(const SwigluActArgs a, const CkShape s) {
  pdl_enter();
  const int64_t I = a.I, G = (I + 31) / 32;
  struct In {
    Words<Code, V> g, u;
    Words<T, V> dh;
    uint32_t eg, eu;
  };
  each_unit<V>(
      s, act_rows(a), I,
      [&](const CkUnit& q) {
        In in;
        if (q.in) {
          in.g.load(a.codes + q.row * 2 * I + q.c);
          in.u.load(a.codes + q.row * 2 * I + I + q.c);
          in.dh.load(static_cast<const T*>(a.dh) + q.row * I + q.c);
          in.eg = a.exps[q.row * 2 * G + q.g];
          in.eu = a.exps[q.row * 2 * G + G + q.g];
        }
        return in;
      },
      [&](const CkUnit& q, const In& in) {
        if (!q.in) return;
        Words<T, V> dg, du, h;
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const u64 g = ck_decode2<V>(in.g, k, ck_scale(in.eg)), u = ck_decode2<V>(in.u, k, ck_scale(in.eu));
          const u64 d = in.dh.get2(k);
          u64 sig, rest;
          sigmoid2<T>(g, sig, rest);
          const u64 silu = fmul2(g, sig);
          dg.put2(k, fmul2(fmul2(d, u), fmul2(sig, ffma2(g, rest, pair2(1.0f, 1.0f)))));
          du.put2(k, fmul2(d, silu));
          h.put2(k, fmul2(u, silu));
        }
        dg.store(static_cast<T*>(a.dgu) + q.row * 2 * I + q.c);
        du.store(static_cast<T*>(a.dgu) + q.row * 2 * I + I + q.c);
        if (a.h) h.store(static_cast<T*>(a.h) + q.row * I + q.c);
      });
}

// ------------------------------------------------- strips of any other width
// A lane's four columns of a strip, 32 apart.
struct Strip {
  float v[4];
  __device__ __forceinline__ u64 pair(int k) const { return pair2(v[2 * k], v[2 * k + 1]); }
  __device__ __forceinline__ void set(int k, u64 x) {
    v[2 * k] = lo2(x);
    v[2 * k + 1] = hi2(x);
  }
};
__device__ __forceinline__ float strip_get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float strip_get(const float* p) { return *p; }
__device__ __forceinline__ void strip_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void strip_put(float* p, float v) { *p = v; }

// Columns of a row that starts at p, `cols` wide; zeros behind it.
template <typename T>
__device__ __forceinline__ Strip strip_load(const T* p, const CkUnit& q, int64_t cols) {
  Strip x;
#pragma unroll
  for (int j = 0; j < 4; ++j) x.v[j] = q.in && q.c + 32 * j < cols ? strip_get(p + q.c + 32 * j) : 0.f;
  return x;
}
template <typename T>
__device__ __forceinline__ void strip_store(T* p, const CkUnit& q, int64_t cols, const Strip& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (q.in && q.c + 32 * j < cols) strip_put(p + q.c + 32 * j, x.v[j]);
}
// The strip's codes and exponents to a row of each.  The whole warp calls.
__device__ __forceinline__ void strip_encode(const Strip& x, const CkUnit& q, int64_t cols, uint8_t* codes,
                                             uint8_t* exps) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __float_as_uint(x.v[j]) & 0x7fffffffu;
    const bool fine = b < 0x7f800000u;
    const uint32_t e = ck_exponent(__reduce_max_sync(0xffffffffu, fine ? b : 0u));
    const float v = fine ? x.v[j] * ck_scale(254u - e) : __uint_as_float(0x7fffffffu);
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(v));
    if (q.in && q.c + 32 * j < cols) codes[q.c + 32 * j] = static_cast<uint8_t>(c & 0xffu);
    if (q.lead && q.c + 32 * j < cols) exps[q.g + j] = static_cast<uint8_t>(e);
  }
}
__device__ __forceinline__ Strip strip_decode(const uint8_t* codes, const uint8_t* exps, const CkUnit& q, int64_t cols) {
  Strip x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = q.in && q.c + 32 * j < cols;
    const uint16_t c = in ? codes[q.c + 32 * j] : 0;
    const float s = in ? ck_scale(exps[q.g + j]) : 0.f;
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    x.v[j] = f16x2_to_f32x2(h).x * s;
  }
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) checkpoint_pack_strip_kernel(const CheckpointArgs a, const CkShape s) {
  pdl_enter();
  const int64_t G = (a.C + 31) / 32;
  each_unit<32, true>(
      s, a.R, a.C, [&](const CkUnit& q) { return strip_load(static_cast<const T*>(a.x) + q.row * a.C, q, a.C); },
      [&](const CkUnit& q, const Strip& x) { strip_encode(x, q, a.C, a.codes + q.row * a.C, a.exps + q.row * G); });
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) checkpoint_unpack_strip_kernel(const CheckpointArgs a, const CkShape s) {
  pdl_enter();
  const int64_t G = (a.C + 31) / 32;
  each_unit<32, true>(
      s, a.R, a.C, [&](const CkUnit& q) { return strip_decode(a.codes + q.row * a.C, a.exps + q.row * G, q, a.C); },
      [&](const CkUnit& q, const Strip& x) { strip_store(static_cast<T*>(a.x_out) + q.row * a.C, q, a.C, x); });
}

struct StripGu {
  Strip g, u, dh;
};

template <typename T>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_strip_kernel(const SwigluActArgs a, const CkShape s) {
  pdl_enter();
  const int64_t I = a.I, G = (I + 31) / 32;
  each_unit<32, true>(
      s, act_rows(a), I,
      [&](const CkUnit& q) {
        const T* src = static_cast<const T*>(a.gu) + q.row * 2 * I;
        return StripGu{strip_load(src, q, I), strip_load(src + I, q, I), Strip{}};
      },
      [&](const CkUnit& q, const StripGu& in) {
        Strip h;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          u64 sig, rest;
          sigmoid2<T>(in.g.pair(k), sig, rest);
          h.set(k, fmul2(fmul2(in.g.pair(k), sig), in.u.pair(k)));
        }
        strip_store(static_cast<T*>(a.h) + q.row * I, q, I, h);
        if (a.codes == nullptr) return;
        strip_encode(in.g, q, I, a.codes + q.row * 2 * I, a.exps + q.row * 2 * G);
        strip_encode(in.u, q, I, a.codes + q.row * 2 * I + I, a.exps + q.row * 2 * G + G);
      });
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) swiglu_act_bwd_strip_kernel(const SwigluActArgs a, const CkShape s) {
  pdl_enter();
  const int64_t I = a.I, G = (I + 31) / 32;
  each_unit<32, true>(
      s, act_rows(a), I,
      [&](const CkUnit& q) {
        return StripGu{strip_decode(a.codes + q.row * 2 * I, a.exps + q.row * 2 * G, q, I),
                       strip_decode(a.codes + q.row * 2 * I + I, a.exps + q.row * 2 * G + G, q, I),
                       strip_load(static_cast<const T*>(a.dh) + q.row * I, q, I)};
      },
      [&](const CkUnit& q, const StripGu& in) {
        Strip dg, du, h;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          u64 sig, rest, one = pair2(1.0f, 1.0f);
          const u64 g = in.g.pair(k), u = in.u.pair(k), d = in.dh.pair(k);
          sigmoid2<T>(g, sig, rest);
          const u64 silu = fmul2(g, sig);
          dg.set(k, fmul2(fmul2(d, u), fmul2(sig, ffma2(g, rest, one))));
          du.set(k, fmul2(d, silu));
          h.set(k, fmul2(u, silu));
        }
        T* out = static_cast<T*>(a.dgu) + q.row * 2 * I;
        strip_store(out, q, I, dg);
        strip_store(out + I, q, I, du);
        if (a.h) strip_store(static_cast<T*>(a.h) + q.row * I, q, I, h);
      });
}

// ----------------------------------------------------------------- launches
// Blocks of about 256 threads (whole rows where a row has fewer units), each
// with about four steps, and at least one wave of them where there are so
// many: the SMs do not run at one pace, so an even share of all rows to one
// wave of blocks waits for the slowest (R = 32768, I = 2432, bf16: SwiGLU with
// checkpoint 115 us, with four steps 94 us), while blocks of one step have no
// next loads to run ahead (108 us).
template <typename A>
static cudaError_t ck_launch(void (*kern)(A, CkShape), const A& a, int64_t R, int64_t cols, int V, cudaStream_t st) {
  const int groups = static_cast<int>((cols + 31) / 32);
  const int upr = V == 1 ? (groups + 3) / 4 * 32 : groups * (32 / V);
  CkShape s{upr, upr >= 256 ? 1 : 256 / upr};
  const int64_t want = static_cast<int64_t>(s.rpb) * upr;
  const int threads = want >= kCkThreads ? kCkThreads : static_cast<int>((want + 31) / 32 * 32);
  const int64_t most = (R + s.rpb - 1) / s.rpb, parts = (upr + threads - 1) / threads;   // steps of a row
  const int64_t wave = static_cast<int64_t>(num_sms()) * resident_blocks(reinterpret_cast<const void*>(kern), threads);
  int64_t blocks = most * (s.rpb > 1 ? 1 : parts) / 4;
  blocks = blocks > wave ? blocks : wave;
  blocks = blocks < most ? blocks : most;
  if (blocks > 0x7fffffff) blocks = 0x7fffffff;
  return launch_dependent_kernel(kern, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, a, s);
}

// Columns a thread: the widest of 16, 8, 4 that divides the width, up to a
// bound by what the registers hold beside the next unit's loads.  fp32 rows
// take 8 (4 in the backward), us with 16 / 8 / 4: R = 4000, I = 8192 forward
// 79 / 69 / 81, backward 120 / 101 / 94.  1: strips.
static inline int ck_vec(int64_t cols, int most) {
  for (int v = most; v >= 4; v /= 2)
    if (cols % v == 0) return v;
  return 1;
}

typedef void (*CheckpointKernel)(CheckpointArgs, CkShape);
typedef void (*SwigluActKernel)(SwigluActArgs, CkShape);

template <typename T>
static cudaError_t checkpoint_pick(bool pack, const CheckpointArgs& a, cudaStream_t st) {
  constexpr int kMost = sizeof(T) == 2 ? 16 : 8;
  const int V = ck_vec(a.C, kMost);
  CheckpointKernel k;
  if (V == kMost) k = pack ? checkpoint_pack_kernel<T, kMost> : checkpoint_unpack_kernel<T, kMost>;
  else if (V == 8) k = pack ? checkpoint_pack_kernel<T, 8> : checkpoint_unpack_kernel<T, 8>;
  else if (V == 4) k = pack ? checkpoint_pack_kernel<T, 4> : checkpoint_unpack_kernel<T, 4>;
  else k = pack ? checkpoint_pack_strip_kernel<T> : checkpoint_unpack_strip_kernel<T>;
  return ck_launch<CheckpointArgs>(k, a, a.R, a.C, V, st);
}

cudaError_t launch_checkpoint(int dtype, bool pack, const CheckpointArgs& a, cudaStream_t st) {
  return dtype == kDtypeBF16 ? checkpoint_pick<__nv_bfloat16>(pack, a, st) : checkpoint_pick<float>(pack, a, st);
}

template <typename T>
static cudaError_t swiglu_act_pick(bool backward, const SwigluActArgs& a, cudaStream_t st) {
  constexpr int kMost = sizeof(T) == 2 ? 16 : 8, kMostBwd = sizeof(T) == 2 ? 16 : 4;
  const int V = ck_vec(a.I, backward ? kMostBwd : kMost);
  SwigluActKernel k;
  if (V == 1) k = backward ? swiglu_act_bwd_strip_kernel<T> : swiglu_act_strip_kernel<T>;
  else if (backward) k = V == kMostBwd ? swiglu_act_bwd_kernel<T, kMostBwd> : V == 8 ? swiglu_act_bwd_kernel<T, 8>
                                                                                   : swiglu_act_bwd_kernel<T, 4>;
  else k = V == kMost ? swiglu_act_kernel<T, kMost> : V == 8 ? swiglu_act_kernel<T, 8> : swiglu_act_kernel<T, 4>;
  return ck_launch<SwigluActArgs>(k, a, a.R, a.I, V, st);
}

cudaError_t launch_swiglu_act(int dtype, bool backward, const SwigluActArgs& a, cudaStream_t st) {
  return dtype == kDtypeBF16 ? swiglu_act_pick<__nv_bfloat16>(backward, a, st)
                             : swiglu_act_pick<float>(backward, a, st);
}

}  // namespace mm
