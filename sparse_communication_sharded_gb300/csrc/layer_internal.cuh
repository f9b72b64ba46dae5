// layer_internal.cuh -- device helpers shared by the training-layer operators
// (include/scape_layers.h): vector loads and stores, the 8-bit block format and
// the activations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "scape_layers.h"

namespace scapek {

int sm_count();

namespace layer {

using bf16 = __nv_bfloat16;
constexpr int kBlock = SCAPE_PACK_BLOCK;

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// A row-major matrix whose every row starts on a 16-byte boundary.
inline bool rows16(const void* p, int64_t ld, size_t elem) {
  return p == nullptr || (aligned(p, 16) && (ld * (int64_t)elem) % 16 == 0);
}
// The same for the 8-byte rows that one thread's eight 8-bit values take.
inline bool rows8(const void* p, int64_t ld) {
  return p == nullptr || (aligned(p, 8) && ld % 8 == 0);
}

// ------------------------------------------------------------------ loads and stores
// VEC consecutive elements as they lie in memory.  Loads fill these and nothing
// else, so that a thread has all its loads in flight before it converts the
// first: a conversion between two loads would wait for the one before it.
// VEC 8 and 16 need 16-byte alignment, VEC 1 none.
template <typename T, int VEC>
struct Raw {
  static constexpr int kWords = VEC * sizeof(T) >= 4 ? VEC * sizeof(T) / 4 : 1;
  uint32_t w[kWords];
};
template <int VEC, typename T>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p, int n) {
  Raw<T, VEC> r;
  if (n >= VEC) {
    if constexpr (VEC >= 8) {
#pragma unroll
      for (int i = 0; i < Raw<T, VEC>::kWords / 4; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
      }
    } else if constexpr (sizeof(T) == 2) {
      r.w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  } else {
    // a row's end: the first n elements, zeros after
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords; ++i) r.w[i] = 0;
    if (VEC > 1 && n > 0) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 2)
            r.w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
          else
            r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
    }
  }
  return r;
}
// The same for rows of any alignment, VEC 8 or 16: a piece of 16 bytes is cut out of
// the two aligned ones that hold it (the second is the neighbour's first, so it
// comes from L1).  What lies between lo and hi is the matrix: pieces whose aligned
// words do not lie there entirely are read element by element.
template <int VEC, typename T>
__device__ __forceinline__ Raw<T, VEC> load_any(const T* p, int n, const T* lo, const T* hi) {
  constexpr int kPer = 16 / sizeof(T);
  Raw<T, VEC> r;
#pragma unroll
  for (int i = 0; i < VEC / kPer; ++i) {
    const T* q = p + i * kPer;
    const int have = n - i * kPer;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(q) & 15u);
    const char* a = reinterpret_cast<const char*>(q) - off;
    uint32_t w[8];
    if (have >= kPer && off == 0) {
      const uint4 u = *reinterpret_cast<const uint4*>(a);
      r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
    } else if (have >= kPer && a >= reinterpret_cast<const char*>(lo) &&
               a + 32 <= reinterpret_cast<const char*>(hi)) {
      const uint4 u = reinterpret_cast<const uint4*>(a)[0], v = reinterpret_cast<const uint4*>(a)[1];
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
      if (off & 8) {
#pragma unroll
        for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        r.w[4 * i + j] = sizeof(T) == 4 ? w[j] : __funnelshift_r(w[j], w[j + 1], (off & 2) * 8);
    } else {
      Raw<T, kPer> part;
#pragma unroll
      for (int j = 0; j < 4; ++j) part.w[j] = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j < have) {
          if constexpr (sizeof(T) == 2)
            part.w[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(q)[j] << (16 * (j % 2));
          else
            part.w[j] = reinterpret_cast<const uint32_t*>(q)[j];
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * i + j] = part.w[j];
    }
  }
  return r;
}
// The same in two steps, so that a thread's loads are in flight together: the
// branches of load_any() keep one waiting for the other.  begin() loads the aligned
// words that hold VEC elements (one word more than they are), end() puts the elements
// together; where those words do not lie in the matrix entirely, end() reads element
// by element.  Of fewer than VEC elements (n, at a row's end) the others are what
// follows in the matrix, or 0.
template <typename T, int VEC>
struct AnyLoad {
  static constexpr int kPer = 16 / sizeof(T), kPieces = VEC / kPer;
  uint4 w[kPieces + 1];
  uint32_t off;
  bool fast;
  __device__ __forceinline__ void begin(const T* p, int n, const T* lo, const T* hi) {
    off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* a = reinterpret_cast<const char*>(p) - off;
    fast = n > 0 && a >= reinterpret_cast<const char*>(lo) &&
           a + 16 * (kPieces + (off ? 1 : 0)) <= reinterpret_cast<const char*>(hi);
#pragma unroll
    for (int i = 0; i <= kPieces; ++i)
      if (fast && (i < kPieces || off)) w[i] = reinterpret_cast<const uint4*>(a)[i];
  }
  __device__ __forceinline__ Raw<T, VEC> end(const T* p, int n) const {
    Raw<T, VEC> r;
    if (fast) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint32_t v[8] = {w[i].x, w[i].y, w[i].z, w[i].w, w[i + 1].x, w[i + 1].y, w[i + 1].z, w[i + 1].w};
        if (off & 8) {
#pragma unroll
          for (int j = 0; j < 6; ++j) v[j] = v[j + 2];
        }
        if (off & 4) {
#pragma unroll
          for (int j = 0; j < 5; ++j) v[j] = v[j + 1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r.w[4 * i + j] = sizeof(T) == 4 ? v[j] : __funnelshift_r(v[j], v[j + 1], (off & 2) * 8);
      }
    } else {
#pragma unroll
      for (int j = 0; j < Raw<T, VEC>::kWords; ++j) r.w[j] = 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (j < n) {
          if constexpr (sizeof(T) == 2)
            r.w[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
          else
            r.w[j] = reinterpret_cast<const uint32_t*>(p)[j];
        }
    }
    return r;
  }
};
template <typename T, int VEC>
__device__ __forceinline__ void to_floats(const Raw<T, VEC>& r, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if constexpr (sizeof(T) == 2)
      v[i] = __uint_as_float(i % 2 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
    else
      v[i] = __uint_as_float(r.w[i]);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <int VEC>
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[VEC]) {
  if constexpr (VEC >= 8) {
#pragma unroll
    for (int i = 0; i < VEC / 8; ++i)
      reinterpret_cast<uint4*>(p)[i] =
          make_uint4(bf16_pair(v[8 * i], v[8 * i + 1]), bf16_pair(v[8 * i + 2], v[8 * i + 3]),
                     bf16_pair(v[8 * i + 4], v[8 * i + 5]), bf16_pair(v[8 * i + 6], v[8 * i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC >= 8) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = v[i];
  }
}

// The first n (0..VEC) elements of a vector at a row's end.
template <int VEC, typename T>
__device__ __forceinline__ void store_part(T* p, int n, const float (&v)[VEC]) {
  if (n >= VEC) {
    store_vec<VEC>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = (T)v[i];
  }
}
// Part of a weight vector of either type (the same for the whole grid), which
// may lie at any element of a flat parameter vector (aligned: on 16 bytes).
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, int is_bf16, bool aligned, int64_t c,
                                            int n, float (&v)[VEC]) {
  if (is_bf16) {
    const bf16* p = static_cast<const bf16*>(w) + c;
    if (VEC == 1 || aligned) {
      to_floats<bf16, VEC>(load_raw<VEC>(p, n), v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
  } else {
    const float* p = static_cast<const float*>(w) + c;
    if (VEC == 1 || aligned) {
      to_floats<float, VEC>(load_raw<VEC>(p, n), v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
  }
}

// ------------------------------------------------------------------ packed pairs of floats
// One instruction for two values: half the issue slots.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ------------------------------------------------------------------ the 8-bit block format
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// Scale code of a block whose largest finite magnitude has these bits.  A
// magnitude 1.f 2^(E-127) is at most 448 2^c = 1.75 2^(c+8) for c = E-127-8
// when 1.f <= 1.75, and for one more otherwise; code = c + 127, at least 1 so
// that the scale and its reciprocal are normal numbers.
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
  const int c = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(c, 1);
}
__device__ __forceinline__ float scale_value(uint32_t code) { return __uint_as_float(code << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return __uint_as_float((254u - code) << 23);
}
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Infinities become NaN (the conversion would clamp them); a NaN stays one.
__device__ __forceinline__ float nan_unless_finite(float x) {
  return abs_bits(x) >= kInfBits ? __uint_as_float(0x7FC00000u) : x;
}

// Bits of the largest magnitude among N values (not counting NaN), and among
// the finite ones.
template <int N>
__device__ __forceinline__ uint32_t part_top(const float (&v)[N]) {
  constexpr int kLanes = N >= 16 ? 4 : 1;  // chains that do not wait for each other
  float t[kLanes] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) t[i % kLanes] = fmaxf(t[i % kLanes], fabsf(v[i]));
  if constexpr (kLanes == 4) t[0] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
  return __float_as_uint(t[0]);
}
template <int N>
__device__ __forceinline__ uint32_t part_top_finite(const float (&v)[N]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = abs_bits(v[i]);
    if (b < kInfBits) t = max(t, b);
  }
  return t;
}
// e4m3 words of N values (N a multiple of 4) at a scale.  Scaling by a power of
// two is exact down to the subnormals, where e4m3 is 0.
template <int N>
__device__ __forceinline__ void to_e4m3(const float (&v)[N], float inv, uint32_t (&w)[N / 4]) {
  const uint64_t inv2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float a, b, c, d;
    unpair(mul2(pair(v[4 * i], v[4 * i + 1]), inv2), a, b);
    unpair(mul2(pair(v[4 * i + 2], v[4 * i + 3]), inv2), c, d);
    w[i] = e4m3_pair(a, b) | (e4m3_pair(c, d) << 16);
  }
}
// Four e4m3 values as two pairs of floats, before their scale (exact).
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint64_t& lo, uint64_t& hi) {
  const __half2_raw l = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(l)), b = __half22float2(__half2(h));
  lo = pair(a.x, a.y);
  hi = pair(b.x, b.y);
}
// One warp's 32 lanes pack VEC values each; with VEC 16 two neighbouring lanes
// hold a block, with VEC 8 four, with VEC 1 the whole warp.  n values of the thread are
// real (the others are 0).  q is on 8 bytes, or 16 where q16 says so (VEC 1: any).
// All 32 lanes call it together.
template <int VEC>
__device__ __forceinline__ void warp_pack(const float (&values)[VEC], int n, uint8_t* q,
                                          uint8_t* scale, bool writes_scale, bool q16) {
  float v[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = values[i];
  uint32_t top = part_top<VEC>(v);
  if constexpr (VEC == 1) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (top >= kInfBits) {
      top = __reduce_max_sync(0xFFFFFFFFu, part_top_finite<VEC>(v));
      v[0] = nan_unless_finite(v[0]);
    }
  } else {
    auto over_lanes = [](uint32_t t) {
      t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
      if (VEC == 8) t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
      return t;
    };
    top = over_lanes(top);
    if (__any_sync(0xFFFFFFFFu, top >= kInfBits)) {
      top = over_lanes(part_top_finite<VEC>(v));
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = nan_unless_finite(v[i]);
    }
  }
  const uint32_t code = scale_code(top);
  const float inv = scale_inverse(code);
  if constexpr (VEC == 1) {
    if (n > 0) *q = (uint8_t)e4m3_pair(v[0] * inv, 0.0f);
  } else {
    uint32_t w[VEC / 4];
    to_e4m3<VEC>(v, inv, w);
    if (n >= VEC) {
      if constexpr (VEC == 16) {
        if (q16) {
          *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          reinterpret_cast<uint2*>(q)[0] = make_uint2(w[0], w[1]);
          reinterpret_cast<uint2*>(q)[1] = make_uint2(w[2], w[3]);
        }
      } else {
        *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
  if (writes_scale) *scale = (uint8_t)code;
}

// ------------------------------------------------------------------ activations
// gelu's 0.5 (1 + tanh u) is the logistic function of 2u, so gelu and silu are
// both z * logistic(a): one exponential and one reciprocal a value, and a
// relative (not absolute) error where the result is small.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// x if it is above 0 (or not a number), else 0.
__device__ __forceinline__ float above_zero(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}
// A constant in both halves of a register pair, which the compiler takes for a
// value it cannot make again: without this it made the constants anew for every
// use, two moves each, half as many instructions again as the arithmetic.
__device__ __forceinline__ uint64_t held(float a) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}

constexpr double kLog2e = 1.4426950408889634074;
constexpr double kGelu2C = 1.5957691216057307117;  // 2 sqrt(2 / pi)
constexpr double kGeluA = 0.044715;
constexpr double kGeluK0 = -kGelu2C * kLog2e;  // 2^(z (K0 + K1 z^2)) = exp(-2u)
constexpr double kGeluK1 = -kGelu2C * kGeluA * kLog2e;
__host__ __device__ constexpr float high(double x) { return (float)x; }
__host__ __device__ constexpr float low(double x) { return (float)(x - (double)(float)x); }

// An activation on pairs of values z = q s with a common scale s, which goes into
// the coefficients.  2^e with e = q (a + b q^2) gives the logistic function
// p = 1 / (1 + 2^e).  Where s is over 2^20 the exponent takes 2^20 for it: any q
// but 0 is then at least 2^-9, so |z| is over 2^11 either way and p is 0 or 1.
template <int ACT>
struct Activation {
  static constexpr bool kLogistic = ACT == SCAPE_ACT_GELU || ACT == SCAPE_ACT_SILU;
  uint64_t s, a, b, one;

  __device__ __forceinline__ explicit Activation(float scale) {
    s = held(scale);
    if constexpr (kLogistic) {
      const float l = fminf(scale, 1048576.0f);
      one = held(1.0f);
      if constexpr (ACT == SCAPE_ACT_GELU) {
        a = held(high(kGeluK0) * l);
        b = held(high(kGeluK1) * l * l * l);
      } else {
        a = held(high(-kLog2e) * l);
      }
    }
  }
  __device__ __forceinline__ uint64_t logistic(uint64_t q) const {
    uint64_t t = a;
    if constexpr (ACT == SCAPE_ACT_GELU) t = fma2(mul2(q, q), b, a);
    float x, y;
    unpair(mul2(q, t), x, y);
    unpair(add2(pair(exp2_fast(x), exp2_fast(y)), one), x, y);
    return pair(reciprocal_fast(x), reciprocal_fast(y));
  }
  // act(q s)
  __device__ __forceinline__ uint64_t value(uint64_t q) const {
    if constexpr (kLogistic) return mul2(mul2(q, s), logistic(q));
    if constexpr (ACT == SCAPE_ACT_RELU) {
      float x, y;
      unpair(mul2(q, s), x, y);
      return pair(above_zero(x), above_zero(y));
    }
    return mul2(q, s);
  }
};

// act(z) for z without a scale.
template <int ACT, int N>
__device__ __forceinline__ void act_values(float (&v)[N]) {
  if constexpr (ACT == SCAPE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = above_zero(v[i]);
  } else if constexpr (ACT != SCAPE_ACT_NONE) {
    const Activation<ACT> f(1.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t z = pair(v[i], N == 1 ? 0.0f : v[(i + 1) % N]);
      float other;
      unpair(mul2(z, f.logistic(z)), v[i], N == 1 ? other : v[(i + 1) % N]);
    }
  }
}

// act'(q s): p + z a'(z) p (1 - p), whose second term is q (c + d q^2) p (1 - p)
// with c = s, d = 0 for silu.  With the exponent's limit on s nothing overflows:
// |z| stays below 2^29.
template <int ACT>
struct Slope : Activation<ACT> {
  uint64_t c, d, minus;
  __device__ __forceinline__ explicit Slope(float scale) : Activation<ACT>(scale) {
    if constexpr (Activation<ACT>::kLogistic) {
      const float l = fminf(scale, 1048576.0f);
      minus = held(-1.0f);
      if constexpr (ACT == SCAPE_ACT_GELU) {
        c = held(high(kGelu2C) * l);
        d = held(high(3.0 * kGelu2C * kGeluA) * l * l * l);
      } else {
        c = held(l);
      }
    }
  }
  __device__ __forceinline__ uint64_t slope(uint64_t q) const {
    if constexpr (Activation<ACT>::kLogistic) {
      const uint64_t p = this->logistic(q);
      uint64_t t = c;
      if constexpr (ACT == SCAPE_ACT_GELU) t = fma2(mul2(q, q), d, c);
      return fma2(mul2(q, t), fma2(mul2(p, minus), p, p), p);
    }
    float x, y;
    unpair(q, x, y);
    if constexpr (ACT == SCAPE_ACT_RELU) {
      x = x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
      y = y > 0.0f ? 1.0f : (y != y ? y : 0.0f);
    } else {
      x = y = 1.0f;
    }
    return pair(x, y);
  }
};

// 32-bit results.  An error d in e is a relative error 0.69 d of 2^e, and at
// e = 100, far out in the tail, the roundings of e alone are 2^-18 or so: no
// bfloat16 result shows it, a 32-bit one does.  So e's roundings and its
// constants' low parts are carried along as d, and 2^e corrected by 1 + d ln 2.
template <int ACT>
__device__ __forceinline__ float exp_exact(float z) {
  constexpr double k0 = ACT == SCAPE_ACT_GELU ? kGeluK0 : -kLog2e;
  float t = high(k0), t_low = low(k0);
  if constexpr (ACT == SCAPE_ACT_GELU) {
    // the product's error and the sum's (either term may be the larger: Knuth, The
    // Art of Computer Programming 2, 4.2.2), not contracted into one rounding
    const float z2 = z * z, a = __fmul_rn(z2, high(kGeluK1));
    t = __fadd_rn(a, high(k0));
    const float b = __fsub_rn(t, a);
    const float sum_low = __fadd_rn(__fsub_rn(a, __fsub_rn(t, b)), __fsub_rn(high(k0), b));
    t_low = fmaf(z2, low(kGeluK1), low(k0)) + (fmaf(z2, high(kGeluK1), -a) + sum_low);
  }
  const float e = z * t;
  const float d = fmaf(z, t_low, fmaf(z, t, -e));
  const float x = exp2_fast(e);
  // where e or z^2 has overflowed d says nothing, and 2^e is 0 or infinite
  return x > 1e-37f && x < 1e37f ? fmaf(x, d * 0.69314718f, x) : x;
}
template <int ACT>
__device__ __forceinline__ float act_exact(float z) {
  if constexpr (ACT == SCAPE_ACT_RELU) return above_zero(z);
  if constexpr (ACT == SCAPE_ACT_GELU || ACT == SCAPE_ACT_SILU) return z * reciprocal_fast(1.0f + exp_exact<ACT>(z));
  return z;
}
// p + z a'(z) p (1 - p), whose 1 - p is 2^e p: a difference would have no digits
// where p is near 1.  Past |z| = 1024 the second term is 0 (limited there, it does
// not overflow); 2^e is limited where p is 0.
template <int ACT>
__device__ __forceinline__ float slope_exact(float z) {
  static_assert(ACT == SCAPE_ACT_GELU || ACT == SCAPE_ACT_SILU, "the others' slopes need no arithmetic");
  const float x = exp_exact<ACT>(z), p = reciprocal_fast(1.0f + x);
  const float l = fminf(fmaxf(z, -1024.0f), 1024.0f);
  const float g = ACT == SCAPE_ACT_GELU ? l * fmaf(l * l, high(3.0 * kGelu2C * kGeluA), high(kGelu2C)) : l;
  return fmaf(g * p, fminf(x, 1e37f) * p, p);
}

// CALL with ACT a constant, for an activation known at run time.
#define SCAPE_ACT_SWITCH(act, CALL)                              \
  switch (act) {                                                 \
    case SCAPE_ACT_RELU: { constexpr int ACT = SCAPE_ACT_RELU; CALL; break; } \
    case SCAPE_ACT_GELU: { constexpr int ACT = SCAPE_ACT_GELU; CALL; break; } \
    case SCAPE_ACT_SILU: { constexpr int ACT = SCAPE_ACT_SILU; CALL; break; } \
    default: { constexpr int ACT = SCAPE_ACT_NONE; CALL; break; }             \
  }

// ------------------------------------------------------------------ launches
// Every kernel here is launched so that it may start while the one before it on
// the stream ends: start() lets the next one do the same, and waits until all
// earlier work is complete and visible.  Nothing is read or written before it.
// What overlaps is the launch and the set-up (64 x 256 through 256 x 256, one
// after the other: 8.2 us a call without, 5.3 to 6.6 with).
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void start() {
  let_next_start();
  wait_for_earlier();
}
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 threads, size_t smem, int cluster,
                          cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ------------------------------------------------------------------ clusters
// Blocks of a cluster that give sums to the first one: cluster_begin() at the
// start, cluster_ready() before the first to_first() (all blocks have begun by
// then), cluster_done() before the first block reads.  All threads call each.
__device__ __forceinline__ uint32_t block_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_begin() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_ready() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_done() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Stores to the same place of the cluster's first block.
__device__ __forceinline__ void to_first(float* p, float v) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(0));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// ------------------------------------------------------------------ column sums
// Of m[rows, cols] in 32 bits: a cluster of `cluster` blocks shares kSumCols
// columns, each block taking its share of the rows; the parts meet in the first
// block's shared memory, in block order.  The clusters are the grid's first.
struct ColumnSums {
  const bf16* m;
  int64_t ld, rows, cols;
  void* out;
  int out_bf16;
};
constexpr int kSumCols = 64;
constexpr int kSumBlocks = 8;
// In clusters of one block where there is little to add up: they start sooner.
inline int sum_cluster(int64_t rows) { return rows <= 256 ? 1 : kSumBlocks; }

// After cluster_begin(); eight columns a thread, rows of any alignment with ANY.
template <int THREADS, bool ANY>
__device__ __forceinline__ void sum_columns(const ColumnSums& a) {
  constexpr int VEC = 8, kPerRow = kSumCols / VEC, kRows = THREADS / kPerRow, kUnroll = 8;
  __shared__ float part[kRows][kSumCols + 4];
  __shared__ float sums[kSumBlocks][kSumCols];
  const bf16* hi = a.m + (a.rows - 1) * a.ld + a.cols;
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  const int at = threadIdx.x % kPerRow, r0 = threadIdx.x / kPerRow;
  const int64_t c = (int64_t)(blockIdx.x / ranks) * kSumCols + at * VEC;
  const int n = (int)min((int64_t)VEC, a.cols - c);
  const int64_t begin = a.rows * rank / ranks, end = a.rows * (rank + 1) / ranks;
  float s[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[j] = 0.0f;
  for (int64_t r = begin + r0; r < end; r += kRows * kUnroll) {
    Raw<bf16, VEC> v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bf16* p = a.m + (r + u * kRows) * a.ld + c;
      const int left = r + u * kRows < end ? n : 0;
      if constexpr (ANY)
        v[u] = load_any<VEC>(p, left, a.m, hi);
      else
        v[u] = load_raw<VEC>(p, left);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[VEC];
      to_floats(v[u], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[j] += f[j];
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) part[r0][at * VEC + j] = s[j];
  __syncthreads();
  cluster_ready();
  // to the first block: kSumCols sums of this one
  if (threadIdx.x < kSumCols) {
    float t = 0.0f;
#pragma unroll 8
    for (int k = 0; k < kRows; ++k) t += part[k][threadIdx.x];
    to_first(&sums[rank][threadIdx.x], t);
  }
  cluster_done();
  if (rank == 0 && threadIdx.x < kSumCols) {
    const int64_t o = (int64_t)(blockIdx.x / ranks) * kSumCols + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kSumBlocks; ++k)
      if (k < ranks) t += sums[k][threadIdx.x];
    if (o < a.cols) {
      if (a.out_bf16)
        static_cast<bf16*>(a.out)[o] = __float2bfloat16_rn(t);
      else
        static_cast<float*>(a.out)[o] = t;
    }
  }
}

// ------------------------------------------------------------------ launchers
cudaError_t launch_pack8(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* q, int64_t ldq, uint8_t* scale, cudaStream_t st);
cudaError_t launch_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                           int64_t cols, int act, void* y, int64_t ldy, int dtype,
                           cudaStream_t st);
// unpack8 to bfloat16 rows on 16 bytes, and column sums of another matrix beside
// it in the same launch.
cudaError_t launch_unpack8_sums(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                                int64_t cols, int act, bf16* y, int64_t ldy, const ColumnSums& sums,
                                cudaStream_t st);
cudaError_t launch_act_grad(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                            const uint8_t* scale, int64_t rows, int64_t cols, int act, void* dz,
                            int64_t lddz, int dtype, cudaStream_t st);

// Lets a kernel use this much dynamic shared memory; CUDA is asked when a kernel
// first wants more than before.
cudaError_t allow_smem(const void* kernel, int bytes);

struct NormFwd {
  const void *x, *res, *w;
  int64_t ldx, ldres, ldy, ldh, ldq;
  int w_bf16;
  int64_t rows;
  int cols;
  float eps;
  void *y, *h;
  float* rstd;
  uint8_t *q, *scale;
  bool q16;  // rows of q on 16 bytes
};
cudaError_t launch_norm_fwd(const NormFwd& a, int dtype, cudaStream_t st);

struct NormBwd {
  const void *dy, *h, *w, *dh;
  int64_t lddy, ldh, lddh, lddx;
  const float* rstd;
  int w_bf16, dw_bf16;
  int64_t rows;
  int cols;
  void *dx, *dw;
  float* partial;  // rows of partial weight gradients, one a block
};
int64_t norm_bwd_partials(int64_t rows, int64_t cols);
cudaError_t launch_norm_bwd(const NormBwd& a, int dtype, cudaStream_t st);

// Column sums of m[rows, cols] (bfloat16) in 32 bits.
cudaError_t launch_colsum(const ColumnSums& a, cudaStream_t st);
// Sum of `parts` rows of partial[parts, cols].
cudaError_t launch_sum_partials(const float* partial, int64_t parts, int64_t cols, void* out,
                                int out_bf16, cudaStream_t st);

}  // namespace layer
}  // namespace scapek
