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
// VEC 8 needs 16-byte alignment, VEC 1 none.
template <typename T, int VEC>
struct Raw {
  static constexpr int kWords = VEC * sizeof(T) >= 4 ? VEC * sizeof(T) / 4 : 1;
  uint32_t w[kWords];
};
template <int VEC, typename T>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p, int n) {
  Raw<T, VEC> r;
  if (n >= VEC) {
    if constexpr (VEC == 8) {
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
  if constexpr (VEC == 8) {
    uint4 u;
    u.x = bf16_pair(v[0], v[1]), u.y = bf16_pair(v[2], v[3]);
    u.z = bf16_pair(v[4], v[5]), u.w = bf16_pair(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
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
__device__ __forceinline__ void to_e4m3(const float (&v)[N], float inv, bool no_inf,
                                        uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float a = v[4 * i] * inv, b = v[4 * i + 1] * inv, c = v[4 * i + 2] * inv,
          d = v[4 * i + 3] * inv;
    if (!no_inf) {
      a = nan_unless_finite(a), b = nan_unless_finite(b);
      c = nan_unless_finite(c), d = nan_unless_finite(d);
    }
    w[i] = e4m3_pair(a, b) | (e4m3_pair(c, d) << 16);
  }
}
// Four e4m3 values as floats (exact).
__device__ __forceinline__ void from_e4m3(uint32_t w, float scale, float* v) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
}
__device__ __forceinline__ float from_e4m3_byte(uint32_t b, float scale) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
  return __half2float(__half(h)) * scale;
}

// One warp's 32 lanes pack VEC values each; with VEC 8 four neighbouring lanes
// hold a block, with VEC 1 the whole warp does.  n values of the thread are
// real (the others are 0).  All 32 lanes call it together.
template <int VEC>
__device__ __forceinline__ void warp_pack(const float (&v)[VEC], int n, uint8_t* q, uint8_t* scale,
                                          bool writes_scale) {
  uint32_t top = part_top<VEC>(v);
  bool no_inf = true;
  if constexpr (VEC == 1) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (top >= kInfBits) {
      top = __reduce_max_sync(0xFFFFFFFFu, part_top_finite<VEC>(v));
      no_inf = false;
    }
  } else {
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (__any_sync(0xFFFFFFFFu, top >= kInfBits)) {
      top = part_top_finite<VEC>(v);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      no_inf = false;
    }
  }
  const uint32_t code = scale_code(top);
  const float inv = scale_inverse(code);
  if constexpr (VEC == 1) {
    const float x = v[0] * inv;
    if (n > 0) *q = (uint8_t)e4m3_pair(no_inf ? x : nan_unless_finite(x), 0.0f);
  } else {
    uint32_t w[2];
    to_e4m3<8>(v, inv, no_inf, w);
    if (n >= 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
  if (writes_scale) *scale = (uint8_t)code;
}

// ------------------------------------------------------------------ activations
// gelu's 0.5 (1 + tanh u) is the logistic function of 2u, so gelu and silu are
// both z * logistic(a): one exponential and one reciprocal a value, and a
// relative (not absolute) error where the result is small.  Two values at a
// time: the multiplications and additions are packed 32-bit pairs, which halves
// their issue slots; the exponential and the reciprocal (16 a clock an SM) are
// then what bounds the arithmetic.
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
__device__ __forceinline__ uint64_t both(float a) { return pair(a, a); }
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
// Limits that keep a NaN.
__device__ __forceinline__ float at_least(float x, float lo) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
  return r;
}
__device__ __forceinline__ float at_most(float x, float hi) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(hi));
  return r;
}

constexpr double kLog2e = 1.4426950408889634074;
constexpr double kGelu2C = 1.5957691216057307117;  // 2 sqrt(2 / pi)
constexpr double kGeluA = 0.044715;
__host__ __device__ constexpr float high(double x) { return (float)x; }
__host__ __device__ constexpr float low(double x) { return (float)(x - (double)(float)x); }

// The logistic function of silu's and gelu's argument a at z, by 2^e with
// e = -a log2(e).  An error d in e is a relative error 0.69 d of the result where
// that is small: at e = 100 the roundings of e alone are 2^-18 or so.  A bfloat16
// result cannot show that; DEEP, for 32-bit results, carries e's roundings and
// its constants' low parts along as d and corrects 2^e by 1 + d ln 2.
template <int ACT, bool DEEP>
__device__ __forceinline__ uint64_t logistic2(uint64_t z) {
  constexpr double k0 = ACT == SCAPE_ACT_GELU ? -kGelu2C * kLog2e : -kLog2e;
  constexpr double k1 = -kGelu2C * kGeluA * kLog2e;
  uint64_t t = both(high(k0)), z2 = 0;
  if constexpr (ACT == SCAPE_ACT_GELU) {
    z2 = mul2(z, z);
    t = fma2(z2, both(high(k1)), both(high(k0)));
  }
  const uint64_t e = mul2(z, t);
  float a, b;
  unpair(e, a, b);
  uint64_t x = pair(exp2_fast(a), exp2_fast(b));
  if constexpr (DEEP) {
    const uint64_t minus = both(-1.0f);
    uint64_t t_low = both(low(k0));
    if constexpr (ACT == SCAPE_ACT_GELU)
      t_low = fma2(z2, both(low(k1)), add2(both(low(k0)), fma2(z2, both(high(k1)), fma2(t, minus, both(high(k0))))));
    const uint64_t d = fma2(z, t_low, fma2(z, t, mul2(e, minus)));
    float da, db;
    unpair(mul2(d, both(0.69314718f)), da, db);
    unpair(x, a, b);
    // where e or z^2 has overflowed d says nothing, and 2^e is 0 or infinite
    x = pair(a > 1e-37f && a < 1e37f ? fmaf(a, da, a) : a,
             b > 1e-37f && b < 1e37f ? fmaf(b, db, b) : b);
  }
  unpair(add2(x, both(1.0f)), a, b);
  return pair(reciprocal_fast(a), reciprocal_fast(b));
}

template <int ACT, bool DEEP = false>
__device__ __forceinline__ void act_pair(float& x, float& y) {
  if constexpr (ACT == SCAPE_ACT_RELU) {
    x = at_least(x, 0.0f);
    y = at_least(y, 0.0f);
  } else if constexpr (ACT == SCAPE_ACT_GELU || ACT == SCAPE_ACT_SILU) {
    const uint64_t z = pair(x, y);
    unpair(mul2(z, logistic2<ACT, DEEP>(z)), x, y);
  }
}
// x, y become the activation's slopes there.  Past |z| = 20 (gelu) and 100 (silu)
// the logistic is 0 or 1 to the last bit and so is the slope; the limit keeps 0
// times an overflowed z^2 out.
template <int ACT>
__device__ __forceinline__ void slope_pair(float& x, float& y) {
  if constexpr (ACT == SCAPE_ACT_RELU) {
    x = x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
    y = y > 0.0f ? 1.0f : (y != y ? y : 0.0f);
  } else if constexpr (ACT == SCAPE_ACT_GELU || ACT == SCAPE_ACT_SILU) {
    constexpr float kLim = ACT == SCAPE_ACT_GELU ? 20.0f : 100.0f;
    const uint64_t z = pair(at_most(at_least(x, -kLim), kLim), at_most(at_least(y, -kLim), kLim));
    const uint64_t p = logistic2<ACT, false>(z);
    uint64_t m = z;  // z da/dz
    if constexpr (ACT == SCAPE_ACT_GELU)
      m = mul2(z, fma2(mul2(z, z), both(high(3.0 * kGelu2C * kGeluA)), both(high(kGelu2C))));
    const uint64_t pq = fma2(mul2(p, both(-1.0f)), p, p);  // p (1 - p)
    unpair(fma2(m, pq, p), x, y);
  } else {
    x = y = 1.0f;
  }
}
template <int ACT, bool DEEP = false, int N>
__device__ __forceinline__ void act_values(float (&v)[N]) {
  if constexpr (N == 1) {
    float other = 0.0f;
    act_pair<ACT, DEEP>(v[0], other);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) act_pair<ACT, DEEP>(v[2 * i], v[2 * i + 1]);
  }
}
template <int ACT, int N>
__device__ __forceinline__ void act_slopes(float (&v)[N]) {
  if constexpr (N == 1) {
    float other = 0.0f;
    slope_pair<ACT>(v[0], other);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) slope_pair<ACT>(v[2 * i], v[2 * i + 1]);
  }
}

// CALL with ACT a constant, for an activation known at run time.
#define SCAPE_ACT_SWITCH(act, CALL)                              \
  switch (act) {                                                 \
    case SCAPE_ACT_RELU: { constexpr int ACT = SCAPE_ACT_RELU; CALL; break; } \
    case SCAPE_ACT_GELU: { constexpr int ACT = SCAPE_ACT_GELU; CALL; break; } \
    case SCAPE_ACT_SILU: { constexpr int ACT = SCAPE_ACT_SILU; CALL; break; } \
    default: { constexpr int ACT = SCAPE_ACT_NONE; CALL; break; }             \
  }

// ------------------------------------------------------------------ launchers
cudaError_t launch_pack8(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* q, int64_t ldq, uint8_t* scale, cudaStream_t st);
cudaError_t launch_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                           int64_t cols, int act, void* y, int64_t ldy, int dtype,
                           cudaStream_t st);
cudaError_t launch_act_grad(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                            const uint8_t* scale, int64_t rows, int64_t cols, int act, void* dz,
                            int64_t lddz, int dtype, cudaStream_t st);

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
int64_t colsum_partials(int64_t rows, int64_t cols);
cudaError_t launch_colsum(const bf16* m, int64_t ld, int64_t rows, int64_t cols, float* partial,
                          void* out, int out_bf16, cudaStream_t st);
// Sum of `parts` rows of partial[parts, cols].
cudaError_t launch_sum_partials(const float* partial, int64_t parts, int64_t cols, void* out,
                                int out_bf16, cudaStream_t st);

}  // namespace layer
}  // namespace scapek
