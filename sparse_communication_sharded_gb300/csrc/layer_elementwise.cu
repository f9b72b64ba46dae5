// layer_elementwise.cu -- 8-bit activation checkpoints: pack, unpack (through an
// activation) and the gradient through an activation kept in 8 bits.
//
// Each is one streaming pass over rows x cols values: bound by memory.  A row is
// cut into units of VEC columns, a thread takes kUnroll units that lie a block's
// width apart, so that their loads are all in flight before the first is used.
#include <algorithm>

#include "layer_internal.cuh"

namespace scapek {
namespace layer {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t mul, shift, d;
  explicit FastDiv(uint32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < div) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return (__umulhi(mul, n) + n) >> shift;
  }
};

// Unit u of a matrix: its row, first column and how many of its VEC columns
// exist.  Rows are padded to whole blocks of 32 columns, so that the lanes that
// share a block are neighbours; units of the padding hold none.
struct Unit {
  int64_t row;
  int64_t col;
  int n;
};
template <int VEC>
__device__ __forceinline__ Unit unit_at(uint32_t u, uint32_t units, const FastDiv& per_row,
                                        int64_t cols) {
  Unit r;
  const uint32_t row = per_row.quot(u);
  r.row = row;
  r.col = (int64_t)(u - row * per_row.d) * VEC;
  const int64_t left = cols - r.col;
  r.n = u < units && left > 0 ? (int)(left < VEC ? left : VEC) : 0;
  return r;
}

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void pack8_kernel(const T* x, int64_t ldx, uint32_t units,
                                                         FastDiv per_row, int64_t cols, uint8_t* q,
                                                         int64_t ldq, uint8_t* scale,
                                                         int64_t blocks_per_row) {
  const uint32_t first = blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  Unit un[kUnroll];
  Raw<T, VEC> raw[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    raw[i] = load_raw<VEC>(x + un[i].row * ldx + un[i].col, un[i].n);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const Unit& u = un[i];
    float v[VEC];
    to_floats(raw[i], v);
    warp_pack<VEC>(v, u.n, q + u.row * ldq + u.col,
                   scale + u.row * blocks_per_row + u.col / kBlock,
                   u.n > 0 && u.col % kBlock == 0);
  }
}

// The 8-bit values of a unit and their scale.
template <int VEC>
struct Packed {
  uint32_t w[VEC == 8 ? 2 : 1];
  uint32_t code;
};
template <int VEC>
__device__ __forceinline__ Packed<VEC> load_packed(const uint8_t* q, int64_t ldq,
                                                   const uint8_t* scale, int64_t blocks_per_row,
                                                   const Unit& u) {
  Packed<VEC> p = {};
  if (u.n > 0) {
    const uint8_t* s = q + u.row * ldq + u.col;
    if (VEC == 8 && u.n == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(s);
      p.w[0] = a.x;
      p.w[VEC == 8 ? 1 : 0] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < u.n) p.w[i / 4] |= (uint32_t)s[i] << (8 * (i % 4));
    }
    p.code = scale[u.row * blocks_per_row + u.col / kBlock];
  }
  return p;
}
template <int VEC>
__device__ __forceinline__ void values_of(const Packed<VEC>& p, float (&v)[VEC]) {
  const float s = scale_value(p.code);
  if constexpr (VEC == 8) {
    from_e4m3(p.w[0], s, v);
    from_e4m3(p.w[1], s, v + 4);
  } else {
    v[0] = from_e4m3_byte(p.w[0], s);
  }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const uint8_t* q, int64_t ldq,
                                                           const uint8_t* scale,
                                                           int64_t blocks_per_row, uint32_t units,
                                                           FastDiv per_row, int64_t cols, T* y,
                                                           int64_t ldy) {
  const uint32_t first = blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  Unit un[kUnroll];
  Packed<VEC> p[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    p[i] = load_packed<VEC>(q, ldq, scale, blocks_per_row, un[i]);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float v[VEC];
    values_of<VEC>(p[i], v);
    act_values<ACT, sizeof(T) == 4>(v);
    store_part<VEC>(y + un[i].row * ldy + un[i].col, un[i].n, v);
  }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void act_grad_kernel(
    const T* dy, int64_t lddy, const uint8_t* q, int64_t ldq, const uint8_t* scale,
    int64_t blocks_per_row, uint32_t units, FastDiv per_row, int64_t cols, T* dz, int64_t lddz) {
  const uint32_t first = blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  Unit un[kUnroll];
  Packed<VEC> p[kUnroll];
  Raw<T, VEC> raw[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    p[i] = load_packed<VEC>(q, ldq, scale, blocks_per_row, un[i]);
    raw[i] = load_raw<VEC>(dy + un[i].row * lddy + un[i].col, un[i].n);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float v[VEC], g[VEC];
    values_of<VEC>(p[i], v);
    act_slopes<ACT>(v);
    to_floats(raw[i], g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] *= g[j];
    store_part<VEC>(dz + un[i].row * lddz + un[i].col, un[i].n, v);
  }
}

// Calls launch(row0, units, per_row, grid) for row ranges of fewer than 2^30
// units each, so that unit numbers stay within the 31 bits of FastDiv.
template <typename F>
cudaError_t for_row_ranges(int64_t rows, int64_t cols, int vec, F&& launch) {
  const int64_t per_row = ceil_div(cols, kBlock) * (kBlock / vec);
  const int64_t step = std::max<int64_t>(1, (int64_t{1} << 30) / per_row);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t units = std::min(step, rows - r) * per_row;
    launch(r, (uint32_t)units, FastDiv((uint32_t)per_row),
           (unsigned)ceil_div(units, kThreads * kUnroll));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int VEC>
cudaError_t run_pack8(const T* x, int64_t ldx, int64_t rows, int64_t cols, uint8_t* q, int64_t ldq,
                      uint8_t* scale, cudaStream_t st) {
  const int64_t bpr = ceil_div(cols, kBlock);
  return for_row_ranges(rows, cols, VEC, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    pack8_kernel<T, VEC><<<grid, kThreads, 0, st>>>(x + r * ldx, ldx, units, d, cols, q + r * ldq,
                                                    ldq, scale + r * bpr, bpr);
  });
}
template <typename T, int VEC>
cudaError_t run_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                        int64_t cols, int act, T* y, int64_t ldy, cudaStream_t st) {
  const int64_t bpr = ceil_div(cols, kBlock);
  return for_row_ranges(rows, cols, VEC, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    SCAPE_ACT_SWITCH(act, (unpack8_kernel<T, VEC, ACT><<<grid, kThreads, 0, st>>>(
                              q + r * ldq, ldq, scale + r * bpr, bpr, units, d, cols, y + r * ldy,
                              ldy)));
  });
}
template <typename T, int VEC>
cudaError_t run_act_grad(const T* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                         const uint8_t* scale, int64_t rows, int64_t cols, int act, T* dz,
                         int64_t lddz, cudaStream_t st) {
  const int64_t bpr = ceil_div(cols, kBlock);
  return for_row_ranges(rows, cols, VEC, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    SCAPE_ACT_SWITCH(act, (act_grad_kernel<T, VEC, ACT><<<grid, kThreads, 0, st>>>(
                              dy + r * lddy, lddy, q + r * ldq, ldq, scale + r * bpr, bpr, units,
                              d, cols, dz + r * lddz, lddz)));
  });
}

}  // namespace

// Eight columns a thread (16-byte loads) where every row is aligned for them,
// else one: a warp then reads 32 neighbouring columns, a whole block, at a time.
cudaError_t launch_pack8(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* q, int64_t ldq, uint8_t* scale, cudaStream_t st) {
  const size_t e = dtype == SCAPE_BF16 ? 2 : 4;
  const bool vec = rows16(x, ldx, e) && rows8(q, ldq);
  if (dtype == SCAPE_BF16) {
    const bf16* p = static_cast<const bf16*>(x);
    return vec ? run_pack8<bf16, 8>(p, ldx, rows, cols, q, ldq, scale, st)
               : run_pack8<bf16, 1>(p, ldx, rows, cols, q, ldq, scale, st);
  }
  const float* p = static_cast<const float*>(x);
  return vec ? run_pack8<float, 8>(p, ldx, rows, cols, q, ldq, scale, st)
             : run_pack8<float, 1>(p, ldx, rows, cols, q, ldq, scale, st);
}

cudaError_t launch_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                           int64_t cols, int act, void* y, int64_t ldy, int dtype,
                           cudaStream_t st) {
  const size_t e = dtype == SCAPE_BF16 ? 2 : 4;
  const bool vec = rows16(y, ldy, e) && rows8(q, ldq);
  if (dtype == SCAPE_BF16) {
    bf16* p = static_cast<bf16*>(y);
    return vec ? run_unpack8<bf16, 8>(q, ldq, scale, rows, cols, act, p, ldy, st)
               : run_unpack8<bf16, 1>(q, ldq, scale, rows, cols, act, p, ldy, st);
  }
  float* p = static_cast<float*>(y);
  return vec ? run_unpack8<float, 8>(q, ldq, scale, rows, cols, act, p, ldy, st)
             : run_unpack8<float, 1>(q, ldq, scale, rows, cols, act, p, ldy, st);
}

cudaError_t launch_act_grad(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                            const uint8_t* scale, int64_t rows, int64_t cols, int act, void* dz,
                            int64_t lddz, int dtype, cudaStream_t st) {
  const size_t e = dtype == SCAPE_BF16 ? 2 : 4;
  const bool vec = rows16(dy, lddy, e) && rows16(dz, lddz, e) && rows8(q, ldq);
  if (dtype == SCAPE_BF16) {
    const bf16* p = static_cast<const bf16*>(dy);
    bf16* o = static_cast<bf16*>(dz);
    return vec ? run_act_grad<bf16, 8>(p, lddy, q, ldq, scale, rows, cols, act, o, lddz, st)
               : run_act_grad<bf16, 1>(p, lddy, q, ldq, scale, rows, cols, act, o, lddz, st);
  }
  const float* p = static_cast<const float*>(dy);
  float* o = static_cast<float*>(dz);
  return vec ? run_act_grad<float, 8>(p, lddy, q, ldq, scale, rows, cols, act, o, lddz, st)
             : run_act_grad<float, 1>(p, lddy, q, ldq, scale, rows, cols, act, o, lddz, st);
}

}  // namespace layer
}  // namespace scapek
