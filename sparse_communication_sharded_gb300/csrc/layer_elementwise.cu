// layer_elementwise.cu -- 8-bit activation checkpoints: pack, unpack (through an
// activation) and the gradient through an activation kept in 8 bits.
//
// Each is one streaming pass over rows x cols values: bound by memory.  A row is
// cut into units of VEC columns, a thread takes unroll() units that lie a block's
// width apart, so that their loads are all in flight before the first is used.
#include <algorithm>

#include "layer_internal.cuh"

namespace scapek {
namespace layer {
namespace {

constexpr int kThreads = 256;
// Units a thread: 32 columns, or 8 of single columns.
template <int VEC>
__host__ __device__ constexpr int unroll() {
  return VEC == 16 ? 2 : VEC == 8 ? 4 : 8;
}

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

// ANY: rows of x of any alignment (lo, hi: where x begins and ends).
template <typename T, int VEC, bool ANY>
__global__ __launch_bounds__(kThreads) void pack8_kernel(const T* x, int64_t ldx, const T* lo, const T* hi,
                                                         uint32_t units, FastDiv per_row, int64_t cols,
                                                         uint8_t* q, int64_t ldq, uint8_t* scale,
                                                         int64_t blocks_per_row) {
  start();
  constexpr int U = unroll<VEC>();
  const uint32_t first = blockIdx.x * (kThreads * U) + threadIdx.x;
  Unit un[U];
  Raw<T, VEC> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    const T* p = x + un[i].row * ldx + un[i].col;
    if constexpr (ANY)
      raw[i] = load_any<VEC>(p, un[i].n, lo, hi);
    else
      raw[i] = load_raw<VEC>(p, un[i].n);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Unit& u = un[i];
    float v[VEC];
    to_floats(raw[i], v);
    warp_pack<VEC>(v, u.n, q + u.row * ldq + u.col,
                   scale + u.row * blocks_per_row + u.col / kBlock,
                   u.n > 0 && u.col % kBlock == 0, VEC == 16);
  }
}

// The 8-bit values of a unit and their scale.
template <int VEC>
struct Packed {
  uint32_t w[VEC >= 4 ? VEC / 4 : 1];
  uint32_t code;
};
// ANY (VEC 8): 8 bytes at any address, cut out of the two aligned 8-byte words that
// hold them where both lie between lo and hi, the matrix.
template <int VEC, bool ANY = false>
__device__ __forceinline__ Packed<VEC> load_packed(const uint8_t* q, int64_t ldq,
                                                   const uint8_t* scale, int64_t blocks_per_row,
                                                   const Unit& u, const uint8_t* lo = nullptr,
                                                   const uint8_t* hi = nullptr) {
  Packed<VEC> p = {};
  if (u.n > 0) {
    const uint8_t* s = q + u.row * ldq + u.col;
    p.code = scale[u.row * blocks_per_row + u.col / kBlock];
    if (VEC == 16 && u.n == 16) {
      const uint4 a = *reinterpret_cast<const uint4*>(s);
      p.w[0] = a.x, p.w[VEC == 16 ? 1 : 0] = a.y;
      p.w[VEC == 16 ? 2 : 0] = a.z, p.w[VEC == 16 ? 3 : 0] = a.w;
    } else if (VEC == 8 && u.n == 8 && !ANY) {
      const uint2 a = *reinterpret_cast<const uint2*>(s);
      p.w[0] = a.x, p.w[VEC >= 8 ? 1 : 0] = a.y;
    } else if (VEC == 8 && u.n == 8 && s - (reinterpret_cast<uintptr_t>(s) & 7) >= lo &&
               s - (reinterpret_cast<uintptr_t>(s) & 7) + 16 <= hi) {
      const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(s) & 7);
      const uint2 a = reinterpret_cast<const uint2*>(s - off)[0], b = reinterpret_cast<const uint2*>(s - off)[1];
      const uint32_t w0 = off & 4 ? a.y : a.x, w1 = off & 4 ? b.x : a.y, w2 = off & 4 ? b.y : b.x;
      p.w[0] = __funnelshift_r(w0, w1, (off & 3) * 8);
      p.w[VEC >= 8 ? 1 : 0] = __funnelshift_r(w1, w2, (off & 3) * 8);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < u.n) p.w[i / 4] |= (uint32_t)s[i] << (8 * (i % 4));
    }
  }
  return p;
}

// SUMS: the grid's first sum_blocks blocks take column sums of another matrix.
template <typename T, int VEC, int ACT, bool ANY, bool SUMS>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const uint8_t* q, int64_t ldq, const uint8_t* lo,
                                                           const uint8_t* hi, const uint8_t* scale,
                                                           int64_t blocks_per_row, uint32_t units,
                                                           FastDiv per_row, int64_t cols, T* y,
                                                           int64_t ldy, const __grid_constant__ ColumnSums sums,
                                                           uint32_t sum_blocks) {
  start();
  uint32_t block = blockIdx.x;
  if constexpr (SUMS) {
    if (block < sum_blocks) {
      cluster_begin();
      sum_columns<kThreads, false>(sums);
      return;
    }
    block -= sum_blocks;
  }
  constexpr int U = unroll<VEC>();
  const uint32_t first = block * (kThreads * U) + threadIdx.x;
  Unit un[U];
  Packed<VEC> p[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    p[i] = load_packed<VEC, ANY>(q, ldq, scale, blocks_per_row, un[i], lo, hi);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Activation<ACT> f(scale_value(p[i].code));
    const Activation<SCAPE_ACT_NONE> scaled(scale_value(p[i].code));
    float v[VEC < 4 ? 4 : VEC];
#pragma unroll
    for (int j = 0; j < (VEC < 4 ? 1 : VEC / 4); ++j) {
      uint64_t lo, hi;
      e4m3_pairs(p[i].w[j], lo, hi);
      if constexpr (sizeof(T) == 4) {
        unpair(scaled.value(lo), v[4 * j], v[4 * j + 1]);
        unpair(scaled.value(hi), v[4 * j + 2], v[4 * j + 3]);
#pragma unroll
        for (int l = 0; l < (VEC < 4 ? VEC : 4); ++l) v[4 * j + l] = act_exact<ACT>(v[4 * j + l]);
      } else {
        unpair(f.value(lo), v[4 * j], v[4 * j + 1]);
        unpair(f.value(hi), v[4 * j + 2], v[4 * j + 3]);
      }
    }
    store_part<VEC>(y + un[i].row * ldy + un[i].col, un[i].n, reinterpret_cast<float (&)[VEC]>(v));
  }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void act_grad_kernel(
    const T* dy, int64_t lddy, const uint8_t* q, int64_t ldq, const uint8_t* scale,
    int64_t blocks_per_row, uint32_t units, FastDiv per_row, int64_t cols, T* dz, int64_t lddz) {
  start();
  constexpr int U = unroll<VEC>();
  const uint32_t first = blockIdx.x * (kThreads * U) + threadIdx.x;
  Unit un[U];
  Packed<VEC> p[U];
  Raw<T, VEC> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    un[i] = unit_at<VEC>(first + i * kThreads, units, per_row, cols);
    p[i] = load_packed<VEC>(q, ldq, scale, blocks_per_row, un[i]);
    raw[i] = load_raw<VEC>(dy + un[i].row * lddy + un[i].col, un[i].n);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float g[VEC];
    to_floats(raw[i], g);
    if constexpr (sizeof(T) == 4 && Slope<ACT>::kLogistic) {
      const float scale = scale_value(p[i].code);
#pragma unroll
      for (int j = 0; j < (VEC < 4 ? 1 : VEC / 4); ++j) {
        uint64_t lo, hi;
        e4m3_pairs(p[i].w[j], lo, hi);
        float q[4];
        unpair(lo, q[0], q[1]);
        unpair(hi, q[2], q[3]);
#pragma unroll
        for (int l = 0; l < (VEC < 4 ? VEC : 4); ++l) g[4 * j + l] *= slope_exact<ACT>(q[l] * scale);
      }
    } else {
      const Slope<ACT> f(scale_value(p[i].code));
      if constexpr (VEC == 1) {
        uint64_t lo, hi;
        e4m3_pairs(p[i].w[0], lo, hi);
        float other;
        unpair(mul2(f.slope(lo), pair(g[0], 0.0f)), g[0], other);
      } else {
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j) {
          uint64_t lo, hi;
          e4m3_pairs(p[i].w[j], lo, hi);
          unpair(mul2(f.slope(lo), pair(g[4 * j], g[4 * j + 1])), g[4 * j], g[4 * j + 1]);
          unpair(mul2(f.slope(hi), pair(g[4 * j + 2], g[4 * j + 3])), g[4 * j + 2], g[4 * j + 3]);
        }
      }
    }
    store_part<VEC>(dz + un[i].row * lddz + un[i].col, un[i].n, g);
  }
}

// Calls launch(row0, units, per_row, grid) for row ranges of fewer than 2^30
// units each, so that unit numbers stay within the 31 bits of FastDiv.
template <int VEC, typename F>
cudaError_t for_row_ranges(int64_t rows, int64_t cols, F&& launch) {
  const int64_t per_row = ceil_div(cols, kBlock) * (kBlock / VEC);
  const int64_t step = std::max<int64_t>(1, (int64_t{1} << 30) / per_row);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t units = std::min(step, rows - r) * per_row;
    const cudaError_t e = launch(r, (uint32_t)units, FastDiv((uint32_t)per_row),
                                 (unsigned)ceil_div(units, kThreads * unroll<VEC>()));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int VEC, bool ANY>
cudaError_t run_pack8(const T* x, int64_t ldx, int64_t rows, int64_t cols, uint8_t* q, int64_t ldq,
                      uint8_t* scale, cudaStream_t st) {
  const int64_t bpr = ceil_div(cols, kBlock);
  const T* end = x + (rows - 1) * ldx + cols;
  return for_row_ranges<VEC>(rows, cols, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    return launch_kernel(pack8_kernel<T, VEC, ANY>, grid, kThreads, 0, 0, st, x + r * ldx, ldx, x, end, units,
                         d, cols, q + r * ldq, ldq, scale + r * bpr, bpr);
  });
}
template <typename T, int VEC, bool ANY, bool SUMS = false>
cudaError_t run_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                        int64_t cols, int act, T* y, int64_t ldy, cudaStream_t st,
                        const ColumnSums& sums = {}) {
  const int64_t bpr = ceil_div(cols, kBlock);
  const int cluster = SUMS ? sum_cluster(sums.rows) : 0;
  unsigned sum_blocks = SUMS ? (unsigned)(ceil_div(sums.cols, kSumCols) * cluster) : 0;
  return for_row_ranges<VEC>(rows, cols, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    cudaError_t e = cudaSuccess;
    if (SUMS) grid = (unsigned)(ceil_div(grid, cluster) * cluster) + sum_blocks;
    SCAPE_ACT_SWITCH(act, e = (launch_kernel(unpack8_kernel<T, VEC, ACT, ANY, SUMS>, grid, kThreads, 0, cluster, st, q + r * ldq, ldq, q, q + (rows - 1) * ldq + cols,
                                             scale + r * bpr, bpr, units, d, cols, y + r * ldy, ldy, sums,
                                             sum_blocks)));
    sum_blocks = 0;  // once
    return e;
  });
}
template <typename T, int VEC>
cudaError_t run_act_grad(const T* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                         const uint8_t* scale, int64_t rows, int64_t cols, int act, T* dz,
                         int64_t lddz, cudaStream_t st) {
  const int64_t bpr = ceil_div(cols, kBlock);
  return for_row_ranges<VEC>(rows, cols, [&](int64_t r, uint32_t units, FastDiv d, unsigned grid) {
    cudaError_t e = cudaSuccess;
    SCAPE_ACT_SWITCH(act, e = (launch_kernel(act_grad_kernel<T, VEC, ACT>, grid, kThreads, 0, 0, st,
                                             dy + r * lddy, lddy, q + r * ldq, ldq, scale + r * bpr, bpr,
                                             units, d, cols, dz + r * lddz, lddz)));
    return e;
  });
}

// Columns a thread, as the rows' alignment allows: 16 (one 16-byte word of 8-bit
// values), 8, or 1: a warp then reads 32 neighbouring columns, a whole block, at
// a time.  16 against 8: unpack8 of 8192 x 5632 to bfloat16 took 25.4 against
// 26.4 us, the fewer addresses for the same bytes.
#define SCAPE_VEC_SWITCH(v16, v8, CALL)                \
  do {                                                 \
    if (v16) { constexpr int VEC = 16; return CALL; }  \
    if (v8) { constexpr int VEC = 8; return CALL; }    \
    { constexpr int VEC = 1; return CALL; }            \
  } while (0)

template <typename T>
cudaError_t pack8_of(const T* x, int64_t ldx, int64_t rows, int64_t cols, uint8_t* q, int64_t ldq,
                     uint8_t* scale, cudaStream_t st) {
  if (rows16(x, ldx, sizeof(T)))
    SCAPE_VEC_SWITCH(rows16(q, ldq, 1), rows8(q, ldq),
                     (run_pack8<T, VEC, false>(x, ldx, rows, cols, q, ldq, scale, st)));
  SCAPE_VEC_SWITCH(false, rows8(q, ldq),
                   (run_pack8<T, VEC, (VEC > 1)>(x, ldx, rows, cols, q, ldq, scale, st)));
}
template <typename T>
cudaError_t unpack8_of(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                       int64_t cols, int act, T* y, int64_t ldy, cudaStream_t st) {
  const bool ok = rows16(y, ldy, sizeof(T));
  if (ok && !rows8(q, ldq)) return run_unpack8<T, 8, true>(q, ldq, scale, rows, cols, act, y, ldy, st);
  SCAPE_VEC_SWITCH(ok && rows16(q, ldq, 1), ok,
                   (run_unpack8<T, VEC, false>(q, ldq, scale, rows, cols, act, y, ldy, st)));
}
template <typename T>
cudaError_t act_grad_of(const T* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                        const uint8_t* scale, int64_t rows, int64_t cols, int act, T* dz,
                        int64_t lddz, cudaStream_t st) {
  const bool ok = rows16(dy, lddy, sizeof(T)) && rows16(dz, lddz, sizeof(T));
  SCAPE_VEC_SWITCH(ok && rows16(q, ldq, 1), ok && rows8(q, ldq),
                   (run_act_grad<T, VEC>(dy, lddy, q, ldq, scale, rows, cols, act, dz, lddz, st)));
}

}  // namespace

cudaError_t launch_pack8(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* q, int64_t ldq, uint8_t* scale, cudaStream_t st) {
  return dtype == SCAPE_BF16
             ? pack8_of(static_cast<const bf16*>(x), ldx, rows, cols, q, ldq, scale, st)
             : pack8_of(static_cast<const float*>(x), ldx, rows, cols, q, ldq, scale, st);
}
cudaError_t launch_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                           int64_t cols, int act, void* y, int64_t ldy, int dtype,
                           cudaStream_t st) {
  return dtype == SCAPE_BF16
             ? unpack8_of(q, ldq, scale, rows, cols, act, static_cast<bf16*>(y), ldy, st)
             : unpack8_of(q, ldq, scale, rows, cols, act, static_cast<float*>(y), ldy, st);
}
cudaError_t launch_unpack8_sums(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t rows,
                                int64_t cols, int act, bf16* y, int64_t ldy, const ColumnSums& sums,
                                cudaStream_t st) {
  if (rows16(q, ldq, 1)) return run_unpack8<bf16, 16, false, true>(q, ldq, scale, rows, cols, act, y, ldy, st, sums);
  return run_unpack8<bf16, 8, true, true>(q, ldq, scale, rows, cols, act, y, ldy, st, sums);
}
cudaError_t launch_act_grad(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                            const uint8_t* scale, int64_t rows, int64_t cols, int act, void* dz,
                            int64_t lddz, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16
             ? act_grad_of(static_cast<const bf16*>(dy), lddy, q, ldq, scale, rows, cols, act,
                           static_cast<bf16*>(dz), lddz, st)
             : act_grad_of(static_cast<const float*>(dy), lddy, q, ldq, scale, rows, cols, act,
                           static_cast<float*>(dz), lddz, st);
}

}  // namespace layer
}  // namespace scapek
