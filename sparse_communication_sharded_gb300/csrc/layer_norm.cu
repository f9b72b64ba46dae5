// layer_norm.cu -- residual RMS norm, forward (with an 8-bit output) and backward.
//
// Bound by memory: a row's inputs are read once into registers, the sum of
// squares (or of gradient products) is taken over the warps that hold the row,
// and the outputs are written from the same registers.
//
// A row of up to kWarpCols columns belongs to one warp (no block barrier), a
// wider one to a block that is as wide as the row needs; rows over kBlockCols
// are read twice by the *_wide kernels.
#include <algorithm>

#include "layer_internal.cuh"

namespace scapek {
namespace layer {
namespace {

constexpr int kWarpCols = 1024;
constexpr int kBlockCols = 8192;
constexpr int kWarpRows = 4;  // rows (warps) a block, for the narrow rows

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Sum over the block, the same bits in every thread.  `red` holds 32 floats of
// this call's own: the next call uses another one, so one barrier will do.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  float s = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.0f;
  return warp_sum(s);
}

// Where a thread's vectors lie: vector i of thread t of `width` covers columns
// (i * width + t) * VEC and on.
template <int VEC>
__device__ __forceinline__ int vec_col(int i, int t, int width) { return (i * width + t) * VEC; }

template <typename T, int VEC, int NV, bool WARP>
__global__ __launch_bounds__(WARP ? 32 * kWarpRows : 512) void norm_fwd_kernel(NormFwd a, bool w_vec) {
  __shared__ float red[2][32];
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int width = WARP ? 32 : blockDim.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
  const int blocks_per_row = (a.cols + kBlock - 1) / kBlock;
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = vec_col<VEC>(i, t, width);
    load_weight<VEC>(a.w, a.w_bf16, w_vec, c, min(max(a.cols - c, 0), VEC), w[i]);
  }
  int flip = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    Raw<T, VEC> rx[NV], rr[NV];
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = static_cast<const T*>(a.res) + row * a.ldres;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
      rx[i] = load_raw<VEC>(x + c, a.cols - c);
      rr[i] = load_raw<VEC>(res + c, a.res ? a.cols - c : 0);
    }
    float v[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_floats(rx[i], v[i]);
      if (a.res) {
        float r[VEC];
        to_floats(rr[i], r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] += r[j];
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += v[i][j] * v[i][j];
    ss = WARP ? warp_sum(ss) : block_sum(ss, red[flip]);
    flip ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
      const int n = a.cols - c;
      if (a.h) store_part<VEC>(static_cast<T*>(a.h) + row * a.ldh + c, n, v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * rstd * w[i][j];
      store_part<VEC>(static_cast<T*>(a.y) + row * a.ldy + c, n, v[i]);
      if (a.q)
        warp_pack<VEC>(v[i], n, a.q + row * a.ldq + c,
                       a.scale + row * blocks_per_row + c / kBlock, n > 0 && c % kBlock == 0);
    }
  }
}

// Any width: the row is read a second time (from the caches) for the outputs.
template <typename T>
__global__ __launch_bounds__(512) void norm_fwd_wide_kernel(NormFwd a) {
  __shared__ float red[2][32];
  const int64_t blocks_per_row = (a.cols + kBlock - 1) / kBlock;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldres : nullptr;
    float ss = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float v = (float)x[c] + (res ? (float)res[c] : 0.0f);
      ss += v * v;
    }
    ss = block_sum(ss, red[flip]);
    flip ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int c0 = 0; c0 < a.cols; c0 += blockDim.x) {
      const int c = c0 + threadIdx.x, n = a.cols - c;
      float v[1] = {0.0f}, w[1] = {0.0f};
      if (n > 0) {
        v[0] = (float)x[c] + (res ? (float)res[c] : 0.0f);
        if (a.h) static_cast<T*>(a.h)[row * a.ldh + c] = (T)v[0];
        load_weight<1>(a.w, a.w_bf16, false, c, 1, w);
        v[0] = v[0] * rstd * w[0];
        static_cast<T*>(a.y)[row * a.ldy + c] = (T)v[0];
      }
      if (a.q)
        warp_pack<1>(v, n, a.q + row * a.ldq + c, a.scale + row * blocks_per_row + c / kBlock,
                     n > 0 && c % kBlock == 0);
    }
  }
}

// A thread keeps its columns' weight gradients in registers over all its rows;
// one row of partial sums a block goes to a.partial, added up by sum_partials.
template <typename T, int VEC, int NV, bool WARP>
__global__ __launch_bounds__(WARP ? 32 * kWarpRows : 512) void norm_bwd_kernel(NormBwd a, bool w_vec) {
  __shared__ float red[2][32];
  __shared__ float cross[WARP ? kWarpRows * kWarpCols : 1];
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int width = WARP ? 32 : blockDim.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
  float acc[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[i][j] = 0.0f;
  int flip = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    const float rstd = a.rstd[row];
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh;
    const T* dh = static_cast<const T*>(a.dh) + row * a.lddh;
    Raw<T, VEC> rg[NV], rn[NV], rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
      rg[i] = load_raw<VEC>(dy + c, a.cols - c);
      rn[i] = load_raw<VEC>(h + c, a.cols - c);
      rd[i] = load_raw<VEC>(dh + c, a.dh ? a.cols - c : 0);
    }
    float g[NV][VEC], n[NV][VEC];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
      to_floats(rg[i], g[i]);
      to_floats(rn[i], n[i]);
      float w[VEC];
      load_weight<VEC>(a.w, a.w_bf16, w_vec, c, min(max(a.cols - c, 0), VEC), w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        n[i][j] *= rstd;
        acc[i][j] += g[i][j] * n[i][j];
        g[i][j] *= w[j];
        s += g[i][j] * n[i][j];
      }
    }
    s = WARP ? warp_sum(s) : block_sum(s, red[flip]);
    flip ^= 1;
    const float mean = s / (float)a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[i][j] = rstd * (g[i][j] - n[i][j] * mean);
      if (a.dh) {
        float d[VEC];
        to_floats(rd[i], d);
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[i][j] += d[j];
      }
      store_part<VEC>(static_cast<T*>(a.dx) + row * a.lddx + c, a.cols - c, g[i]);
    }
  }
  if (!a.dw) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (WARP) {
    // the block's warps hold the same columns: add them up in warp order
    float* mine = cross + (threadIdx.x >> 5) * kWarpCols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) mine[vec_col<VEC>(i, t, 32) + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarpRows; ++k) s += cross[k * kWarpCols + c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = vec_col<VEC>(i, t, width);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < a.cols) out[c + j] = acc[i][j];
    }
  }
}

template <typename T>
__global__ __launch_bounds__(512) void norm_bwd_wide_kernel(NormBwd a) {
  __shared__ float red[2][32];
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    float s = 0.0f, w[1];
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      load_weight<1>(a.w, a.w_bf16, false, c, 1, w);
      s += (float)dy[c] * w[0] * ((float)h[c] * rstd);
    }
    s = block_sum(s, red[flip]);
    flip ^= 1;
    const float mean = s / (float)a.cols;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      load_weight<1>(a.w, a.w_bf16, false, c, 1, w);
      float d = rstd * ((float)dy[c] * w[0] - (float)h[c] * rstd * mean);
      if (dh) d += (float)dh[c];
      dx[c] = (T)d;
    }
  }
}
// Weight gradient of wide rows, before dx is written (dx may be dy): block
// (x, y) sums rows y, y + gridDim.y, ... of its 256 columns.
template <typename T>
__global__ __launch_bounds__(256) void norm_dw_wide_kernel(NormBwd a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
    s += (float)static_cast<const T*>(a.dy)[row * a.lddy + c] *
         ((float)static_cast<const T*>(a.h)[row * a.ldh + c] * a.rstd[row]);
  a.partial[(int64_t)blockIdx.y * a.cols + c] = s;
}

// Column sums: a block takes 64 columns (two a thread) and every gridDim.y-th
// group of 8 rows.
constexpr int kSumCols = 64;
__global__ __launch_bounds__(256) void colsum_kernel(const bf16* m, int64_t ld, int64_t rows,
                                                     int64_t cols, float* partial) {
  __shared__ float part[8][kSumCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + lane;
  float s0 = 0.0f, s1 = 0.0f;
  for (int64_t r = (int64_t)blockIdx.y * 8 + warp; r < rows; r += (int64_t)gridDim.y * 8) {
    if (c < cols) s0 += __bfloat162float(m[r * ld + c]);
    if (c + 32 < cols) s1 += __bfloat162float(m[r * ld + c + 32]);
  }
  part[warp][lane] = s0;
  part[warp][lane + 32] = s1;
  __syncthreads();
  if (threadIdx.x < kSumCols) {
    const int64_t o = (int64_t)blockIdx.x * kSumCols + threadIdx.x;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += part[k][threadIdx.x];
    if (o < cols) partial[(int64_t)blockIdx.y * cols + o] = s;
  }
}

// 32 columns a block, 8 warps over the rows of partial sums.
__global__ __launch_bounds__(256) void sum_partials_kernel(const float* partial, int64_t parts,
                                                           int64_t cols, void* out, int out_bf16) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int64_t p = warp; p < parts; p += 8) s += partial[p * cols + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float r = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) r += part[k][lane];
    if (out_bf16)
      static_cast<bf16*>(out)[c] = __float2bfloat16_rn(r);
    else
      static_cast<float*>(out)[c] = r;
  }
}

// Launch shape of a row kernel: warps own rows up to kWarpCols, blocks above.
struct Shape {
  bool warp;
  int nv;  // vectors of 8 a thread
  int threads;
  unsigned grid;
};
Shape shape_of(int64_t rows, int64_t cols, int blocks_per_sm) {
  Shape s;
  s.warp = cols <= kWarpCols;
  if (s.warp) {
    s.nv = cols <= 256 ? 1 : cols <= 512 ? 2 : 4;
    s.threads = 32 * kWarpRows;
    s.grid = (unsigned)std::min<int64_t>(ceil_div(rows, kWarpRows), (int64_t)sm_count() * blocks_per_sm);
  } else {
    s.nv = cols <= 2048 ? 1 : 2;
    s.threads = (int)(ceil_div(ceil_div(cols, 8 * s.nv), 32) * 32);
    s.grid = (unsigned)std::min<int64_t>(rows, (int64_t)sm_count() * blocks_per_sm);
  }
  return s;
}

// Runs CALL with NV and WARP as constants for a shape (NV counts vectors of
// 8 values, so a VEC 1 kernel has 8 NV of them).
#define SCAPE_SHAPE_SWITCH(s, CALL)                                        \
  if (s.warp) {                                                            \
    constexpr bool WARP = true;                                            \
    if (s.nv == 1) { constexpr int NV = 1; CALL; }                         \
    else if (s.nv == 2) { constexpr int NV = 2; CALL; }                    \
    else { constexpr int NV = 4; CALL; }                                   \
  } else {                                                                 \
    constexpr bool WARP = false;                                           \
    if (s.nv == 1) { constexpr int NV = 1; CALL; }                         \
    else { constexpr int NV = 2; CALL; }                                   \
  }

constexpr int kFwdBlocksPerSm = 8;
constexpr int kBwdBlocksPerSm = 4;

template <typename T>
cudaError_t run_norm_fwd(const NormFwd& a, cudaStream_t st) {
  if (a.cols > kBlockCols) {
    norm_fwd_wide_kernel<T><<<(unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * 4), 512, 0, st>>>(a);
    return cudaGetLastError();
  }
  const Shape s = shape_of(a.rows, a.cols, kFwdBlocksPerSm);
  const size_t e = sizeof(T);
  const bool vec = rows16(a.x, a.ldx, e) && rows16(a.res, a.ldres, e) && rows16(a.y, a.ldy, e) &&
                   rows16(a.h, a.ldh, e) && rows8(a.q, a.ldq);
  const bool wv = aligned(a.w, 16);
  if (vec) {
    SCAPE_SHAPE_SWITCH(s, (norm_fwd_kernel<T, 8, NV, WARP><<<s.grid, s.threads, 0, st>>>(a, wv)));
  } else {
    SCAPE_SHAPE_SWITCH(s, (norm_fwd_kernel<T, 1, NV * 8, WARP><<<s.grid, s.threads, 0, st>>>(a, wv)));
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_norm_bwd(const NormBwd& a, cudaStream_t st) {
  const int64_t parts = norm_bwd_partials(a.rows, a.cols);
  if (a.cols > kBlockCols) {
    if (a.dw) {
      norm_dw_wide_kernel<T><<<dim3((unsigned)ceil_div(a.cols, 256), (unsigned)parts), 256, 0, st>>>(a);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    norm_bwd_wide_kernel<T><<<(unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * 4), 512, 0, st>>>(a);
  } else {
    const Shape s = shape_of(a.rows, a.cols, kBwdBlocksPerSm);
    const size_t e = sizeof(T);
    const bool vec = rows16(a.dy, a.lddy, e) && rows16(a.h, a.ldh, e) &&
                     rows16(a.dh, a.lddh, e) && rows16(a.dx, a.lddx, e);
    const bool wv = aligned(a.w, 16);
    if (vec) {
      SCAPE_SHAPE_SWITCH(s, (norm_bwd_kernel<T, 8, NV, WARP><<<s.grid, s.threads, 0, st>>>(a, wv)));
    } else {
      SCAPE_SHAPE_SWITCH(s, (norm_bwd_kernel<T, 1, NV * 8, WARP><<<s.grid, s.threads, 0, st>>>(a, wv)));
    }
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dw) return e;
  return launch_sum_partials(a.partial, parts, a.cols, a.dw, a.dw_bf16, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_norm_fwd<bf16>(a, st) : run_norm_fwd<float>(a, st);
}
int64_t norm_bwd_partials(int64_t rows, int64_t cols) {
  if (cols > kBlockCols) return std::min<int64_t>(ceil_div(rows, 8), 64);
  return shape_of(rows, cols, kBwdBlocksPerSm).grid;
}
cudaError_t launch_norm_bwd(const NormBwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_norm_bwd<bf16>(a, st) : run_norm_bwd<float>(a, st);
}

int64_t colsum_partials(int64_t rows, int64_t cols) {
  const int64_t across = ceil_div(cols, kSumCols);
  const int64_t want = std::max<int64_t>(1, (int64_t)sm_count() * 8 / across);
  return std::max<int64_t>(1, std::min(want, ceil_div(rows, 32)));
}
cudaError_t launch_colsum(const bf16* m, int64_t ld, int64_t rows, int64_t cols, float* partial,
                          void* out, int out_bf16, cudaStream_t st) {
  const int64_t parts = colsum_partials(rows, cols);
  colsum_kernel<<<dim3((unsigned)ceil_div(cols, kSumCols), (unsigned)parts), 256, 0, st>>>(
      m, ld, rows, cols, partial);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_sum_partials(partial, parts, cols, out, out_bf16, st);
}
cudaError_t launch_sum_partials(const float* partial, int64_t parts, int64_t cols, void* out,
                                int out_bf16, cudaStream_t st) {
  sum_partials_kernel<<<(unsigned)ceil_div(cols, 32), 256, 0, st>>>(partial, parts, cols, out, out_bf16);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace scapek
