// layer_norm.cu -- residual RMS norm, forward (with an 8-bit output) and backward.
//
// Bound by memory: a row's inputs are read once into registers, the sum of
// squares (or of gradient products) is taken over the warps that hold the row,
// and the outputs are written from the same registers.
//
// A row of up to 1024 columns (backward 512) belongs to one warp (no block barrier), a
// wider one to a block that is as wide as the row needs; rows over kBlockCols
// are read twice by the *_wide kernels.
#include <algorithm>

#include "layer_internal.cuh"

namespace scapek {
namespace layer {
namespace {

constexpr int kWarpCols = 1024;   // forward
constexpr int kWarpColsBwd = 512;  // backward, which holds twice as much a column
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

// Vector i of thread t of `width` covers columns (i * width + t) * VEC and on.

// WIDTH threads own a row: 32 (a warp) or a block of that many; 0: the block's
// size, known at launch only.
template <int WIDTH>
struct Team {
  static constexpr bool kWarp = WIDTH == 32;
  static constexpr int kThreads = kWarp ? 32 * kWarpRows : WIDTH ? WIDTH : 512;
  __device__ static int lane() { return kWarp ? threadIdx.x & 31 : threadIdx.x; }
  __device__ static int width() { return WIDTH ? WIDTH : blockDim.x; }
  __device__ static int64_t first() {
    return kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  }
  __device__ static int64_t step() { return kWarp ? (int64_t)gridDim.x * kWarpRows : gridDim.x; }
};

template <typename T, int VEC, int NV, int WIDTH>
__global__ __launch_bounds__(Team<WIDTH>::kThreads) void norm_fwd_kernel(
    const __grid_constant__ NormFwd a, bool w_vec) {
  using TM = Team<WIDTH>;
  __shared__ float red[2][32];
  const int t = TM::lane(), width = TM::width();
  const int blocks_per_row = (a.cols + kBlock - 1) / kBlock;
  const int mine = a.cols - t * VEC;  // columns from this thread's first on
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    load_weight<VEC>(a.w, a.w_bf16, w_vec, (i * width + t) * VEC, mine - i * width * VEC, w[i]);
  int flip = 0;
  for (int64_t row = TM::first(); row < a.rows; row += TM::step()) {
    Raw<T, VEC> rx[NV], rr[NV];
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + t * VEC;
    const T* res = static_cast<const T*>(a.res) + row * a.ldres + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = load_raw<VEC>(x + i * width * VEC, mine - i * width * VEC);
      rr[i] = load_raw<VEC>(res + i * width * VEC, a.res ? mine - i * width * VEC : 0);
    }
    float v[NV][VEC];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_floats(rx[i], v[i]);
      if (a.res) {
        float r[VEC];
        to_floats(rr[i], r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += v[i][j] * v[i][j];
    }
    ss = TM::kWarp ? warp_sum(ss) : block_sum(ss, red[flip]);
    flip ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    if (a.h) {
      T* h = static_cast<T*>(a.h) + row * a.ldh + t * VEC;
#pragma unroll
      for (int i = 0; i < NV; ++i) store_part<VEC>(h + i * width * VEC, mine - i * width * VEC, v[i]);
    }
    T* y = static_cast<T*>(a.y) + row * a.ldy + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * rstd * w[i][j];
      store_part<VEC>(y + i * width * VEC, mine - i * width * VEC, v[i]);
    }
    if (a.q) {
      uint8_t* q = a.q + row * a.ldq + t * VEC;
      uint8_t* scale = a.scale + row * blocks_per_row + t * VEC / kBlock;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = mine - i * width * VEC;
        warp_pack<VEC>(v[i], n, q + i * width * VEC, scale + i * width * VEC / kBlock,
                       n > 0 && t * VEC % kBlock == 0);
      }
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
// The next row's loads are in flight while this one is summed over the block.
template <typename T, int VEC, int NV, int WIDTH>
__global__ __launch_bounds__(Team<WIDTH>::kThreads) void norm_bwd_kernel(
    const __grid_constant__ NormBwd a, bool w_vec) {
  using TM = Team<WIDTH>;
  __shared__ float red[2][32];
  __shared__ float cross[TM::kWarp ? kWarpRows * kWarpColsBwd : 1];
  const int t = TM::lane(), width = TM::width();
  const int mine = a.cols - t * VEC;
  // eight columns' weights stay in registers, more are read again every row
  constexpr bool kHoldWeight = NV * VEC <= 8;
  float acc[NV][VEC], held[kHoldWeight ? NV : 1][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (kHoldWeight)
      load_weight<VEC>(a.w, a.w_bf16, w_vec, (i * width + t) * VEC, mine - i * width * VEC, held[i % (kHoldWeight ? NV : 1)]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[i][j] = 0.0f;
  }
  Raw<T, VEC> rg[NV], rn[NV], rd[NV];
  float rstd = 0.0f;
  auto load_row = [&](int64_t row) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy + t * VEC;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh + t * VEC;
    const T* dh = static_cast<const T*>(a.dh) + row * a.lddh + t * VEC;
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = mine - i * width * VEC;
      rg[i] = load_raw<VEC>(dy + i * width * VEC, n);
      rn[i] = load_raw<VEC>(h + i * width * VEC, n);
      rd[i] = load_raw<VEC>(dh + i * width * VEC, a.dh ? n : 0);
    }
  };
  int flip = 0;
  int64_t row = TM::first();
  if (row < a.rows) load_row(row);
  while (row < a.rows) {
    const float r = rstd;
    float g[NV][VEC], n[NV][VEC];
    Raw<T, VEC> d[NV];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_floats(rg[i], g[i]);
      to_floats(rn[i], n[i]);
      d[i] = rd[i];
    }
    const int64_t next = row + TM::step();
    if (next < a.rows) load_row(next);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[VEC];
      if (!kHoldWeight)
        load_weight<VEC>(a.w, a.w_bf16, w_vec, (i * width + t) * VEC, mine - i * width * VEC, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        n[i][j] *= r;
        acc[i][j] += g[i][j] * n[i][j];
        g[i][j] *= kHoldWeight ? held[i % (kHoldWeight ? NV : 1)][j] : w[j];
        s += g[i][j] * n[i][j];
      }
    }
    s = TM::kWarp ? warp_sum(s) : block_sum(s, red[flip]);
    flip ^= 1;
    const float mean = s / (float)a.cols;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float add[VEC];
      to_floats(d[i], add);
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[i][j] = r * (g[i][j] - n[i][j] * mean) + (a.dh ? add[j] : 0.0f);
      store_part<VEC>(dx + i * width * VEC, mine - i * width * VEC, g[i]);
    }
    row = next;
  }
  if (!a.dw) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (TM::kWarp) {
    // the block's warps hold the same columns: add them up in warp order
    float* own = cross + (threadIdx.x >> 5) * kWarpColsBwd;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) own[(i * 32 + t) * VEC + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarpRows; ++k) s += cross[k * kWarpColsBwd + c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (i * width * VEC + j < mine) out[(i * width + t) * VEC + j] = acc[i][j];
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

// Column sums in one launch: a cluster of kSumBlocks blocks shares kSumCols
// columns, each block taking its share of the rows; the parts meet in the first
// block's shared memory, in block order.
constexpr int kSumCols = 64;
constexpr int kSumBlocks = 8;
constexpr int kSumThreads = 512;

template <int VEC>
__global__ __launch_bounds__(kSumThreads) __cluster_dims__(kSumBlocks, 1, 1) void colsum_kernel(
    const bf16* m, int64_t ld, int64_t rows, int64_t cols, void* out, int out_bf16) {
  // VEC 8: eight threads a row, VEC 1: 64
  constexpr int kPerRow = kSumCols / VEC, kRows = kSumThreads / kPerRow;
  __shared__ float part[kRows][kSumCols + 4];
  __shared__ float sums[kSumBlocks][kSumCols];
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int at = threadIdx.x % kPerRow, r0 = threadIdx.x / kPerRow;
  const int64_t c = (int64_t)(blockIdx.x / kSumBlocks) * kSumCols + at * VEC;
  const int n = (int)min((int64_t)VEC, cols - c);
  const int64_t begin = rows * rank / kSumBlocks, end = rows * (rank + 1) / kSumBlocks;
  float s[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[j] = 0.0f;
  constexpr int kUnroll = 4;
  for (int64_t r = begin + r0; r < end; r += kRows * kUnroll) {
    Raw<bf16, VEC> v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      v[u] = load_raw<VEC>(m + (r + u * kRows) * ld + c, r + u * kRows < end ? n : 0);
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
  // to the first block: kSumCols sums of this one
  if (threadIdx.x < kSumCols) {
    float t = 0.0f;
#pragma unroll 8
    for (int k = 0; k < kRows; ++k) t += part[k][threadIdx.x];
    uint32_t to = (uint32_t)__cvta_generic_to_shared(&sums[rank][threadIdx.x]);
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(to) : "r"(0));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(t) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
  if (rank == 0 && threadIdx.x < kSumCols) {
    const int64_t o = (int64_t)(blockIdx.x / kSumBlocks) * kSumCols + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kSumBlocks; ++k) t += sums[k][threadIdx.x];
    if (o < cols) {
      if (out_bf16)
        static_cast<bf16*>(out)[o] = __float2bfloat16_rn(t);
      else
        static_cast<float*>(out)[o] = t;
    }
  }
}

// 32 columns a block, 32 warps over the rows of partial sums.
__global__ __launch_bounds__(1024) void sum_partials_kernel(const float* partial, int64_t parts,
                                                            int64_t cols, void* out, int out_bf16) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
    constexpr int kUnroll = 8;
    for (int64_t p = warp; p < parts; p += 32 * kUnroll) {
      float v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u] = p + u * 32 < parts ? partial[(p + u * 32) * cols + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) s += v[u];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  // warp w sums the 32 parts of column w
  const float r = warp_sum(part[lane][warp]);
  const int64_t o = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) {
    if (out_bf16)
      static_cast<bf16*>(out)[o] = __float2bfloat16_rn(r);
    else
      static_cast<float*>(out)[o] = r;
  }
}

// Launch shape of a row kernel: warps own rows up to kWarpCols, blocks above.
// Eight columns a thread need a block as wide as the row; single columns (rows
// of any alignment) need a width known to the compiler, so that a thread's
// addresses are one register and constants (777 x 1283 float32 with the 8-bit
// output: 10.8 us with the width in a register).
struct Shape {
  int nv;     // vectors of 8 (or their 8 single columns) a thread
  int width;  // threads a row
  int threads;
  unsigned grid;
};
Shape shape_of(int64_t rows, int64_t cols, bool vec, int warp_cols, int blocks_per_sm) {
  Shape s;
  const int64_t most = (int64_t)sm_count() * blocks_per_sm;
  if (cols <= warp_cols) {
    s.nv = cols <= 256 ? 1 : cols <= 512 ? 2 : 4;
    s.width = 32;
    s.threads = 32 * kWarpRows;
    s.grid = (unsigned)std::min(ceil_div(rows, kWarpRows), most);
  } else {
    s.nv = cols <= (vec ? 2048 : 4096) ? 1 : 2;
    s.threads = vec ? (int)(ceil_div(ceil_div(cols, 8 * s.nv), 32) * 32) : cols <= 1024 ? 128 : cols <= 2048 ? 256 : 512;
    s.width = vec ? 0 : s.threads;
    s.grid = (unsigned)std::min(rows, most);
  }
  return s;
}

// Runs CALL with VEC, NV and WIDTH as constants for a shape (rows of up to
// WARP_COLS columns belong to a warp).
#define SCAPE_SHAPE_SWITCH(vec, s, WARP_COLS, CALL)                                         \
  if (vec) {                                                                                \
    constexpr int VEC = 8;                                                                  \
    if (s.width == 32) {                                                                    \
      constexpr int WIDTH = 32;                                                             \
      if (s.nv == 1) { constexpr int NV = 1; CALL; }                                        \
      else if (s.nv == 2) { constexpr int NV = 2; CALL; }                                   \
      else { constexpr int NV = WARP_COLS / 256; CALL; }                                    \
    } else {                                                                                \
      constexpr int WIDTH = 0;                                                              \
      if (s.nv == 1) { constexpr int NV = 1; CALL; }                                        \
      else { constexpr int NV = 2; CALL; }                                                  \
    }                                                                                       \
  } else {                                                                                  \
    constexpr int VEC = 1;                                                                  \
    if (s.width == 32) {                                                                    \
      constexpr int WIDTH = 32;                                                             \
      if (s.nv == 1) { constexpr int NV = 8; CALL; }                                        \
      else if (s.nv == 2) { constexpr int NV = 16; CALL; }                                  \
      else { constexpr int NV = WARP_COLS / 32; CALL; }                                     \
    } else if (s.width == 128) {                                                            \
      constexpr int WIDTH = 128, NV = 8;                                                    \
      CALL;                                                                                 \
    } else if (s.width == 256) {                                                            \
      constexpr int WIDTH = 256, NV = 8;                                                    \
      CALL;                                                                                 \
    } else {                                                                                \
      constexpr int WIDTH = 512;                                                            \
      if (s.nv == 1) { constexpr int NV = 8; CALL; }                                        \
      else { constexpr int NV = 16; CALL; }                                                 \
    }                                                                                       \
  }

constexpr int kFwdBlocksPerSm = 8;
constexpr int kBwdBlocksPerSm = 4;

template <typename T>
cudaError_t run_norm_fwd(const NormFwd& a, cudaStream_t st) {
  if (a.cols > kBlockCols) {
    norm_fwd_wide_kernel<T><<<(unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * 4), 512, 0, st>>>(a);
    return cudaGetLastError();
  }
  const size_t e = sizeof(T);
  const bool vec = rows16(a.x, a.ldx, e) && rows16(a.res, a.ldres, e) && rows16(a.y, a.ldy, e) &&
                   rows16(a.h, a.ldh, e) && rows8(a.q, a.ldq);
  const bool wv = aligned(a.w, 16);
  const Shape s = shape_of(a.rows, a.cols, vec, kWarpCols, kFwdBlocksPerSm);
  SCAPE_SHAPE_SWITCH(vec, s, kWarpCols, (norm_fwd_kernel<T, VEC, NV, WIDTH><<<s.grid, s.threads, 0, st>>>(a, wv)));
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
    const size_t e = sizeof(T);
    const bool vec = rows16(a.dy, a.lddy, e) && rows16(a.h, a.ldh, e) &&
                     rows16(a.dh, a.lddh, e) && rows16(a.dx, a.lddx, e);
    const bool wv = aligned(a.w, 16);
    const Shape s = shape_of(a.rows, a.cols, vec, kWarpColsBwd, kBwdBlocksPerSm);
    SCAPE_SHAPE_SWITCH(vec, s, kWarpColsBwd, (norm_bwd_kernel<T, VEC, NV, WIDTH><<<s.grid, s.threads, 0, st>>>(a, wv)));
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
  return shape_of(rows, cols, true, kWarpColsBwd, kBwdBlocksPerSm).grid;  // the grid does not go by `vec`
}
cudaError_t launch_norm_bwd(const NormBwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_norm_bwd<bf16>(a, st) : run_norm_bwd<float>(a, st);
}

cudaError_t launch_colsum(const bf16* m, int64_t ld, int64_t rows, int64_t cols, void* out,
                          int out_bf16, cudaStream_t st) {
  const unsigned grid = (unsigned)ceil_div(cols, kSumCols) * kSumBlocks;
  if (rows16(m, ld, 2))
    colsum_kernel<8><<<grid, kSumThreads, 0, st>>>(m, ld, rows, cols, out, out_bf16);
  else
    colsum_kernel<1><<<grid, kSumThreads, 0, st>>>(m, ld, rows, cols, out, out_bf16);
  return cudaGetLastError();
}
cudaError_t launch_sum_partials(const float* partial, int64_t parts, int64_t cols, void* out,
                                int out_bf16, cudaStream_t st) {
  sum_partials_kernel<<<(unsigned)ceil_div(cols, 32), 1024, 0, st>>>(partial, parts, cols, out, out_bf16);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace scapek
