// layer_skinny.cu -- the linear layer and its gradients for a few rows, where the
// matrix is read (or the gradient written) once and nothing else is in the way:
// bound by memory and, at these sizes, by latency.
//
// The tensor cores would multiply a tile of 128 rows for them and cost a launch's
// set-up (tensor maps, barriers, tensor memory); here a thread multiplies what it
// loads.  4096 x 1024, forward / input gradient / weight and bias gradient, in us:
// 1 row 4.1 / 4.6 / 2.9, 4 rows 5.7 / 6.9 / 3.8, 8 rows 8.5 / 11.2 / 5.1; on the
// tensor cores 7.6 / 9.5 / 10.5 for up to 64 rows.  Hence up to 4 rows (weight
// gradient 8) here.
// Any alignment is read in place: 8 columns a thread where rows allow it, single
// ones (32 neighbours a warp) where not.
#include <algorithm>

#include "layer_gemm.cuh"

namespace scapek {
namespace layer {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ------------------------------------------------------------------ forward
// A block (or a cluster, which cuts the contraction) makes 32 columns of y: each
// warp the dot products of 4 rows of the weight with R rows of x.
constexpr int kCols = 32;
constexpr int kColsPerWarp = kCols / kWarps;

template <int R, int VEC>
__global__ __launch_bounds__(kThreads) void skinny_forward_kernel(
    const bf16* x, int64_t ldx, const bf16* w, int64_t ldw, int rows, int64_t k, int64_t n,
    const __grid_constant__ Epilogue e) {
  constexpr int kRun = 1024;
  __shared__ __align__(16) float xs[R][kRun];
  __shared__ float sums[8][R][kCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  cluster_begin();
  start();
  const int64_t c0 = (int64_t)(blockIdx.x / ranks) * kCols;
  // this block's part of the contraction, in whole warp steps
  constexpr int kStep = 32 * VEC;
  const int64_t steps = (k + kStep - 1) / kStep;
  const int64_t k0 = steps * rank / ranks * kStep, k1 = min(k, steps * (rank + 1) / ranks * kStep);
  float acc[R][kColsPerWarp];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < kColsPerWarp; ++j) acc[r][j] = 0.0f;
  const int64_t col = c0 + warp * kColsPerWarp;
  // several steps' loads in flight; x comes from shared memory, a run at a time
  constexpr int kUnroll = VEC == 1 ? 8 : R == 1 ? 4 : 2;
  for (int64_t from = k0; from < k1; from += kRun) {
    const int run = (int)min((int64_t)kRun, k1 - from);
    __syncthreads();
    for (int i = threadIdx.x; i < R * kRun; i += kThreads) {
      const int r = i / kRun, j = i % kRun;
      xs[r][j] = r < rows && j < run ? __bfloat162float(x[r * ldx + from + j]) : 0.0f;
    }
    __syncthreads();
    for (int at = lane * VEC; at < run; at += kStep * kUnroll) {
      Raw<bf16, VEC> rw[kUnroll][kColsPerWarp];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int j = 0; j < kColsPerWarp; ++j)
          rw[u][j] = load_raw<VEC>(w + (col + j) * ldw + from + at + u * kStep,
                                   col + j < n ? run - at - u * kStep : 0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (at + u * kStep >= run) break;
        float fw[kColsPerWarp][VEC];
#pragma unroll
        for (int j = 0; j < kColsPerWarp; ++j) to_floats(rw[u][j], fw[j]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float* fx = &xs[r][at + u * kStep];
#pragma unroll
          for (int j = 0; j < kColsPerWarp; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[r][j] = fmaf(fx[i], fw[j][i], acc[r][j]);
        }
      }
    }
  }
  cluster_ready();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < kColsPerWarp; ++j) {
      const float s = warp_total(acc[r][j]);
      if (lane == 0) to_first(&sums[rank][r][warp * kColsPerWarp + j], s);
    }
  cluster_done();
  if (rank != 0) return;
  // one warp a row, one column a lane
  for (int r = warp; r < rows; r += kWarps) {
    const int64_t c = c0 + lane;
    const int left = c < n ? 1 : 0;
    float z[1] = {0.0f};
    for (uint32_t q = 0; q < ranks; ++q) z[0] += sums[q][r][lane];
    if (left && e.bias) z[0] += __bfloat162float(e.bias[c]);
    if (!left) z[0] = 0.0f;
    if (e.q)
      warp_pack<1>(z, left, e.q + r * e.ldq + c, e.scale + r * e.blocks_per_row + c / kBlock,
                   left && lane == 0, false);
    SCAPE_ACT_SWITCH(e.act, act_values<ACT>(z));
    if (left) {
      if (e.res) z[0] += __bfloat162float(e.res[r * e.ldres + c]);
      static_cast<bf16*>(e.out)[r * e.ldo + c] = __float2bfloat16_rn(z[0]);
    }
  }
}

// ------------------------------------------------------------------ input gradient
// A cluster makes kGradCols columns of dx; its blocks cut the rows of the weight
// (the contraction).  A thread takes VEC columns of every kLanes-th weight row.
constexpr int kGradCols = 64;

template <int R, int VEC>
__global__ __launch_bounds__(kThreads) void skinny_input_grad_kernel(
    const bf16* dy, int64_t lddy, const bf16* w, int64_t ldw, int rows, int64_t k, int64_t n,
    const __grid_constant__ Epilogue e) {
  constexpr int kPerRow = kGradCols / VEC;     // threads across the columns
  constexpr int kLanes = kThreads / kPerRow;   // weight rows at a time
  constexpr int kParts = VEC == 8 ? kWarps : kLanes;
  // values of dy for a run of weight rows; later the threads' partial sums
  constexpr int kRun = 512;
  __shared__ __align__(16) union {
    float g[kRun][R];
    float part[kParts][R][kGradCols];
  } sh;
  __shared__ float sums[8][R][kGradCols];
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  cluster_begin();
  start();
  const int64_t c0 = (int64_t)(blockIdx.x / ranks) * kGradCols;
  const int at = threadIdx.x % kPerRow, first = threadIdx.x / kPerRow;
  const int64_t c = c0 + at * VEC;
  const int have = (int)min((int64_t)VEC, k - c);
  const int64_t n0 = n * rank / ranks, n1 = n * (rank + 1) / ranks;
  float acc[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[r][i] = 0.0f;
  constexpr int kUnroll = 4;
  for (int64_t from = n0; from < n1; from += kRun) {
    const int run = (int)min((int64_t)kRun, n1 - from);
    __syncthreads();
    for (int i = threadIdx.x; i < kRun * R; i += kThreads) {
      const int r = i / kRun, j = i % kRun;
      sh.g[j][r] = j < run && r < rows ? __bfloat162float(dy[r * lddy + from + j]) : 0.0f;
    }
    __syncthreads();
    for (int i = first; i < run; i += kLanes * kUnroll) {
      Raw<bf16, VEC> rw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        rw[u] = load_raw<VEC>(w + (from + i + u * kLanes) * ldw + c, i + u * kLanes < run ? have : 0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (i + u * kLanes >= run) break;
        float f[VEC];
        to_floats(rw[u], f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float g = sh.g[i + u * kLanes][r];
#pragma unroll
          for (int j = 0; j < VEC; ++j) acc[r][j] = fmaf(g, f[j], acc[r][j]);
        }
      }
    }
  }
  __syncthreads();
  if constexpr (VEC == 8) {
    // a warp holds 4 weight rows of the same 64 columns
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        acc[r][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[r][j], 8);
        acc[r][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[r][j], 16);
        if ((threadIdx.x & 31) < 8) sh.part[threadIdx.x >> 5][r][at * VEC + j] = acc[r][j];
      }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < VEC; ++j) sh.part[first % kParts][r][at * VEC + j] = acc[r][j];
  }
  __syncthreads();
  cluster_ready();
  for (int i = threadIdx.x; i < rows * kGradCols; i += kThreads) {
    const int r = i / kGradCols, j = i % kGradCols;
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) s += sh.part[p][r][j];
    to_first(&sums[rank][r][j], s);
  }
  cluster_done();
  if (rank != 0) return;
  for (int i = threadIdx.x; i < rows * kGradCols; i += kThreads) {
    const int r = i / kGradCols, j = i % kGradCols;
    const int64_t o = c0 + j;
    if (o >= k) continue;
    float s = 0.0f;
    for (uint32_t q = 0; q < ranks; ++q) s += sums[q][r][j];
    if (e.act != SCAPE_ACT_NONE) {
      const uint32_t b = e.pre_q[r * e.ldpre + o];
      const float scale = scale_value(e.pre_scale[r * e.blocks_per_row + o / kBlock]);
      uint64_t lo, hi;
      e4m3_pairs(b, lo, hi);
      float slope = 1.0f, other;
      SCAPE_ACT_SWITCH(e.act, unpair(Slope<ACT>(scale).slope(lo), slope, other));
      s *= slope;
    }
    static_cast<bf16*>(e.out)[r * e.ldo + o] = __float2bfloat16_rn(s);
  }
}

// ------------------------------------------------------------------ weight gradient
// Written once, from R values a column that a thread keeps: kPerWarp rows of dW a
// warp.  The input is made from its 8-bit form here, and the blocks of the first
// columns also write the bias gradient.
constexpr int kPerWarp = 8;

template <int R, int VEC, typename T>
__global__ __launch_bounds__(kThreads) void skinny_weight_grad_kernel(
    const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const uint8_t* q, int64_t ldq,
    const uint8_t* scale, bool x16, bool q8, int act, int rows, int64_t k, int64_t n, T* dw,
    int64_t lddw, T* db) {
  start();
  // a lane's columns: VEC 8 neighbours, or 8 singles that lie 32 apart
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t across = (k + 255) / 256, down = blockIdx.x / across;
  const int64_t base = (blockIdx.x - down * across) * 256;
  auto column = [&](int i) { return VEC == 8 ? base + lane * 8 + i : base + i * 32 + lane; };
  const int64_t blocks_per_row = (k + kBlock - 1) / kBlock;
  const int have = VEC == 8 ? (int)min((int64_t)8, k - column(0)) : 0;
  float a[R][8];
  if (VEC == 8 && q && q8) {
    // 8 neighbours of one block: a word pair and a scale
    uint2 w[R];
    uint32_t code[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[r] = make_uint2(0, 0), code[r] = 1;
      if (r >= rows || have <= 0) continue;
      const uint8_t* p = q + r * ldq + column(0);
      code[r] = scale[r * blocks_per_row + column(0) / kBlock];
      if (have == 8) {
        w[r] = *reinterpret_cast<const uint2*>(p);
      } else {
        for (int i = 0; i < have; ++i) (i < 4 ? w[r].x : w[r].y) |= (uint32_t)p[i] << (8 * (i & 3));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t s = pair(scale_value(code[r]), scale_value(code[r]));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint64_t lo, hi;
        e4m3_pairs(h ? w[r].y : w[r].x, lo, hi);
        unpair(mul2(lo, s), a[r][4 * h], a[r][4 * h + 1]);
        unpair(mul2(hi, s), a[r][4 * h + 2], a[r][4 * h + 3]);
      }
    }
  } else if (VEC == 8 && x && x16) {
    Raw<bf16, 8> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = load_raw<8>(x + r * ldx + column(0), r < rows ? have : 0);
#pragma unroll
    for (int r = 0; r < R; ++r) to_floats(raw[r], a[r]);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // a row's loads first, then what they mean
      uint32_t w[8], code[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = column(i);
        w[i] = 0, code[i] = 1;
        if (r < rows && c < k) {
          if (x) {
            w[i] = reinterpret_cast<const uint16_t*>(x)[r * ldx + c];
          } else {
            w[i] = q[r * ldq + c];
            code[i] = scale[r * blocks_per_row + c / kBlock];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (x) {
          a[r][i] = __uint_as_float(w[i] << 16);
        } else {
          uint64_t lo, hi;
          e4m3_pairs(w[i], lo, hi);
          float other;
          unpair(mul2(lo, pair(scale_value(code[i]), scale_value(code[i]))), a[r][i], other);
        }
      }
    }
  }
  if (act != SCAPE_ACT_NONE) {
    // rounded to bfloat16: the forward product took it so, and the tensor cores'
    // form of this product, for more rows, has to (its error in the gradient, 2^-9 of
    // a term at most and as often up as down, is below the result's own rounding)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      SCAPE_ACT_SWITCH(act, act_values<ACT>(a[r]));
#pragma unroll
      for (int i = 0; i < 8; ++i) a[r][i] = __bfloat162float(__float2bfloat16_rn(a[r][i]));
    }
  }
  const int64_t n0 = (down * kWarps + warp) * kPerWarp;
  // lane j of the first kPerWarp holds row n0 + j of dy, one value for each of R
  float g[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    g[r] = r < rows && lane < kPerWarp && n0 + lane < n ? __bfloat162float(dy[r * lddy + n0 + lane]) : 0.0f;
  if (db && base == 0 && lane < kPerWarp && n0 + lane < n) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) s += g[r];
    db[n0 + lane] = (T)s;
  }
#pragma unroll
  for (int j = 0; j < kPerWarp; ++j) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float d = __shfl_sync(0xFFFFFFFFu, g[r], j);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(d, a[r][i], s[i]);
    }
    if (n0 + j >= n) continue;
    T* o = dw + (n0 + j) * lddw;
    if constexpr (VEC == 8) {
      store_part<8>(o + column(0), (int)min((int64_t)8, k - column(0)), s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column(i) < k) o[column(i)] = (T)s[i];
    }
  }
}

// ------------------------------------------------------------------ launch
// Blocks a cluster: as many as there are SMs for, while each has `least` or more
// of the contraction.
int cuts(int64_t clusters, int64_t contraction, int64_t least) {
  int s = 1;
  while (s < 8 && clusters * s * 2 <= 2 * sm_count() && contraction / (s * 2) >= least) s *= 2;
  return s;
}
// CALL with the rows' bound R (1 or 4) and columns a thread as constants.
#define SCAPE_ROWS_SWITCH(rows, vec, CALL)             \
  if (vec) {                                           \
    constexpr int VEC = 8;                             \
    if (rows == 1) { constexpr int R = 1; CALL; }      \
    else { constexpr int R = 4; CALL; }                \
  } else {                                             \
    constexpr int VEC = 1;                             \
    if (rows == 1) { constexpr int R = 1; CALL; }      \
    else { constexpr int R = 4; CALL; }                \
  }

template <int R, int VEC>
cudaError_t run_forward(const GemmCall& c, int64_t clusters, int s, cudaStream_t st) {
  return launch_kernel(skinny_forward_kernel<R, VEC>, (unsigned)(clusters * s), kThreads, 0, s, st, c.a.p, c.a.ld,
                       c.b.p, c.b.ld, (int)c.m, c.k, c.n, c.e);
}
template <int R, int VEC>
cudaError_t run_input_grad(const GemmCall& c, int64_t clusters, int s, cudaStream_t st) {
  return launch_kernel(skinny_input_grad_kernel<R, VEC>, (unsigned)(clusters * s), kThreads, 0, s, st, c.a.p, c.a.ld,
                       c.b.p, c.b.ld, (int)c.m, c.n, c.k, c.e);
}
template <int R, int VEC, typename T>
cudaError_t run_weight_grad(const SkinnyWeightGrad& a, cudaStream_t st) {
  const bool x16 = rows16(a.x, a.ldx, 2), q8 = rows8(a.q, a.ldq);
  const unsigned grid = (unsigned)(ceil_div(a.k, 256) * ceil_div(a.n, kWarps * kPerWarp));
  return launch_kernel(skinny_weight_grad_kernel<R, VEC, T>, grid, kThreads, 0, 0, st, a.dy, a.lddy, a.x, a.ldx, a.q,
                       a.ldq, a.scale, x16, q8, a.act, (int)a.rows, a.k, a.n, static_cast<T*>(a.dw), a.lddw,
                       static_cast<T*>(a.db));
}
template <typename T>
cudaError_t weight_grad_of(const SkinnyWeightGrad& a, cudaStream_t st) {
  const bool vec = rows16(a.dw, a.lddw, sizeof(T));
  if (a.rows > 4) return vec ? run_weight_grad<kSkinnyWeightRows, 8, T>(a, st) : run_weight_grad<kSkinnyWeightRows, 1, T>(a, st);
  cudaError_t e = cudaSuccess;
  SCAPE_ROWS_SWITCH(a.rows, vec, e = (run_weight_grad<R, VEC, T>(a, st)));
  return e;
}
static_assert(kSkinnyRows == 4, "the rows' bounds that the kernels are made for");

}  // namespace

// The weight's rows alone decide how it is read: x comes value by value into shared
// memory, dy too (one row at an odd address through 4096 x 4096: 7.5 us, and 28.6
// when its alignment counted).
cudaError_t skinny_forward(const GemmCall& c, cudaStream_t st) {
  const bool vec = rows16(c.b.p, c.b.ld, 2);
  const int64_t clusters = ceil_div(c.n, kCols);
  const int s = cuts(clusters, c.k, 512);
  cudaError_t e = cudaSuccess;
  SCAPE_ROWS_SWITCH(c.m, vec, e = (run_forward<R, VEC>(c, clusters, s, st)));
  return e;
}
cudaError_t skinny_input_grad(const GemmCall& c, cudaStream_t st) {
  const bool vec = rows16(c.b.p, c.b.ld, 2);
  const int64_t clusters = ceil_div(c.n, kGradCols);
  const int s = cuts(clusters, c.k, 128);
  cudaError_t e = cudaSuccess;
  SCAPE_ROWS_SWITCH(c.m, vec, e = (run_input_grad<R, VEC>(c, clusters, s, st)));
  return e;
}
cudaError_t skinny_weight_grad(const SkinnyWeightGrad& a, cudaStream_t st) {
  return a.out_f32 ? weight_grad_of<float>(a, st) : weight_grad_of<bf16>(a, st);
}

}  // namespace layer
}  // namespace scapek
