// layer_norm.cu -- residual RMS norm, forward (with an 8-bit output) and backward.
//
// Bound by memory: a row's inputs are read once into registers, the sum of
// squares (or of gradient products) is taken over the warps that hold the row,
// and the outputs are written from the same registers.  What stands between that
// and the copy rate is the work a row costs each thread whatever its width (the
// sum over the block, addresses), so a thread takes 16 columns and works on pairs
// (8 columns and single floats: 33 instructions a value, 13.4 us for 4096 x 1280
// with all outputs).
//
// A row of up to 1024 columns (backward 512) belongs to one warp (no block
// barrier), a wider one to a block that is as wide as the row needs; rows over
// kBlockCols are read twice by the *_wide kernels.
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
// Sum over the block, the same bits in every thread.  `red` holds 16 floats of
// this call's own: the next call uses another one, so one barrier will do.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  float s = 0.0f;
  for (int i = 0; i < warps; i += 4) {  // unused places hold 0
    const float4 r = *reinterpret_cast<const float4*>(red + i);
    s += (r.x + r.y) + (r.z + r.w);
  }
  return s;
}
// The places of warps that the block does not have; block_sum's own barrier makes
// them visible.
__device__ __forceinline__ void clear_sums(float (*red)[16]) {
  if (threadIdx.x < 32 && (threadIdx.x & 15) >= blockDim.x >> 5) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.0f;
}
// 1 / sqrt(x): the hardware's estimate and one Newton step.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return isinf(r) || r == 0.0f ? r : r * fmaf(-0.5f * x * r, r, 1.5f);
}

// A thread's NV vectors as pairs of floats: pair k holds its values 2k, 2k + 1.
template <typename T, int VEC, int NV>
__device__ __forceinline__ uint64_t raw_pair(const Raw<T, VEC> (&r)[NV], int k) {
  if constexpr (VEC == 1) {
    float a[1], b[1];
    to_floats(r[2 * k], a);
    to_floats(r[2 * k + 1], b);
    return pair(a[0], b[0]);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t w = r[2 * k / VEC].w[k % (VEC / 2)];
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    const uint32_t* w = &r[2 * k / VEC].w[2 * k % VEC];
    return pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
  }
}
template <int VEC, int NV>
__device__ __forceinline__ void load_weights(uint64_t (&w)[NV * VEC / 2], const void* p, int is_bf16,
                                             bool aligned, int t, int width, int mine) {
  float f[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    load_weight<VEC>(p, is_bf16, aligned, (i * width + t) * VEC, mine - i * width * VEC, f[i]);
#pragma unroll
  for (int k = 0; k < NV * VEC / 2; ++k)
    w[k] = pair(f[2 * k / VEC][2 * k % VEC], f[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
}
template <int VEC, int NV>
__device__ __forceinline__ void split_pairs(const uint64_t (&p)[NV * VEC / 2], float (&v)[NV][VEC]) {
#pragma unroll
  for (int k = 0; k < NV * VEC / 2; ++k)
    unpair(p[k], v[2 * k / VEC][2 * k % VEC], v[(2 * k + 1) / VEC][(2 * k + 1) % VEC]);
}
__device__ __forceinline__ float pair_sum(uint64_t p) {
  float a, b;
  unpair(p, a, b);
  return a + b;
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

// The forward pass's rows on their way into shared memory, kDepth of them ahead:
// every thread copies its own 16-byte pieces to places of its own and waits for its
// own copies, so no barrier is needed and no register holds them (8192 x 2048 with
// all outputs: 23.5 us, from registers 27.5, three rows ahead 23.8; with 16 columns a thread, rows over
// 4096, it was slower, 49 against 45 us for 4096 x 5632).
template <typename T, int VEC, int NV>
struct Ring {
  static constexpr int kVecPieces = VEC * (int)sizeof(T) / 16;
  static constexpr int kPieces = NV * kVecPieces;
  static constexpr int kDepth = 2;
  static constexpr int kBytesPerThread = kDepth * 2 * kPieces * 16;  // x and the residual
  uint32_t base, pitch;
  __device__ explicit Ring(const void* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16), pitch(blockDim.x * 16) {}
  __device__ uint32_t at(int stage, int tensor, int piece) const {
    return base + ((stage * 2 + tensor) * kPieces + piece) * pitch;
  }
  // A row of one tensor, from this thread's first column on; `mine` columns left.
  __device__ void copy(int stage, int tensor, const T* p, int step, int mine) const {
    constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVecPieces; ++j) {
        const int left = mine - i * step - j * kPer;
        const int bytes = left >= kPer ? 16 : left > 0 ? left * (int)sizeof(T) : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, tensor, i * kVecPieces + j)),
                     "l"(bytes ? p + i * step + j * kPer : p), "r"(bytes)
                     : "memory");
      }
  }
  __device__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest of kDepth rows has landed.
  __device__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory"); }
  template <typename R>
  __device__ void read(int stage, int tensor, R (&r)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVecPieces; ++j)
        asm volatile("ld.shared::cta.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[i].w[4 * j]), "=r"(r[i].w[4 * j + 1]), "=r"(r[i].w[4 * j + 2]), "=r"(r[i].w[4 * j + 3])
                     : "r"(at(stage, tensor, i * kVecPieces + j))
                     : "memory");
  }
};

// ANY: rows of x and the residual of any alignment (the outputs' are aligned).
template <typename T, int VEC, int NV, int WIDTH, bool ANY>
__global__ __launch_bounds__(Team<WIDTH>::kThreads) void norm_fwd_kernel(
    const __grid_constant__ NormFwd a, bool w_vec, float inv_cols) {
  using TM = Team<WIDTH>;
  constexpr int P = NV * VEC / 2;
  start();
  __shared__ __align__(16) float red[2][16];
  if (!TM::kWarp) clear_sums(red);
  const int t = TM::lane(), width = TM::width();
  const int blocks_per_row = (a.cols + kBlock - 1) / kBlock;
  const int mine = a.cols - t * VEC;  // columns from this thread's first on
  uint64_t w[P];
  load_weights<VEC, NV>(w, a.w, a.w_bf16, w_vec, t, width, mine);
  constexpr bool kRing = VEC == 8 && !ANY;
  using RG = Ring<T, 8, NV>;
  extern __shared__ __align__(16) uint4 ring_memory[];
  const RG ring(ring_memory);
  auto copy_row = [&](int64_t row, int stage) {
    if (row < a.rows) {
      ring.copy(stage, 0, static_cast<const T*>(a.x) + row * a.ldx + t * VEC, width * VEC, mine);
      if (a.res) ring.copy(stage, 1, static_cast<const T*>(a.res) + row * a.ldres + t * VEC, width * VEC, mine);
    }
    RG::commit();
  };
  int flip = 0, stage = 0;
  if constexpr (kRing) {
#pragma unroll
    for (int d = 0; d < RG::kDepth; ++d) copy_row(TM::first() + d * TM::step(), d);
  }
  for (int64_t row = TM::first(); row < a.rows; row += TM::step()) {
    Raw<T, VEC> rx[NV], rr[NV];
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + t * VEC;
    const T* res = static_cast<const T*>(a.res) + row * a.ldres + t * VEC;
    if constexpr (kRing) {
      RG::wait();
      ring.read(stage, 0, rx);
      if (a.res) ring.read(stage, 1, rr);
      copy_row(row + RG::kDepth * TM::step(), stage);
      if (++stage == RG::kDepth) stage = 0;
    }
#pragma unroll
    for (int i = 0; i < (kRing ? 0 : NV); ++i) {
      const int n = mine - i * width * VEC;
      if constexpr (ANY) {
        const T *x0 = static_cast<const T*>(a.x), *r0 = static_cast<const T*>(a.res);
        rx[i] = load_any<VEC>(x + i * width * VEC, n, x0, x0 + (a.rows - 1) * a.ldx + a.cols);
        if (a.res) rr[i] = load_any<VEC>(res + i * width * VEC, n, r0, r0 + (a.rows - 1) * a.ldres + a.cols);
      } else {
        rx[i] = load_raw<VEC>(x + i * width * VEC, n);
        if (a.res) rr[i] = load_raw<VEC>(res + i * width * VEC, n);
      }
    }
    uint64_t v[P], sum = pair(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      v[k] = raw_pair(rx, k);
      if (a.res) v[k] = add2(v[k], raw_pair(rr, k));
      sum = fma2(v[k], v[k], sum);
    }
    float ss = pair_sum(sum);
    ss = TM::kWarp ? warp_sum(ss) : block_sum(ss, red[flip]);
    flip ^= 1;
    const float rstd = inverse_root(fmaf(ss, inv_cols, a.eps));
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    float f[NV][VEC];
    if (a.h) {
      T* h = static_cast<T*>(a.h) + row * a.ldh + t * VEC;
      split_pairs<VEC, NV>(v, f);
#pragma unroll
      for (int i = 0; i < NV; ++i) store_part<VEC>(h + i * width * VEC, mine - i * width * VEC, f[i]);
    }
#pragma unroll
    for (int k = 0; k < P; ++k) v[k] = mul2(mul2(v[k], pair(rstd, rstd)), w[k]);
    split_pairs<VEC, NV>(v, f);
    T* y = static_cast<T*>(a.y) + row * a.ldy + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) store_part<VEC>(y + i * width * VEC, mine - i * width * VEC, f[i]);
    if (a.q) {
      uint8_t* q = a.q + row * a.ldq + t * VEC;
      uint8_t* scale = a.scale + row * blocks_per_row + t * VEC / kBlock;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = mine - i * width * VEC;
        warp_pack<VEC>(f[i], n, q + i * width * VEC, scale + i * width * VEC / kBlock,
                       n > 0 && t * VEC % kBlock == 0, a.q16);
      }
    }
  }
}

// Any width: the row is read a second time (from the caches) for the outputs.
template <typename T>
__global__ __launch_bounds__(512) void norm_fwd_wide_kernel(NormFwd a) {
  start();
  __shared__ __align__(16) float red[2][16];
  clear_sums(red);
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
    const float rstd = inverse_root(ss / (float)a.cols + a.eps);
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
                     n > 0 && c % kBlock == 0, false);
    }
  }
}

// A thread keeps its columns' weight gradients in registers over all its rows;
// one row of partial sums a block goes to a.partial, added up by sum_partials.
// The next row's loads are in flight while this one is summed over the block (in
// registers: a ring of shared memory as the forward pass has was slower here,
// 8192 x 2048 in 32.2 against 30.1 us).
template <typename T, int VEC, int NV, int WIDTH>
__global__ __launch_bounds__(Team<WIDTH>::kThreads, (VEC == 8 && sizeof(T) == 2 && NV == 1 ? 1024 : 512) / Team<WIDTH>::kThreads) void norm_bwd_kernel(
    const __grid_constant__ NormBwd a, bool w_vec, float inv_cols) {
  using TM = Team<WIDTH>;
  constexpr int P = NV * VEC / 2;
  start();
  __shared__ __align__(16) float red[2][16];
  __shared__ float cross[TM::kWarp ? kWarpRows * kWarpColsBwd : 1];
  if (!TM::kWarp) clear_sums(red);
  const int t = TM::lane(), width = TM::width();
  const int mine = a.cols - t * VEC;
  uint64_t acc[P], w[P];
  load_weights<VEC, NV>(w, a.w, a.w_bf16, w_vec, t, width, mine);
#pragma unroll
  for (int k = 0; k < P; ++k) acc[k] = pair(0.0f, 0.0f);
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
      if (a.dh) rd[i] = load_raw<VEC>(dh + i * width * VEC, n);
    }
  };
  int flip = 0;
  int64_t row = TM::first();
  if (row < a.rows) load_row(row);
  while (row < a.rows) {
    const uint64_t r2 = pair(rstd, rstd);
    uint64_t g[P], n[P], sum = pair(0.0f, 0.0f);
    Raw<T, VEC> d[NV];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      g[k] = raw_pair(rg, k);
      n[k] = mul2(raw_pair(rn, k), r2);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = rd[i];
    const int64_t next = row + TM::step();
    if (next < a.rows) load_row(next);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      acc[k] = fma2(g[k], n[k], acc[k]);
      g[k] = mul2(g[k], w[k]);
      sum = fma2(g[k], n[k], sum);
    }
    float s = pair_sum(sum);
    s = TM::kWarp ? warp_sum(s) : block_sum(s, red[flip]);
    flip ^= 1;
    const uint64_t mean = pair(-s * inv_cols, -s * inv_cols);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      g[k] = fma2(n[k], mean, g[k]);
      g[k] = a.dh ? fma2(g[k], r2, raw_pair(d, k)) : mul2(g[k], r2);
    }
    float f[NV][VEC];
    split_pairs<VEC, NV>(g, f);
    T* dx = static_cast<T*>(a.dx) + row * a.lddx + t * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) store_part<VEC>(dx + i * width * VEC, mine - i * width * VEC, f[i]);
    row = next;
  }
  if (!a.dw) return;
  float f[NV][VEC];
  split_pairs<VEC, NV>(acc, f);
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (TM::kWarp) {
    // the block's warps hold the same columns: add them up in warp order
    float* own = cross + (threadIdx.x >> 5) * kWarpColsBwd;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) own[(i * 32 + t) * VEC + j] = f[i][j];
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
        if (i * width * VEC + j < mine) out[(i * width + t) * VEC + j] = f[i][j];
    }
  }
}

template <typename T>
__global__ __launch_bounds__(512) void norm_bwd_wide_kernel(NormBwd a) {
  start();
  __shared__ __align__(16) float red[2][16];
  clear_sums(red);
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
  start();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
    s += (float)static_cast<const T*>(a.dy)[row * a.lddy + c] *
         ((float)static_cast<const T*>(a.h)[row * a.ldh + c] * a.rstd[row]);
  a.partial[(int64_t)blockIdx.y * a.cols + c] = s;
}

constexpr int kColsumThreads = 512;
template <bool ANY>
__global__ __launch_bounds__(kColsumThreads) void colsum_kernel(const __grid_constant__ ColumnSums a) {
  cluster_begin();
  start();
  sum_columns<kColsumThreads, ANY>(a);
}

// Sums of partial[parts, cols]: 32 columns a cluster, each of its blocks' warps
// taking every 16th of its rows; the blocks' parts meet in the first one's shared
// memory.  (One block of 1024 threads for 32 columns took 9 us for 1216 rows of
// 256 columns: the rows of one block come through one SM.)
constexpr int kPartBlocks = 8;
constexpr int kPartWarps = 16;
__global__ __launch_bounds__(32 * kPartWarps) void sum_partials_kernel(
    const float* partial, int64_t parts, int64_t cols, void* out, int out_bf16) {
  __shared__ float part[kPartWarps][33];
  __shared__ float sums[kPartBlocks][32];
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  cluster_begin();
  start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)(blockIdx.x / ranks) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
    constexpr int kUnroll = 8;
    const int kStep = ranks * kPartWarps;
    for (int64_t p = rank * kPartWarps + warp; p < parts; p += kStep * kUnroll) {
      float v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        v[u] = p + u * kStep < parts ? partial[(p + u * kStep) * cols + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) s += v[u];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  cluster_ready();
  if (warp == 0) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kPartWarps; ++k) t += part[k][lane];
    to_first(&sums[rank][lane], t);
  }
  cluster_done();
  if (rank == 0 && warp == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kPartBlocks; ++k)
      if (k < ranks) t += sums[k][lane];
    if (out_bf16)
      static_cast<bf16*>(out)[c] = __float2bfloat16_rn(t);
    else
      static_cast<float*>(out)[c] = t;
  }
}

// Launch shape of a row kernel: warps own rows up to warp_cols, blocks above, as
// wide as the row at 8 columns a thread (16 past 4096).  Single columns (rows of
// any alignment) need a width known to the compiler, so that a thread's
// addresses are one register and constants (777 x 1283 float32 with the 8-bit
// output: 10.8 us with the width in a register, 6.0 without).
struct Shape {
  int per;    // columns a thread
  int width;  // threads a row; 0: the block's
  int threads;
  unsigned grid;
};
Shape shape_of(int64_t rows, int64_t cols, bool vec, int warp_cols, int threads_per_sm) {
  Shape s;
  if (cols <= warp_cols) {
    s.per = cols <= 256 ? 8 : cols <= 512 ? 16 : 32;
    s.width = 32;
    s.threads = 32 * kWarpRows;
  } else {
    s.per = !vec || cols > 4096 ? 16 : 8;
    s.threads = vec ? (int)(ceil_div(ceil_div(cols, s.per), 32) * 32)
                    : cols <= 1024 ? 64 : cols <= 2048 ? 128 : cols <= 4096 ? 256 : 512;
    s.width = vec ? 0 : s.threads;
  }
  const int64_t rows_per_block = s.width == 32 ? kWarpRows : 1;
  s.grid = (unsigned)std::min(ceil_div(rows, rows_per_block),
                              (int64_t)sm_count() * std::max(1, threads_per_sm / s.threads));
  return s;
}

// Runs CALL with VEC, NV and WIDTH as constants for a shape (rows of up to
// WARP_COLS columns belong to a warp).
#define SCAPE_SHAPE_SWITCH(vec, s, WARP_COLS, CALL)                                      \
  if (vec) {                                                                             \
    if (s.width == 0 && s.per == 8) { constexpr int VEC = 8, WIDTH = 0, NV = 1; CALL; }  \
    else if (s.width == 0) { constexpr int VEC = 16, WIDTH = 0, NV = 1; CALL; }          \
    else if (s.per == 8) { constexpr int VEC = 8, WIDTH = 32, NV = 1; CALL; }            \
    else if (s.per == 16) { constexpr int VEC = 8, WIDTH = 32, NV = 2; CALL; }           \
    else { constexpr int VEC = 8, WIDTH = 32, NV = WARP_COLS / 256; CALL; }              \
  } else {                                                                               \
    constexpr int VEC = 1;                                                               \
    if (s.width == 32 && s.per == 8) { constexpr int WIDTH = 32, NV = 8; CALL; }         \
    else if (s.width == 32 && s.per == 16) { constexpr int WIDTH = 32, NV = 16; CALL; }  \
    else if (s.width == 32) { constexpr int WIDTH = 32, NV = WARP_COLS / 32; CALL; }     \
    else if (s.width == 64) { constexpr int WIDTH = 64, NV = 16; CALL; }                 \
    else if (s.width == 128) { constexpr int WIDTH = 128, NV = 16; CALL; }               \
    else if (s.width == 256) { constexpr int WIDTH = 256, NV = 16; CALL; }               \
    else { constexpr int WIDTH = 512, NV = 16; CALL; }                                   \
  }

template <typename T, int VEC, int NV>
constexpr size_t ring_bytes(int threads) {
  return VEC == 8 ? (size_t)Ring<T, 8, NV>::kBytesPerThread * threads : 0;
}
// Launches a row kernel with its ring of shared memory.
template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), const Shape& s, size_t smem, cudaStream_t st, const A&... args) {
  if (smem > 32 * 1024) {  // with the static part, what a kernel may have unasked is 48 KB
    const cudaError_t e = allow_smem((const void*)kernel, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, s.grid, s.threads, smem, 0, st, args...);
}

// Threads an SM that the grids are made for.  Backward: all that fit at once, as
// blocks keep their weight gradients to the end.  Forward: about two rounds, so
// that blocks that end early make room (one round 28.8 us, two 27.8, sixteen 28.7
// for 8192 x 2048 with all outputs).
constexpr int kFwdThreads = 2048;
template <typename T>
constexpr int bwd_threads() { return sizeof(T) == 2 ? 1024 : 512; }

template <typename T>
cudaError_t run_norm_fwd(NormFwd a, cudaStream_t st) {
  if (a.cols > kBlockCols) {
    return launch_kernel(norm_fwd_wide_kernel<T>, (unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * 4),
                         512, 0, 0, st, a);
  }
  const size_t e = sizeof(T);
  const bool vec = rows16(a.y, a.ldy, e) && rows16(a.h, a.ldh, e) && rows8(a.q, a.ldq);
  const bool any = !rows16(a.x, a.ldx, e) || !rows16(a.res, a.ldres, e);
  a.q16 = rows16(a.q, a.ldq, 1);
  const bool wv = aligned(a.w, 16);
  const float inv = (float)(1.0 / a.cols);
  const Shape s = shape_of(a.rows, a.cols, vec, kWarpCols, kFwdThreads);
  cudaError_t err = cudaSuccess;
  if (any) {
    SCAPE_SHAPE_SWITCH(vec, s, kWarpCols, err = (launch_rows(norm_fwd_kernel<T, VEC, NV, WIDTH, (VEC > 1)>, s, 0,
                                                             st, a, wv, inv)));
  } else {
    SCAPE_SHAPE_SWITCH(vec, s, kWarpCols, err = (launch_rows(norm_fwd_kernel<T, VEC, NV, WIDTH, false>, s,
                                                             ring_bytes<T, VEC, NV>(s.threads), st, a, wv, inv)));
  }
  return err;
}

template <typename T>
cudaError_t run_norm_bwd(const NormBwd& a, cudaStream_t st) {
  int64_t parts = norm_bwd_partials(a.rows, a.cols);
  cudaError_t err = cudaSuccess;
  if (a.cols > kBlockCols) {
    if (a.dw)
      err = launch_kernel(norm_dw_wide_kernel<T>, dim3((unsigned)ceil_div(a.cols, 256), (unsigned)parts), 256, 0,
                          0, st, a);
    if (err == cudaSuccess)
      err = launch_kernel(norm_bwd_wide_kernel<T>, (unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * 4),
                          512, 0, 0, st, a);
  } else {
    const size_t e = sizeof(T);
    const bool vec = rows16(a.dy, a.lddy, e) && rows16(a.h, a.ldh, e) &&
                     rows16(a.dh, a.lddh, e) && rows16(a.dx, a.lddx, e);
    const bool wv = aligned(a.w, 16);
    const float inv = (float)(1.0 / a.cols);
    const Shape s = shape_of(a.rows, a.cols, vec, kWarpColsBwd, vec && a.cols <= 4096 ? bwd_threads<T>() : 512);
    SCAPE_SHAPE_SWITCH(vec, s, kWarpColsBwd, err = (launch_rows(norm_bwd_kernel<T, VEC, NV, WIDTH>, s,
                                                                0, st, a, wv, inv)));
    parts = s.grid;
  }
  if (err != cudaSuccess || !a.dw) return err;
  return launch_sum_partials(a.partial, parts, a.cols, a.dw, a.dw_bf16, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_norm_fwd<bf16>(a, st) : run_norm_fwd<float>(a, st);
}
int64_t norm_bwd_partials(int64_t rows, int64_t cols) {
  if (cols > kBlockCols) return std::min<int64_t>(ceil_div(rows, 8), 64);
  return std::max(shape_of(rows, cols, true, kWarpColsBwd, 1024).grid,
                  shape_of(rows, cols, false, kWarpColsBwd, 512).grid);
}
cudaError_t launch_norm_bwd(const NormBwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_norm_bwd<bf16>(a, st) : run_norm_bwd<float>(a, st);
}

cudaError_t launch_colsum(const ColumnSums& a, cudaStream_t st) {
  const int blocks = sum_cluster(a.rows);
  return launch_kernel(rows16(a.m, a.ld, 2) ? colsum_kernel<false> : colsum_kernel<true>,
                       (unsigned)(ceil_div(a.cols, kSumCols) * blocks), kColsumThreads, 0, blocks, st, a);
}
cudaError_t launch_sum_partials(const float* partial, int64_t parts, int64_t cols, void* out,
                                int out_bf16, cudaStream_t st) {
  const int blocks = parts <= 128 ? 1 : kPartBlocks;  // as in sum_cluster()
  return launch_kernel(sum_partials_kernel, (unsigned)(ceil_div(cols, 32) * blocks), 32 * kPartWarps, 0, blocks,
                       st, partial, parts, cols, out, out_bf16);
}

}  // namespace layer
}  // namespace scapek
