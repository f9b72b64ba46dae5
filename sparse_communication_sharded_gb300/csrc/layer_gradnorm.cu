// layer_gradnorm.cu -- the norm of a set of tensors, and their clipping.
//
// Bound by memory: every element is read once for the norm, and read again and
// written once for the clipping.  The tensors' places come as kernel arguments, so a
// call needs no copy of a table and can be captured.  They are cut into chunks of
// kChunk pieces of 16 bytes; a block takes a run of chunks, finds the first one's
// tensor by halving, and leaves one 64-bit sum.
//
// A chunk's squares are added up in 32 bits a thread, a few dozen at a time, and
// those sums in 64.  Where such a sum is below 2^-80 or above 2^100 (or not a number)
// squares may have left float32's range: it is formed again from elements scaled by a
// power of two.  What a small element adds to a sum in between, its square rounds to
// nothing beside it anyway.
//
// 570 M elements of bfloat16 in 219 tensors: 175 us, 96% of the copy rate, and 5 for
// the launch that adds up the blocks' sums; 355 M of float32 clipped into bfloat16: 211
// and 321, 98%.  Four blocks of 256 threads an SM (three: norm 183 -> 209; sixteen, of
// which four run at a time: 185).
#include <algorithm>

#include "layer_tokens.h"

namespace scapek {
namespace layer {
namespace {

constexpr int kThreads = 256, kUnroll = 4, kChunk = kThreads * kUnroll;
constexpr int kBlocksPerSm = 4;

// Tensors of one launch.  A short table is a shorter launch.
constexpr int kShort = 48, kLong = 768;
template <int N>
struct Table {
  int n, chunks;
  int first[N];  // a tensor's first chunk
  int64_t numel[N];
  const void* in[N];
  void* out[N];
  uint8_t in_bf16[N], out_bf16[N];
};
static_assert(sizeof(Table<kLong>) < 32000, "kernel arguments end at 32764 bytes");

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int chunk) {
  int lo = 0, hi = t.n;  // first[lo] <= chunk, and < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// A piece on a 16-byte boundary, zeros from `left` elements on.
template <typename T>
__device__ __forceinline__ Raw<T, 16 / sizeof(T)> load_piece(const T* p, int64_t left) {
  constexpr int kPer = 16 / (int)sizeof(T);
  Raw<T, kPer> r;
  if (left >= kPer) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[k] = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (k < left) {
        if constexpr (sizeof(T) == 2)
          r.w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << (16 * (k % 2));
        else
          r.w[k] = reinterpret_cast<const uint32_t*>(p)[k];
      }
  }
  return r;
}

// Sum over the block, the same bits in every thread.
__device__ __forceinline__ double block_sum64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
  return s;
}

// ------------------------------------------------------------------ squares
struct Squares {
  double sum = 0.0;
  float recent = 0.0f;
  int batches = 0;

  template <typename T, int U>
  __device__ __forceinline__ static float of(const Raw<T, 16 / sizeof(T)> (&r)[U], float scale) {
    constexpr int kPer = 16 / (int)sizeof(T);
    const uint64_t s2 = pair(scale, scale);
    uint64_t t = pair(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[kPer];
      to_floats(r[u], f);
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const uint64_t v = mul2(pair(f[k], f[k + 1]), s2);
        t = fma2(v, v, t);
      }
    }
    float a, b;
    unpair(t, a, b);
    return a + b;
  }
  template <typename T, int U>
  __device__ __forceinline__ void add(const Raw<T, 16 / sizeof(T)> (&r)[U]) {
    const float t = of<T, U>(r, 1.0f);
    if (t >= 0x1p-80f && t <= 0x1p100f) {
      recent += t;
      if (++batches == 8) sum += (double)recent, recent = 0.0f, batches = 0;
      return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) any |= r[u].w[k];
    if ((any & (sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) == 0) return;
    if (t < 0x1p-80f)
      sum += (double)of<T, U>(r, 0x1p100f) * 0x1p-200;
    else
      sum += (double)of<T, U>(r, 0x1p-70f) * 0x1p140;
  }
};

template <typename T>
__device__ __forceinline__ void chunk_squares(Squares& s, const T* p, int64_t numel, int64_t chunk) {
  constexpr int kPer = 16 / (int)sizeof(T);
  const int phase = phase_of(p);
  Raw<T, kPer> r[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = (chunk * kChunk + u * kThreads + threadIdx.x) * kPer - phase;
    if (c >= 0) {
      r[u] = load_piece(p + c, numel - c);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[u].w[k] = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < numel) {
          if constexpr (sizeof(T) == 2)
            r[u].w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[c + k] << (16 * (k % 2));
          else
            r[u].w[k] = reinterpret_cast<const uint32_t*>(p)[c + k];
        }
    }
  }
  s.add<T, kUnroll>(r);
}

template <int N>
__global__ __launch_bounds__(kThreads) void squares_kernel(const __grid_constant__ Table<N> t, double* partial) {
  start();
  __shared__ double red[kThreads / 32];
  const int begin = (int)((int64_t)t.chunks * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
  Squares s;
  int i = tensor_of(t, begin);
  for (int c = begin; c < end; ++c) {
    while (i + 1 < t.n && t.first[i + 1] <= c) ++i;
    if (t.in_bf16[i])
      chunk_squares(s, static_cast<const bf16*>(t.in[i]), t.numel[i], c - t.first[i]);
    else
      chunk_squares(s, static_cast<const float*>(t.in[i]), t.numel[i], c - t.first[i]);
  }
  const double v = block_sum64(s.sum + (double)s.recent, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The norm from all blocks' sums, the same bits in every block.
__device__ __forceinline__ double norm_of(const double* partial, int parts, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += partial[i];
  return sqrt(block_sum64(v, red));
}
__global__ __launch_bounds__(kThreads) void norm_kernel(const double* partial, int parts, float* norm) {
  start();
  __shared__ double red[kThreads / 32];
  const double n = norm_of(partial, parts, red);
  if (threadIdx.x == 0) *norm = (float)n;
}

// ------------------------------------------------------------------ clipping
// Pieces of 8 elements on the output's boundaries, U of a thread's kUnroll at a time.
// ANY: they are on no boundary of the input.
template <bool ANY, int U, typename TI, typename TO>
__device__ __forceinline__ void chunk_scale(const TI* p, TO* o, int64_t numel, int64_t chunk, float factor) {
  const int phase = phase_of(o) % (16 / (int)sizeof(TO));
#pragma unroll 1
  for (int u0 = 0; u0 < kUnroll; u0 += U) {
    const int64_t first = (chunk * kChunk + u0 * kThreads + threadIdx.x) * 8 - phase;
    Raw<TI, 8> r[U];
    AnyLoad<TI, 8> any[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = first + u * kThreads * 8;
      const int n = c >= 0 ? (int)max((int64_t)0, min((int64_t)8, numel - c)) : 0;
      if constexpr (ANY)
        any[u].begin(p + c, n, p, p + numel);
      else
        r[u] = load_raw<8>(p + c, n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = first + u * kThreads * 8;
      const int n = c >= 0 ? (int)max((int64_t)0, min((int64_t)8, numel - c)) : 0;
      if constexpr (ANY) r[u] = any[u].end(p + c, n);
      float f[8];
      to_floats(r[u], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= factor;
      store_part<8>(o + c, n, f);
      if (c < 0) {
        // a tensor's first elements, at the end of the piece
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k >= 0 && c + k < numel) o[c + k] = (TO)((float)p[c + k] * factor);
      }
    }
  }
}
// Whether pieces on the output's boundaries are on 16 bytes of the input.
inline bool same_boundaries(const void* in, bool in_bf16, const void* out, bool out_bf16) {
  const int out_elem = out_bf16 ? 2 : 4, in_elem = in_bf16 ? 2 : 4;
  const int phase = (int)(reinterpret_cast<uintptr_t>(out) & 15u) / out_elem;
  return (reinterpret_cast<uintptr_t>(in) - (uintptr_t)(phase * in_elem)) % 16 == 0;
}

// ANY: some tensor's pieces are on no boundaries of the input (a kernel of its own, as
// its loads take twice the registers).
template <int N, bool ANY>
__global__ __launch_bounds__(kThreads, kBlocksPerSm) void clip_kernel(const __grid_constant__ Table<N> t,
                                                                      const double* partial, int parts,
                                                                      float max_norm, float eps, float* norm,
                                                                      bool in_place) {
  start();
  __shared__ double red[kThreads / 32];
  const double n = norm_of(partial, parts, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  const double q = (double)max_norm / (n + (double)eps);
  const float factor = q >= 1.0 ? 1.0f : (float)q;  // NaN stays
  if (in_place && factor == 1.0f) return;  // one of itself is itself
  const int begin = (int)((int64_t)t.chunks * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
  int i = tensor_of(t, begin);
  for (int c = begin; c < end; ++c) {
    while (i + 1 < t.n && t.first[i + 1] <= c) ++i;
    const int64_t m = t.numel[i], k = c - t.first[i];
    if (t.in_bf16[i]) {
      const bf16* p = static_cast<const bf16*>(t.in[i]);
      if (t.out_bf16[i])
        chunk_scale<ANY, ANY ? 1 : kUnroll>(p, static_cast<bf16*>(t.out[i]), m, k, factor);
      else
        chunk_scale<ANY, ANY ? 1 : kUnroll>(p, static_cast<float*>(t.out[i]), m, k, factor);
    } else {
      const float* p = static_cast<const float*>(t.in[i]);
      if (t.out_bf16[i])
        chunk_scale<ANY, ANY ? 1 : kUnroll>(p, static_cast<bf16*>(t.out[i]), m, k, factor);
      else
        chunk_scale<ANY, ANY ? 1 : kUnroll>(p, static_cast<float*>(t.out[i]), m, k, factor);
    }
  }
}

// ------------------------------------------------------------------ launches
// Pieces of a tensor, with room for one that starts before it.
int64_t chunks_of(int64_t numel, int per) { return ceil_div(ceil_div(numel + 7, per), kChunk); }
int grid_of(int64_t chunks) { return (int)std::min<int64_t>(chunks, (int64_t)sm_count() * kBlocksPerSm); }

// Calls use(table) for runs of the set's tensors that fit one, skipping empty ones.
template <int N, typename F>
cudaError_t in_tables(const GradSet& a, bool scaling, F&& use) {
  Table<N> t;
  t.n = t.chunks = 0;
  for (int i = 0; i < a.n; ++i) {
    if (a.numel[i] > 0) {
      const bool in16 = a.dtype[i] == SCAPE_BF16;
      const int64_t c = chunks_of(a.numel[i], scaling || in16 ? 8 : 4);
      if (c > 0x3FFFFFFF) return cudaErrorInvalidValue;
      if (t.n == N || (int64_t)t.chunks + c > 0x7FFFFFFF) {
        const cudaError_t e = use(t);
        if (e != cudaSuccess) return e;
        t.n = t.chunks = 0;
      }
      t.first[t.n] = t.chunks;
      t.numel[t.n] = a.numel[i];
      t.in[t.n] = a.grads[i];
      t.in_bf16[t.n] = in16;
      t.out[t.n] = a.out ? a.out[i] : nullptr;
      t.out_bf16[t.n] = a.out && a.out_dtype[i] == SCAPE_BF16;
      t.chunks += (int)c;
      ++t.n;
    }
  }
  return t.n ? use(t) : cudaSuccess;
}

template <int N>
cudaError_t run_grad_norm(const GradSet& a, cudaStream_t st) {
  int parts = 0;
  cudaError_t e = in_tables<N>(a, false, [&](const Table<N>& t) {
    const int grid = grid_of(t.chunks);
    if (parts + grid > a.partials) return cudaErrorInvalidValue;
    const cudaError_t r = launch_kernel(squares_kernel<N>, (unsigned)grid, kThreads, 0, 0, st, t, a.partial + parts);
    parts += grid;
    return r;
  });
  if (e != cudaSuccess) return e;
  if (!a.out) return launch_kernel(norm_kernel, 1u, kThreads, 0, 0, st, (const double*)a.partial, parts, a.norm);
  float* norm = a.norm;
  return in_tables<N>(a, true, [&](const Table<N>& t) {
    bool same = true, in_place = true;
    for (int i = 0; i < t.n; ++i) in_place &= t.in[i] == t.out[i];
    for (int i = 0; i < t.n; ++i) same &= same_boundaries(t.in[i], t.in_bf16[i], t.out[i], t.out_bf16[i]);
    auto* const kernel = same ? clip_kernel<N, false> : clip_kernel<N, true>;
    const cudaError_t r = launch_kernel(kernel, (unsigned)grid_of(t.chunks), kThreads, 0, 0, st, t,
                                        (const double*)a.partial, parts, a.max_norm, a.eps, norm, in_place);
    norm = nullptr;  // told once
    return r;
  });
}

}  // namespace

// Blocks of all launches: a table is full with kLong tensors, or once it has more than
// 2^30 chunks and the next tensor's no longer fit (kShort tables: one is enough).
int64_t grad_norm_partials(int n, const int64_t* numel) {
  int64_t chunks = 0, some = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0) chunks += chunks_of(numel[i], 4), ++some;
  const int64_t tables = ceil_div(some, kLong) + (chunks >> 30);
  return std::min<int64_t>(chunks, tables * sm_count() * kBlocksPerSm);
}
cudaError_t launch_grad_norm(const GradSet& a, cudaStream_t st) {
  int64_t some = 0;
  for (int i = 0; i < a.n; ++i) some += a.numel[i] > 0;
  if (some == 0) return cudaMemsetAsync(a.norm, 0, sizeof(float), st);
  return some <= kShort ? run_grad_norm<kShort>(a, st) : run_grad_norm<kLong>(a, st);
}

}  // namespace layer
}  // namespace scapek
