// layer_logprobs.cu -- log probabilities of given tokens, entropy and alternatives
// of rows of logits, their gradient, and a loss that takes its gradient along.
//
// With m a row's largest logit and d = x - m: S = sum exp d, lse = m + ln S,
// entropy = ln S - (sum exp(d) d) / S.  A thread keeps m, S and the entropy's sum of
// its own pieces (16 bytes at the row's 16-byte boundaries) while it reads them, once;
// a larger m scales S by exp(m - m'), and the threads' sums are joined the same way.
// Exponents are of base 2: a = d log2 e.
#include <algorithm>
#include <type_traits>

#include "layer_tokens.h"

namespace scapek {
namespace layer {
namespace {

constexpr float kLog2eF = 1.44269504f, kLn2F = 0.693147181f;
constexpr float kLowest = -3.402823466e38f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ int64_t load_target(const Tokens& t, int64_t i) {
  return t.bytes == 8 ? static_cast<const int64_t*>(t.p)[i] : (int64_t)static_cast<const int32_t*>(t.p)[i];
}
template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  return (float)*p;
}

// A row (of any alignment) as pieces of 16 bytes at 16-byte boundaries: piece v holds
// columns v kPer - phase and on; the first and the last may be part of one.
template <typename T>
struct RowPieces {
  static constexpr int kPer = 16 / (int)sizeof(T);
  const T* x;
  int phase, cols, pieces;
  __device__ RowPieces(const T* row, int cols_)
      : x(row), phase((int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T))), cols(cols_) {
    pieces = (int)(((int64_t)phase + cols + kPer - 1) / kPer);
  }
  __device__ int column(int v) const { return v * kPer - phase; }
  __device__ bool whole(int v) const { return column(v) >= 0 && column(v) + kPer <= cols; }
  __device__ uint4 load_whole(int v) const { return *reinterpret_cast<const uint4*>(x + column(v)); }
  // Columns outside the row are -infinity.
  __device__ uint4 load_part(int v) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    const int c = column(v);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (c + i >= 0 && c + i < cols) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t e = reinterpret_cast<const uint16_t*>(x)[c + i];
          w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | (e << 16) : (w[i / 2] & 0xFFFF0000u) | e;
        } else {
          w[i] = reinterpret_cast<const uint32_t*>(x)[c + i];
        }
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ uint4 load(int v) const { return whole(v) ? load_whole(v) : load_part(v); }
};
template <typename T>
__device__ __forceinline__ uint4 minus_infinity() {
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}
// A piece's values as pairs of floats.
template <typename T>
__device__ __forceinline__ void piece_pairs(const uint4& u, uint64_t (&p)[8 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    p[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
    p[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}
// The largest of a piece's values that are not NaN (-infinity if all are).
template <typename T>
__device__ __forceinline__ float piece_top(const uint4& u) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    __nv_bfloat162 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    const __nv_bfloat162 m = __hmax2(__hmax2(t[0], t[1]), __hmax2(t[2], t[3]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
}

// ------------------------------------------------------------------ sums of a row
template <bool ENT>
struct Sums {
  float m = kLowest, s = 0.0f, a = 0.0f;  // a: sum of exp(d) times d log2 e

  // A larger m.  The exponent is limited, so that 0 sums stay 0.
  __device__ __forceinline__ void raise(float top) {
    const float e = fmaxf((m - top) * kLog2eF, -1e4f), f = exp2_fast(e);
    if (ENT) a = f * fmaf(e, s, a);
    s *= f;
    m = top;
  }
  // A few pieces' values.
  template <typename T, int U>
  __device__ __forceinline__ void add(const uint4 (&u)[U]) {
    float top = piece_top<T>(u[0]);
#pragma unroll
    for (int i = 1; i < U; ++i) top = fmaxf(top, piece_top<T>(u[i]));
    if (top > m) raise(top);
    const uint64_t minus = pair(-m, -m), log2e = pair(kLog2eF, kLog2eF);
    uint64_t s2 = pair(s, 0.0f), a2 = pair(a, 0.0f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      uint64_t p[8 / sizeof(T)];
      piece_pairs<T>(u[i], p);
#pragma unroll
      for (int k = 0; k < 8 / (int)sizeof(T); ++k) {
        const uint64_t e = mul2(add2(p[k], minus), log2e);
        float x, y;
        unpair(e, x, y);
        const uint64_t f = pair(exp2_fast(x), exp2_fast(y));
        s2 = add2(s2, f);
        // where 2^e is 0 its product with an infinite e would be NaN
        if (ENT) a2 = fma2(f, pair(fmaxf(x, -1e4f), fmaxf(y, -1e4f)), a2);
      }
    }
    float x, y;
    unpair(s2, x, y);
    s = x + y;
    if (ENT) {
      unpair(a2, x, y);
      a = x + y;
    }
  }
  // Of the warp, the same bits in every lane.
  __device__ __forceinline__ void over_warp() {
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    raise(top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(kAll, s, o);
      if (ENT) a += __shfl_xor_sync(kAll, a, o);
    }
  }
};
// The same where they are stored.
struct Part {
  float m, s, a;
};
// The sum of n parts, in their order.
template <bool ENT>
__device__ __forceinline__ Sums<ENT> join_parts(const Part* part, int n) {
  float top = part[0].m;
  for (int i = 1; i < n; ++i) top = fmaxf(top, part[i].m);
  Sums<ENT> r;
  r.m = top;
  for (int i = 0; i < n; ++i) {
    Sums<ENT> p;
    p.m = part[i].m, p.s = part[i].s, p.a = part[i].a;
    p.raise(top);
    r.s += p.s;
    if (ENT) r.a += p.a;
  }
  return r;
}
// Stores to rank's copy of a place in shared memory.
__device__ __forceinline__ uint32_t place_in(const void* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  return a;
}
template <bool ENT>
__device__ __forceinline__ void send(const Part* place, uint32_t rank, const Sums<ENT>& v) {
  const uint32_t a = place_in(place, rank);
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v.m) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(v.s) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(v.a) : "memory");
}
__device__ __forceinline__ void send(const uint64_t* place, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(place_in(place, rank)), "l"(v) : "memory");
}

// ------------------------------------------------------------------ alternatives
// A logit and its column as one number: larger logits first, of equal ones (0 and -0
// are) the lower column; NaN last.  0 is no logit at all.
__device__ __forceinline__ uint64_t key_of(float x, int col) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t o = x != x ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
  return (uint64_t)o << 32 | (0xFFFFFFFFu - (uint32_t)col);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o == 0 ? 0x7FC00000u : o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t max_over_warp(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t n = __shfl_xor_sync(kAll, k, o);
    k = n > k ? n : k;
  }
  return k;
}
template <typename T, typename F>
__device__ __forceinline__ void for_values(const RowPieces<T>& row, int v, F&& f) {
  constexpr int kPer = RowPieces<T>::kPer;
  uint64_t p[8 / sizeof(T)];
  piece_pairs<T>(row.load(v), p);
  const int c = row.column(v);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) {
    float x, y;
    unpair(p[k], x, y);
    if (c + 2 * k >= 0 && c + 2 * k < row.cols) f(x, c + 2 * k);
    if (c + 2 * k + 1 >= 0 && c + 2 * k + 1 < row.cols) f(y, c + 2 * k + 1);
  }
}

constexpr int kThreads = 256, kUnroll = 4, kMaxCluster = 8;
constexpr int kCandidates = 512;  // keys that pass the bound, before they are ranked

struct TopScratch {
  float group[32];
  uint64_t keys[kCandidates];
  uint64_t best[SCAPE_TOP_MAX];
  uint64_t of_warp[kThreads / 32];
  int count;
};
struct TopShared {
  TopScratch scratch;
  uint64_t all[kMaxCluster * SCAPE_TOP_MAX];
};
// The `top` largest keys of this block's pieces [v0, v1) into t.best (0 where there are
// fewer), from each thread's largest value.  The threads form 32 groups; the top-th
// of the groups' largest values is a bound that at least `top` values reach and, with
// values spread over the groups, few more, so only threads whose own largest reaches
// it read their pieces again (from the caches) and collect what does.  Where that
// is too many (equal values) or too few (NaN, -infinity), the keys are found one
// after the other, each the largest below the last.
template <typename T>
__device__ void find_top(const RowPieces<T>& row, int v0, int v1, int top, float largest, TopScratch& t) {
  const int lane = threadIdx.x & 31, threads = blockDim.x, lanes = threads / 32;
  float g = largest;
  for (int o = 1; o < lanes; o <<= 1) g = fmaxf(g, __shfl_xor_sync(kAll, g, o));
  if (threadIdx.x % lanes == 0) t.group[threadIdx.x / lanes] = g;
  if (threadIdx.x == 0) t.count = 0;
  __syncthreads();
  g = t.group[lane];
  int rank = 0;
  for (int i = 0; i < 32; ++i) {
    const float o = __shfl_sync(kAll, g, i);
    rank += o > g || (o == g && i < lane);
  }
  const float bound = __shfl_sync(kAll, g, __ffs(__ballot_sync(kAll, rank == top - 1)) - 1);
  if (largest >= bound) {
    for (int v = v0 + threadIdx.x; v < v1; v += threads)
      for_values(row, v, [&](float x, int c) {
        if (x >= bound) {
          const int at = atomicAdd(&t.count, 1);
          if (at < kCandidates) t.keys[at] = key_of(x, c);
        }
      });
  }
  if (threadIdx.x < SCAPE_TOP_MAX) t.best[threadIdx.x] = 0;
  __syncthreads();
  const int n = t.count;
  if (n >= top && n <= kCandidates) {
    for (int i = threadIdx.x; i < n; i += threads) {
      const uint64_t k = t.keys[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += t.keys[j] > k;
      if (r < top) t.best[r] = k;
    }
  } else {
    uint64_t last = ~0ull;
    for (int j = 0; j < top; ++j) {
      uint64_t k = 0;
      for (int v = v0 + threadIdx.x; v < v1; v += threads)
        for_values(row, v, [&](float x, int c) {
          const uint64_t q = key_of(x, c);
          if (q < last && q > k) k = q;
        });
      k = max_over_warp(k);
      if (lane == 0) t.of_warp[threadIdx.x >> 5] = k;
      __syncthreads();
      for (int w = 0; w < threads / 32; ++w) k = t.of_warp[w] > k ? t.of_warp[w] : k;
      if (threadIdx.x == 0) t.best[j] = k;
      last = k;
      __syncthreads();
      if (k == 0) break;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ forward
// A cluster of blocks (one, where there are rows enough) takes a row.
template <typename T, bool ENT, bool TOP>
__global__ __launch_bounds__(kThreads, 4) void logprobs_kernel(const __grid_constant__ Logprobs a) {
  cluster_begin();
  start();
  __shared__ Part of_warp[kThreads / 32], of_block[kMaxCluster];
  __shared__ std::conditional_t<TOP, TopShared, int> shared;
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  const int64_t row = blockIdx.x / ranks;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const RowPieces<T> pieces(x, (int)a.vocab);
  const int v0 = (int)((int64_t)pieces.pieces * rank / ranks), v1 = (int)((int64_t)pieces.pieces * (rank + 1) / ranks);
  const int64_t target = load_target(a.targets, row);
  const bool in = target >= 0 && target < a.vocab;
  float chosen = 0.0f;
  if (threadIdx.x == 0 && rank == 0 && in) chosen = load_logit(x + target);
  Sums<ENT> own;
  for (int v = v0 + threadIdx.x; v < v1; v += kUnroll * blockDim.x) {
    uint4 u[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int w = v + i * blockDim.x;
      u[i] = w < v1 ? pieces.load(w) : minus_infinity<T>();
    }
    own.template add<T, kUnroll>(u);
  }
  const float largest = own.m;
  own.over_warp();
  if ((threadIdx.x & 31) == 0) {
    of_warp[threadIdx.x >> 5] = {own.m, own.s, own.a};
  }
  __syncthreads();
  cluster_ready();
  if constexpr (TOP) {
    find_top(pieces, v0, v1, a.top, largest, shared.scratch);
    if ((int)threadIdx.x < a.top) send(&shared.all[rank * a.top + threadIdx.x], 0, shared.scratch.best[threadIdx.x]);
  }
  if (threadIdx.x == 0) send(&of_block[rank], 0, join_parts<ENT>(of_warp, blockDim.x / 32));
  cluster_done();
  if (rank != 0) return;
  const Sums<ENT> all = join_parts<ENT>(of_block, (int)ranks);
  const float ln_s = logf(all.s), lse = all.m + ln_s;
  if (threadIdx.x == 0) {
    float lp = in ? (chosen - all.m) - ln_s : target < 0 ? 0.0f : __uint_as_float(0x7FC00000u);
    if (in && chosen == -INFINITY && all.s == 0.0f) lp = -INFINITY;
    if (a.loss && target >= 0) lp *= -(a.weight ? a.weight[row] : a.weight_all);
    if (a.logprob) a.logprob[row] = lp;
    if (a.lse) a.lse[row] = lse;
    if (ENT) a.entropy[row] = all.s == 0.0f ? 0.0f : ln_s - all.a * kLn2F / all.s;
  }
  if constexpr (TOP) {
    const uint64_t* tops = shared.all;
    const int n = (int)ranks * a.top;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const uint64_t k = tops[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += tops[j] > k;
      if (r >= a.top || k == 0) continue;
      const float v = logit_of(k);
      a.top_token[row * a.top + r] = (int64_t)(0xFFFFFFFFu - (uint32_t)k);
      a.top_logprob[row * a.top + r] = v == -INFINITY && all.s == 0.0f ? v : (v - all.m) - ln_s;
    }
  }
}

// ------------------------------------------------------------------ gradient
// Past this a float32 lse has lost what ln S adds to the row's largest logit (a row
// masked whole with the type's lowest value: lse is that value, and exp(x - lse)
// would be 1 everywhere), so the row's sums are formed again.
constexpr float kFarLse = 4096.0f;

// Such a row, by one block, which alone reads and writes it.
template <typename T, bool ENT>
__device__ __noinline__ void far_row(const T* x, T* dx, int cols, int64_t target, float g, float dh, float h) {
  __shared__ Part part[kThreads / 32];
  float top = kLowest, s = 0.0f;
  for (int c = threadIdx.x; c < cols; c += blockDim.x) top = fmaxf(top, (float)x[c]);
  for (int c = threadIdx.x; c < cols; c += blockDim.x) s += exp2_fast(((float)x[c] - top) * kLog2eF);
  Sums<false> own;
  own.m = top, own.s = s;
  own.over_warp();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = {own.m, own.s, 0.0f};
  __syncthreads();
  own = join_parts<false>(part, blockDim.x / 32);
  const float ln_s = logf(own.s);
  for (int c = threadIdx.x; c < cols; c += blockDim.x) {
    const float d = ((float)x[c] - own.m) - ln_s, p = exp2_fast(d * kLog2eF);
    float e = c == target ? -g * expm1f(d) : -g * p;
    if (ENT) e -= p * dh * (fmaxf(d, -1e4f) + h);
    dx[c] = (T)e;
  }
}

// A block takes kUnroll pieces a thread of one row, on the output's boundaries.
template <typename T, bool ENT>
__global__ __launch_bounds__(kThreads) void logprobs_bwd_kernel(const __grid_constant__ LogprobsBwd a, int chunks,
                                                                int64_t rows) {
  start();
  constexpr int kPer = RowPieces<T>::kPer;
  const int64_t row = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x % chunks);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  const T *lo = static_cast<const T*>(a.x), *hi = lo + (rows - 1) * a.ldx + a.vocab;
  const RowPieces<T> out(dx, (int)a.vocab);
  const int64_t target = load_target(a.targets, row);
  float g = a.dlogprob ? a.dlogprob[row] : a.dlogprob_all;
  if (a.negate) g = -g;
  g = target < 0 ? 0.0f : target < a.vocab ? g : __uint_as_float(0x7FC00000u);
  const float lse0 = a.lse[row], lse = lse0 == -INFINITY ? 0.0f : lse0;
  const float dh = ENT ? a.dentropy[row] : 0.0f, h = ENT ? a.entropy[row] : 0.0f;
  const bool none = !ENT && target < 0;
  if (fabsf(lse) > kFarLse && !none) {
    if (chunk == 0) far_row<T, ENT>(x, dx, (int)a.vocab, target, g, dh, h);
    return;
  }
  const int first = chunk * (kUnroll * (int)blockDim.x) + (int)threadIdx.x;
  const uint64_t minus = pair(-lse, -lse), log2e = pair(kLog2eF, kLog2eF);
  Raw<T, kPer> u[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int v = first + i * blockDim.x, c = out.column(v);
    if (none || v >= out.pieces) {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[i].w[k] = 0;
    } else if (out.whole(v)) {
      u[i] = load_any<kPer>(x + c, kPer, lo, hi);
    } else {
      const RowPieces<T> in(x, (int)a.vocab);
      // this piece's columns of the input, whose own boundaries may be others
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < in.cols) {
          if constexpr (sizeof(T) == 2)
            w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(x)[c + k] << (16 * (k % 2));
          else
            w[k] = reinterpret_cast<const uint32_t*>(x)[c + k];
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) u[i].w[k] = w[k];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int v = first + i * blockDim.x;
    if (v >= out.pieces) continue;
    const int c = out.column(v);
    float f[kPer];
    to_floats(u[i], f);
    if (none) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) f[k] = 0.0f;
    } else {
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const uint64_t d = add2(pair(f[k], f[k + 1]), minus);
        float p, q, dp, dq;
        unpair(mul2(d, log2e), p, q);
        p = exp2_fast(p), q = exp2_fast(q);
        if (ENT) {
          unpair(d, dp, dq);
          f[k] = -p * fmaf(dh, fmaxf(dp, -1e4f) + h, g);
          f[k + 1] = -q * fmaf(dh, fmaxf(dq, -1e4f) + h, g);
        } else {
          f[k] = -p * g;
          f[k + 1] = -q * g;
        }
      }
      const int64_t at = target - c;
      if (at >= 0 && at < kPer) {
        // 1 - p without the difference, which has no digits where p is near 1
        const float d = load_logit(x + target) - lse, p = exp2_fast(d * kLog2eF);
        float e = -g * expm1f(d);
        if (ENT) e -= p * dh * (fmaxf(d, -1e4f) + h);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (at == k) f[k] = e;
      }
    }
    T* p = dx + c;
    if (out.whole(v)) {
      if constexpr (sizeof(T) == 2)
        store_vec<8>(p, f);
      else
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < out.cols) p[k] = (T)f[k];
    }
  }
}

// ------------------------------------------------------------------ launches
int threads_for(int64_t pieces) {
  int t = kThreads;
  while (t > 32 && pieces * 2 <= t) t /= 2;
  return t;
}

template <typename T>
cudaError_t run_logprobs(const Logprobs& a, cudaStream_t st) {
  const int64_t pieces = ceil_div(a.vocab + RowPieces<T>::kPer - 1, RowPieces<T>::kPer);
  int cluster = 1;
  while (cluster < kMaxCluster && a.targets.count * cluster * 2 <= sm_count() &&
         pieces >= (int64_t)cluster * 2 * kThreads)
    cluster *= 2;
  const int threads = threads_for(ceil_div(pieces, cluster));
  const int64_t grid = a.targets.count * cluster;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  void (*kernel)(Logprobs) =
      a.top ? (a.entropy ? logprobs_kernel<T, true, true> : logprobs_kernel<T, false, true>)
            : (a.entropy ? logprobs_kernel<T, true, false> : logprobs_kernel<T, false, false>);
  return launch_kernel(kernel, (unsigned)grid, threads, 0, cluster, st, a);
}

template <typename T>
cudaError_t run_logprobs_bwd(const LogprobsBwd& a, cudaStream_t st) {
  const int64_t pieces = ceil_div(a.vocab + RowPieces<T>::kPer - 1, RowPieces<T>::kPer);
  const int threads = threads_for(ceil_div(pieces, kUnroll));
  const int64_t chunks = ceil_div(pieces, threads * kUnroll), grid = a.targets.count * chunks;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(a.dentropy ? logprobs_bwd_kernel<T, true> : logprobs_bwd_kernel<T, false>, (unsigned)grid,
                       threads, 0, 0, st, a, (int)chunks, a.targets.count);
}

template <typename T>
cudaError_t run_token_loss(const TokenLoss& a, cudaStream_t st) {
  Logprobs f = {};
  f.x = a.x, f.ldx = a.ldx, f.targets = a.targets, f.vocab = a.vocab;
  f.logprob = a.loss, f.lse = a.lse, f.loss = true, f.weight = a.weight, f.weight_all = a.weight_all;
  const cudaError_t e = run_logprobs<T>(f, st);
  if (e != cudaSuccess) return e;
  LogprobsBwd b = {};
  b.x = a.x, b.ldx = a.ldx, b.targets = a.targets, b.vocab = a.vocab;
  b.lse = a.lse, b.dlogprob = a.weight, b.dlogprob_all = a.weight_all, b.negate = true;
  b.dx = a.dx, b.lddx = a.lddx;
  return run_logprobs_bwd<T>(b, st);
}

}  // namespace

cudaError_t launch_logprobs(const Logprobs& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_logprobs<bf16>(a, st) : run_logprobs<float>(a, st);
}
cudaError_t launch_logprobs_bwd(const LogprobsBwd& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_logprobs_bwd<bf16>(a, st) : run_logprobs_bwd<float>(a, st);
}
bool loss_on_chip(const void*, int64_t, int, int64_t, int64_t, const void*, int64_t) { return false; }
cudaError_t launch_token_loss(const TokenLoss& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_token_loss<bf16>(a, st) : run_token_loss<float>(a, st);
}

}  // namespace layer
}  // namespace scapek
