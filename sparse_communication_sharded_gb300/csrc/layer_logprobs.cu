// layer_logprobs.cu -- log probabilities of given tokens, entropy and alternatives
// of rows of logits, their gradient, and a loss that takes its gradient along.
//
// With m a row's largest logit and d = x - m: S = sum exp d, lse = m + ln S,
// entropy = ln S - (sum exp(d) d) / S, for any m near the row's largest.  A thread
// keeps m, S and the entropy's sum of its own pieces (16 bytes at the row's 16-byte
// boundaries) while it reads them, once.  Its m is the largest of its first values:
// later ones may be above it, and only where some add 1024 to S (or are no numbers)
// is m raised, which scales S by exp(m - m'); the threads' sums are joined the same
// way.  (Exponents up to 10 keep their digits; the largest of every few values is an
// instruction a value.)  The m of a row is one of its values, at most ln 1024 below its
// largest, so where it is not the largest the others' probability is 1/1025 or more and
// the difference of two numbers that the entropy is stays above 0 by 1e4 roundings.
// Exponents are of base 2: a = d log2 e.
//
// Memory bounds these kernels only if the instructions stay few: a value's share of
// the copy rate is 10 of an SM's lane-instructions in bfloat16, an exponential alone
// is 8 of them where its unit does 16 a clock.
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
  // Whole pieces among [v0, v1): all but the row's first and last, if they are not.
  __device__ int first_whole(int v0) const { return v0 == 0 && phase > 0 ? 1 : v0; }
  __device__ int end_whole(int v1) const { return v1 == pieces && column(v1) > cols ? v1 - 1 : v1; }
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
};
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
// The largest of some pieces' values that are not NaN (if any is not).
template <typename T, int U>
__device__ __forceinline__ float pieces_top(const uint4 (&u)[U]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[k]));
    }
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < U; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u[i].x), __uint_as_float(u[i].y)),
                         fmaxf(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
    return m;
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
  template <typename T, int U>
  __device__ __forceinline__ void sum(const uint4 (&u)[U], float& s_out, float& a_out) const {
    const uint64_t minus = pair(-m, -m), log2e = pair(kLog2eF, kLog2eF);
    uint64_t s2[2] = {pair(s, 0.0f), pair(0.0f, 0.0f)}, a2[2] = {pair(a, 0.0f), pair(0.0f, 0.0f)};
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
        s2[k % 2] = add2(s2[k % 2], f);
        // where 2^e is 0 its product with an infinite e would be NaN
        if (ENT) a2[k % 2] = fma2(f, pair(fmaxf(x, -1e4f), fmaxf(y, -1e4f)), a2[k % 2]);
      }
    }
    float x, y;
    unpair(add2(s2[0], s2[1]), x, y);
    s_out = x + y;
    if (ENT) {
      unpair(add2(a2[0], a2[1]), x, y);
      a_out = x + y;
    }
  }
  // A few pieces' values.
  template <typename T, int U>
  __device__ __forceinline__ void add(const uint4 (&u)[U]) {
    if (m == kLowest) {
      const float top = pieces_top<T, U>(u);
      if (top > m) raise(top);
    }
    float s1, a1 = 0.0f;
    for (bool raised = false;; raised = true) {
      sum<T, U>(u, s1, a1);
      if (s1 - s < 1024.0f || raised) break;
      const float top = pieces_top<T, U>(u);
      if (top > m) raise(top);
    }
    s = s1, a = a1;
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
// Where the rank-th block's pieces start; a cluster has a power of two of blocks.
__device__ __forceinline__ int share_of(int pieces, uint32_t rank, uint32_t ranks) {
  return (int)(((uint64_t)pieces * rank) >> (31 - __clz(ranks)));
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
// A piece's values inside the row, with their columns.
template <typename T, typename F>
__device__ __forceinline__ void for_values(const RowPieces<T>& row, int v, const uint4& u, F&& f) {
  constexpr int kPer = RowPieces<T>::kPer;
  uint64_t p[8 / sizeof(T)];
  piece_pairs<T>(u, p);
  const int c = row.column(v);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) {
    float x, y;
    unpair(p[k], x, y);
    if (c + 2 * k >= 0 && c + 2 * k < row.cols) f(x, c + 2 * k);
    if (c + 2 * k + 1 >= 0 && c + 2 * k + 1 < row.cols) f(y, c + 2 * k + 1);
  }
}

constexpr int kMaxThreads = 1024, kMaxCluster = 8;
constexpr int kCandidates = 512;  // keys that pass the bound, before they are ranked
constexpr int kMarks = 512;       // batches that hold some

struct TopScratch {
  float group[32];
  uint64_t keys[kCandidates];
  uint64_t best[SCAPE_TOP_MAX];
  uint64_t of_warp[32];
  int marks[kMarks];
  int count, marked;
  uint64_t all[kMaxCluster * SCAPE_TOP_MAX];  // the cluster's, in its first block
};
// The `top` largest keys of this block's values into t.best, in falling order (0 where
// there are fewer), from each thread's largest value.  The threads form 32 groups; the
// top-th of the groups' largest values is a bound that at least `top` values reach
// and, with values spread over the groups, few more.  mark(bound, f) calls f(batch) for
// the thread's batches of pieces that hold a value that reaches it; these are shared
// out among all threads, a piece each: look(batch, piece, f) calls f(value, column).
// Where too many values pass (equal ones) or too few (NaN, -infinity), the keys are
// found one after the other, each the largest below the last: every(f) calls f for
// all of the thread's values.
template <typename M, typename L, typename V>
__device__ __forceinline__ void find_top(M&& mark, L&& look, V&& every, int pieces, int top, float largest,
                                         TopScratch& t) {
  const int lane = threadIdx.x & 31, threads = blockDim.x, lanes = threads / 32;
  float g = largest;
  for (int o = 1; o < lanes; o <<= 1) g = fmaxf(g, __shfl_xor_sync(kAll, g, o));
  if (threadIdx.x % lanes == 0) t.group[threadIdx.x / lanes] = g;
  if (threadIdx.x == 0) t.count = t.marked = 0;
  __syncthreads();
  g = t.group[lane];
  int rank = 0;
  for (int i = 0; i < 32; ++i) {
    const float o = __shfl_sync(kAll, g, i);
    rank += o > g || (o == g && i < lane);
  }
  const float bound = __shfl_sync(kAll, g, __ffs(__ballot_sync(kAll, rank == top - 1)) - 1);
  // the order of marks and keys changes nothing: keys differ and are ranked
  if (largest >= bound)
    mark(bound, [&](int batch) {
      const int at = atomicAdd(&t.marked, 1);
      if (at < kMarks) t.marks[at] = batch;
    });
  __syncthreads();
  const int marked = t.marked;
  if (marked <= kMarks)
    for (int i = threadIdx.x; i < marked * pieces; i += threads)
      look(t.marks[i / pieces], i % pieces, [&](float x, int c) {
        if (x >= bound) {
          const int at = atomicAdd(&t.count, 1);
          if (at < kCandidates) t.keys[at] = key_of(x, c);
        }
      });
  if (threadIdx.x < SCAPE_TOP_MAX) t.best[threadIdx.x] = 0;
  __syncthreads();
  const int n = t.count;
  if (marked <= kMarks && n >= top && n <= kCandidates) {
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
      every([&](float x, int c) {
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

// ------------------------------------------------------------------ results of a row
// x - lse from the row's sums; -infinity where nothing is left.
template <bool ENT>
__device__ __forceinline__ float log_probability(float x, const Sums<ENT>& all, float ln_s) {
  return x == -INFINITY && all.s == 0.0f ? x : (x - all.m) - ln_s;
}
// What lse = m + ln S has lost in its rounding: the sum's error is a number in 32 bits.
__device__ __forceinline__ float rest_of(float m, float ln_s, float lse) {
  const float b = lse - m;
  return fabsf(lse) < INFINITY ? (m - (lse - b)) + (ln_s - b) : 0.0f;
}
// By one thread; chosen: the target's logit, if there is one.
template <bool ENT>
__device__ __forceinline__ void write_row(const Logprobs& a, int64_t row, int64_t target, float chosen,
                                          const Sums<ENT>& all, float ln_s) {
  float lp = target < 0 ? 0.0f : target < a.vocab ? log_probability(chosen, all, ln_s) : __uint_as_float(0x7FC00000u);
  if (a.loss && target >= 0) lp *= -(a.weight ? a.weight[row] : a.weight_all);
  a.logprob[row] = lp;
  const float lse = all.m + ln_s;
  if (a.lse) a.lse[row] = lse;
  if (a.rest) a.rest[row] = rest_of(all.m, ln_s, lse);
  if (ENT) a.entropy[row] = all.s == 0.0f ? 0.0f : ln_s - all.a * kLn2F / all.s;
}
// Of the n keys of a cluster's blocks, the largest.
template <bool ENT>
__device__ __forceinline__ void write_top(const Logprobs& a, int64_t row, const uint64_t* keys, int n,
                                          const Sums<ENT>& all, float ln_s) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t k = keys[i];
    int r = i;
    if (n > a.top) {
      r = 0;
      for (int j = 0; j < n; ++j) r += keys[j] > k;
    }
    if (r >= a.top || k == 0) continue;
    a.top_token[row * a.top + r] = (int64_t)(0xFFFFFFFFu - (uint32_t)k);
    a.top_logprob[row * a.top + r] = log_probability(logit_of(k), all, ln_s);
  }
}

// A row's pieces [v0, v1) of a block, of which [w0, w1) are whole.
template <typename T>
struct Share {
  RowPieces<T> row;
  int v0, v1, w0, w1;
  __device__ Share(const T* x, int64_t vocab, uint32_t rank, uint32_t ranks) : row(x, (int)vocab) {
    v0 = share_of(row.pieces, rank, ranks);
    v1 = share_of(row.pieces, rank + 1, ranks);
    w0 = row.first_whole(v0);
    w1 = max(w0, row.end_whole(v1));
  }
  __device__ bool part_before() const { return v0 < w0 && v0 < v1; }
  __device__ bool part_after() const { return w1 < v1; }
  __device__ const uint4* whole_pieces() const { return reinterpret_cast<const uint4*>(row.x - row.phase) + w0; }
};

// ------------------------------------------------------------------ forward
// A block, or a cluster of them each with a part of the row, takes one row; every
// thread has a ring of its own pieces in shared memory, kAhead batches deep, and waits
// for nothing but its own copies until the threads' sums are joined.  Seven blocks of
// 128 threads an SM, so that others read meanwhile (8192 x 32000 in bfloat16 with
// entropy: 82 us, 94% of the copy rate; blocks that go from row to row 88, four of 256
// threads 103, pieces read into registers 105).  Six with alternatives, whose search
// takes more registers (4096 x 32000 with five: 63 us, three of 256 threads 88, without
// alternatives 42).
constexpr int kTeam = 128, kUnroll = 4, kAhead = 3;
constexpr int kBlocks = 7, kBlocksTop = 6;  // an SM

template <typename T, bool ENT, bool TOP>
__global__ __launch_bounds__(kTeam, TOP ? kBlocksTop : kBlocks) void logprobs_kernel(
    const __grid_constant__ Logprobs a, int batches) {
  cluster_begin();
  start();
  extern __shared__ __align__(16) uint4 ring[];  // [kAhead][kUnroll][threads]
  // and, for the alternatives, each batch's largest value: the thread's own, every
  // threads-th
  float* const tops = reinterpret_cast<float*>(ring + kAhead * kUnroll * blockDim.x) + threadIdx.x;
  __shared__ Part of_warp[kTeam / 32], of_block[kMaxCluster];
  __shared__ std::conditional_t<TOP, TopScratch, int> scratch;
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  const int lane = threadIdx.x & 31, threads = blockDim.x, warps = threads / 32;
  const int64_t row = blockIdx.x / ranks;
  const Share<T> r(static_cast<const T*>(a.x) + row * a.ldx, a.vocab, rank, ranks);
  const uint4* const whole = r.whole_pieces();
  const int n = r.w1 - r.w0;
  const uint32_t own_ring = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
  int ahead = (int)threadIdx.x;  // the piece that the ring is to be given next
  auto copy = [&](int stage) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (ahead + i * threads < n)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(own_ring + (stage * kUnroll + i) * threads * 16),
                     "l"(whole + ahead + i * threads)
                     : "memory");
    ahead += kUnroll * threads;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) copy(s);
  const int64_t target = load_target(a.targets, row);
  const bool in = target >= 0 && target < a.vocab;
  float chosen = 0.0f;
  if (threadIdx.x == 0 && rank == 0 && in) chosen = (float)r.row.x[target];
  Sums<ENT> own;
  float largest = kLowest, batch_top;
  auto take = [&](auto& u) {
    constexpr int U = sizeof(u) / sizeof(uint4);
    own.template add<T, U>(u);
    if (TOP) batch_top = fmaxf(batch_top, pieces_top<T, U>(u));
  };
  int stage = 0, left = n - (int)threadIdx.x;
  for (int b = 0; b < batches; ++b) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const uint4* p = ring + stage * kUnroll * threads + threadIdx.x;
    batch_top = kLowest;
    if (left > (kUnroll - 1) * threads) {
      uint4 u[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) u[i] = p[i * threads];
      take(u);
    } else {
      for (int l = left; l > 0; l -= threads, p += threads) {
        const uint4 u[1] = {*p};
        take(u);
      }
    }
    if (TOP) tops[b * threads] = batch_top, largest = fmaxf(largest, batch_top);
    left -= kUnroll * threads;
    copy(stage);
    if (++stage == kAhead) stage = 0;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      if (!(i ? r.part_after() : r.part_before())) continue;
      const uint4 u[1] = {r.row.load_part(i ? r.w1 : r.v0)};
      take(u);
      if (TOP) largest = fmaxf(largest, batch_top);
    }
  }
  own.over_warp();
  if (lane == 0) of_warp[threadIdx.x >> 5] = {own.m, own.s, own.a};
  __syncthreads();
  cluster_ready();
  if constexpr (TOP) {
    find_top(
        [&](float bound, auto&& f) {
          for (int b = 0; b < batches; ++b)
            if (tops[b * threads] >= bound) f(b * threads + (int)threadIdx.x);
          if (threadIdx.x == 0 && (r.part_before() || r.part_after())) f(-1);
        },
        [&](int batch, int piece, auto&& f) {  // out of the caches
          if (batch < 0) {
            if (piece == 0 && r.part_before()) for_values(r.row, r.v0, r.row.load_part(r.v0), f);
            if (piece == 1 && r.part_after()) for_values(r.row, r.w1, r.row.load_part(r.w1), f);
            return;
          }
          const int v = batch / threads * (kUnroll * threads) + batch % threads + piece * threads;
          if (v < n) for_values(r.row, r.w0 + v, whole[v], f);
        },
        [&](auto&& f) {
          for (int v = (int)threadIdx.x; v < n; v += threads) for_values(r.row, r.w0 + v, whole[v], f);
          if (threadIdx.x != 0) return;
          if (r.part_before()) for_values(r.row, r.v0, r.row.load_part(r.v0), f);
          if (r.part_after()) for_values(r.row, r.w1, r.row.load_part(r.w1), f);
        },
        kUnroll, a.top, largest, scratch);
  }
  if (ranks > 1) {
    if constexpr (TOP) {
      if ((int)threadIdx.x < a.top) send(&scratch.all[rank * a.top + threadIdx.x], 0, scratch.best[threadIdx.x]);
    }
    if (threadIdx.x == 0) send(&of_block[rank], 0, join_parts<ENT>(of_warp, warps));
    cluster_done();
  }
  if (rank != 0 || (!TOP && threadIdx.x != 0)) return;
  const Sums<ENT> all = ranks > 1 ? join_parts<ENT>(of_block, (int)ranks) : join_parts<ENT>(of_warp, warps);
  const float ln_s = logf(all.s);
  if (threadIdx.x == 0) write_row(a, row, target, chosen, all, ln_s);
  if constexpr (TOP) write_top(a, row, ranks > 1 ? scratch.all : scratch.best, (int)ranks * a.top, all, ln_s);
}

// ------------------------------------------------------------------ loss
// What a row's gradient is of its exponentials: w / S, w 0 without a target and NaN with
// one that is none of the columns.
__device__ __forceinline__ float loss_weight(const Logprobs& a, int64_t target, float w) {
  return target < 0 ? 0.0f : target < a.vocab ? w : __uint_as_float(0x7FC00000u);
}
__device__ __forceinline__ float loss_scale(const Sums<false>& all, float w) {
  return all.s == 0.0f ? 0.0f * w : w / all.s;
}
template <typename T, int N>
__device__ __forceinline__ void loss_gradient(const uint4& u, float m, float scale, float (&f)[N]) {
  const uint64_t minus = pair(-m, -m), log2e = pair(kLog2eF, kLog2eF), scale2 = pair(scale, scale);
  uint64_t q[N / 2];
  piece_pairs<T>(u, q);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    float x, y;
    unpair(mul2(add2(q[k], minus), log2e), x, y);
    unpair(mul2(pair(exp2_fast(x), exp2_fast(y)), scale2), f[2 * k], f[2 * k + 1]);
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* o, const float (&f)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2)
    store_vec<8>(o, f);
  else
    *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
}

// The row stays in shared memory between its sums and its gradient, so logits are
// read once.  A block, or a cluster of them each with a part of the row, takes one
// row; every thread copies its own pieces to places of its own, which it alone reads.
// Two or more blocks an SM and no more than a row's life for each: while some wait
// for their row or their barrier others compute or store, and none waits for the
// slowest.  (8192 x 50304 in bfloat16: 234 us, what a copy of as many bytes takes; as
// many blocks as fit, going from row to row, 255; one block an SM with the next row on
// its way 277; sums and gradient in a kernel each 384.)
template <typename T>
__global__ __launch_bounds__(kMaxThreads) void token_loss_kernel(const __grid_constant__ Logprobs a) {
  cluster_begin();
  start();
  constexpr int kPer = RowPieces<T>::kPer, kHeldUnroll = 2;
  extern __shared__ __align__(16) uint4 held[];  // the block's pieces
  __shared__ Part of_warp[kMaxThreads / 32], of_block[kMaxCluster];
  const uint32_t rank = block_rank(), ranks = cluster_blocks();
  const int lane = threadIdx.x & 31, threads = blockDim.x, warps = threads / 32;
  const int64_t row = blockIdx.x / ranks;
  const Share<T> r(static_cast<const T*>(a.x) + row * a.ldx, a.vocab, rank, ranks);
  const int n = r.w1 - r.w0 - (int)threadIdx.x;  // pieces from this thread's first one on
  uint4* const mine = held + threadIdx.x;        // every threads-th
  {
    uint32_t to = (uint32_t)__cvta_generic_to_shared(mine);
    const uint4* from = r.whole_pieces() + threadIdx.x;
    for (int left = n; left > 0; left -= threads, to += threads * 16, from += threads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the pieces that are part of a row at its ends are the first thread's
  __shared__ uint4 ends[2];
  if (threadIdx.x == 0) {
    if (r.part_before()) ends[0] = r.row.load_part(r.v0);
    if (r.part_after()) ends[1] = r.row.load_part(r.w1);
  }
  const int64_t target = load_target(a.targets, row);
  float w = a.weight ? a.weight[row] : a.weight_all;
  cluster_ready();
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  Sums<false> own;
  {
    const uint4* p = mine;
    int left = n;
    for (; left > (kHeldUnroll - 1) * threads; left -= kHeldUnroll * threads, p += kHeldUnroll * threads) {
      uint4 u[kHeldUnroll];
#pragma unroll
      for (int i = 0; i < kHeldUnroll; ++i) u[i] = p[i * threads];
      own.template add<T, kHeldUnroll>(u);
    }
    for (; left > 0; left -= threads, p += threads) {
      const uint4 u[1] = {*p};
      own.template add<T, 1>(u);
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) {
        const uint4 u[1] = {ends[i]};
        if (i ? r.part_after() : r.part_before()) own.template add<T, 1>(u);
      }
    }
  }
  own.over_warp();
  if (lane == 0) of_warp[threadIdx.x >> 5] = {own.m, own.s, 0.0f};
  __syncthreads();
  const Part p0 = of_warp[lane < warps ? lane : 0];
  own.m = p0.m, own.s = lane < warps ? p0.s : 0.0f;
  own.over_warp();
  if (ranks > 1) {
    if (threadIdx.x < ranks) send(&of_block[rank], threadIdx.x, own);
    cluster_done();
    own = join_parts<false>(of_block, (int)ranks);
  }
  const bool none = target < 0, in = !none && target < a.vocab;
  w = loss_weight(a, target, w);
  const float scale = loss_scale(own, w);
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  T* o = dx + r.row.column(r.w0 + threadIdx.x);
  const uint4* p = mine;
  for (int left = n; left > 0; left -= threads, p += threads, o += threads * kPer) {
    float f[kPer];
    if (none) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) f[k] = 0.0f;
    } else {
      loss_gradient<T>(*p, own.m, scale, f);
    }
    store_piece(o, f);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      if (!(i ? r.part_after() : r.part_before())) continue;
      float f[kPer];
      loss_gradient<T>(ends[i], own.m, scale, f);
      const int c = r.row.column(i ? r.w1 : r.v0);
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < r.row.cols) dx[c + k] = none ? (T)0.0f : (T)f[k];
    }
  }
  // the target, by the thread that has its piece (and has stored its gradient)
  if (in) {
    const uint32_t at = (uint32_t)target + (uint32_t)r.row.phase;
    const int v = (int)(at / kPer), k = (int)(at % kPer);
    const bool whole = v >= r.w0 && v < r.w1;
    if (v >= r.v0 && v < r.v1 && (int)threadIdx.x == (whole ? (v - r.w0) & (threads - 1) : 0)) {
      const uint4 u = whole ? mine[(v - r.w0) & -threads] : ends[v < r.w0 ? 0 : 1];
      const uint32_t words[4] = {u.x, u.y, u.z, u.w};
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == k) x = __uint_as_float(sizeof(T) == 2 ? (i % 2 ? words[i / 2] & 0xFFFF0000u : words[i / 2] << 16)
                                                       : words[i * (int)sizeof(T) / 4]);
      const float d = log_probability(x, own, logf(own.s));
      dx[target] = (T)(w * expm1f(d));  // p - 1 without the difference
      a.logprob[row] = -w * d;
    }
  } else if (rank == 0 && threadIdx.x == 0) {
    a.logprob[row] = w;  // 0 or NaN
  }
}

// ------------------------------------------------------------------ short rows
// A warp takes a row, each lane U of its pieces in registers, with the next row's on
// their way; with LOSS its gradient goes out from there.  What bounds it is a row's own
// work, the joining of 32 lanes' sums and what lane 0 does with them.  16384 rows in
// bfloat16, log probabilities and loss: of 256 columns 7.9 and 10.8 us, of 1000 9.2 and
// 15.6 (a block a row 19 and 20.7), of 2000, where U is 8 and four blocks fit, 13.5 and
// 25.6 (24.8 and 34.5).  Longer rows have no room in registers.
constexpr int kShortWarps = 4;
constexpr int short_blocks(int u) { return u <= 4 ? 6 : 4; }  // an SM

template <typename T, bool ENT, bool LOSS, int U>
__global__ __launch_bounds__(kShortWarps * 32, short_blocks(U)) void short_rows_kernel(
    const __grid_constant__ Logprobs a) {
  start();
  constexpr int kPer = RowPieces<T>::kPer;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kShortWarps;
  uint4 next[U];
  int64_t next_target = 0;
  float next_w = 0.0f;
  auto load = [&](int64_t row) {
    if (row >= a.targets.count) return;
    const RowPieces<T> r(static_cast<const T*>(a.x) + row * a.ldx, (int)a.vocab);
    next_target = load_target(a.targets, row);
    if (LOSS) next_w = a.weight ? a.weight[row] : a.weight_all;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = lane + i * 32;
      constexpr uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -infinity
      next[i] = make_uint4(none, none, none, none);
      if (r.whole(v)) next[i] = *reinterpret_cast<const uint4*>(r.x + r.column(v));
    }
    if (r.phase == 0 && r.cols % kPer == 0) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = lane + i * 32;
      if (v < r.pieces && !r.whole(v)) next[i] = r.load_part(v);
    }
  };
  int64_t row = (int64_t)blockIdx.x * kShortWarps + (threadIdx.x >> 5);
  load(row);
  for (; row < a.targets.count; row += step) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = next[i];
    const int64_t target = next_target;
    const float weight = next_w;
    load(row + step);
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const bool in = target >= 0 && target < a.vocab;
    const float chosen = in ? (float)x[target] : 0.0f;
    Sums<ENT> own;
    own.template add<T, U>(u);
    own.over_warp();
    const float ln_s = logf(own.s);
    if constexpr (!LOSS) {
      if (lane == 0) write_row(a, row, target, chosen, own, ln_s);
    } else {
      const float w = loss_weight(a, target, weight), scale = loss_scale(own, w);
      T* dx = static_cast<T*>(a.dx) + row * a.lddx;
      const RowPieces<T> r(dx, (int)a.vocab);
      __syncwarp();  // all have the target's logit, which may be in the gradient's place
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = lane + i * 32, c = r.column(v);
        if (v >= r.pieces) continue;
        float f[kPer];
        loss_gradient<T>(u[i], own.m, scale, f);
        if (target < 0) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) f[k] = 0.0f;
        }
        if (r.whole(v)) {
          store_piece(dx + c, f);
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (c + k >= 0 && c + k < r.cols) dx[c + k] = (T)f[k];
        }
      }
      __syncwarp();  // the target's, over what its piece had
      if (lane == 0) {
        const float d = log_probability(chosen, own, ln_s);
        if (in) dx[target] = (T)(w * expm1f(d));
        a.logprob[row] = in ? -w * d : w;  // 0 or NaN
      }
    }
  }
}

// ------------------------------------------------------------------ gradient
// p = exp((x - lse) - rest).  Without the rest p is off by what lse's rounding is, 2^-24
// |lse| of itself: 2^-12 here, where lse tells ln S to 2^-12, and in a row masked whole
// with the type's lowest value it says nothing of ln S (lse is that value, and exp(x -
// lse) would be 1 everywhere).  So past this the row's sums are formed again.
constexpr float kFarLse = 4096.0f;
constexpr int kBwdThreads = 256, kBwdRows = 8;
template <bool ANY>
constexpr int kBwdUnroll = ANY ? 2 : 4;

// Such a row, by the threads of one threadIdx.y, which alone read and write it.
template <typename T, bool ENT>
__device__ __noinline__ void far_row(const T* x, T* dx, int cols, int64_t target, float g, float dh, float h) {
  __shared__ Part part[kBwdThreads / 32];
  float top = kLowest, s = 0.0f;
  for (int c = threadIdx.x; c < cols; c += blockDim.x) top = fmaxf(top, (float)x[c]);
  for (int c = threadIdx.x; c < cols; c += blockDim.x) s += exp2_fast(((float)x[c] - top) * kLog2eF);
  Sums<false> own;
  own.m = top, own.s = s;
  own.over_warp();
  if (blockDim.x > 32) {  // the block's only row
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = {own.m, own.s, 0.0f};
    __syncthreads();
    own = join_parts<false>(part, blockDim.x / 32);
  }
  const float ln_s = logf(own.s);
  for (int c = threadIdx.x; c < cols; c += blockDim.x) {
    const float d = ((float)x[c] - own.m) - ln_s, p = exp2_fast(d * kLog2eF);
    float e = c == target ? -g * expm1f(d) : -g * p;
    if (ENT) e -= p * dh * (fmaxf(d, -1e4f) + h);
    dx[c] = (T)e;
  }
}

// A block takes kBwdUnroll pieces a thread of one row, on the output's boundaries.
// REST: lse comes in two numbers, and a row's loads need not wait for lse to tell whether
// it is far (4096 x 32000 in bfloat16 with the entropy: 78 us, without REST 85; without
// the entropy 82 and 79, at other places 97 and 100).
// MANY: a warp's are a row, and a block takes kBwdRows of them (16384 x 256 in bfloat16:
// 7.5 us, a block a row 17).
// ANY: they are on no boundaries of the logits' rows, and a load is two (4096 x 32000
// in bfloat16 without entropy: 79 us, ANY 100; with four pieces at a time 112).
template <typename T, bool ENT, bool ANY, bool MANY, bool REST>
__global__ __launch_bounds__(kBwdThreads) void logprobs_bwd_kernel(const __grid_constant__ LogprobsBwd a, int chunks,
                                                                   int64_t rows) {
  start();
  constexpr int kPer = RowPieces<T>::kPer, U = kBwdUnroll<ANY>;
  const int64_t row = MANY ? (int64_t)blockIdx.x * kBwdRows + threadIdx.y : blockIdx.x / chunks;
  if (MANY && row >= rows) return;
  const int chunk = MANY ? 0 : (int)(blockIdx.x % chunks);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  const T *lo = static_cast<const T*>(a.x), *hi = lo + (rows - 1) * a.ldx + a.vocab;
  const RowPieces<T> out(dx, (int)a.vocab);
  const int64_t target = load_target(a.targets, row);
  float g = a.dlogprob ? a.dlogprob[row] : a.dlogprob_all;
  if (a.negate) g = -g;
  g = target < 0 ? 0.0f : target < a.vocab ? g : __uint_as_float(0x7FC00000u);
  // The target's column, or one that no piece has: pieces reach over both ends of a row
  // (from column 1 - kPer on), and a target that is none or too large may be a number there.
  const int64_t chosen = target >= 0 && target < a.vocab ? target : -kPer;
  const float lse0 = a.lse[row], rest0 = REST ? a.rest[row] : 0.0f;  // (one load does not wait for the other)
  const float lse = lse0 == -INFINITY ? 0.0f : lse0, rest = lse0 == -INFINITY ? 0.0f : rest0;
  const float dh = ENT ? a.dentropy[row] : 0.0f, h = ENT ? a.entropy[row] : 0.0f;
  const bool none = !ENT && target < 0;
  if (!REST && fabsf(lse) > kFarLse && !none) {
    if (chunk == 0) far_row<T, ENT>(x, dx, (int)a.vocab, target, g, dh, h);
    return;
  }
  const int first = chunk * (U * (int)blockDim.x) + (int)threadIdx.x;
  // p is exp(x - lse) times the rest's exponential, which goes to the row's factors.
  // (Before the loads or after them: 8192 x 50304 in bfloat16 at other places, the loss,
  // 454 us or 429, 2000 x 50304 in float32 211 or 227.)
  float g_all = g, dh_all = dh, h_all = h;
  auto join_rest = [&] {
    if (!REST) return;
    const float e = exp2_fast(-rest * kLog2eF);
    g_all *= e, dh_all *= e, h_all -= rest;
  };
  if (sizeof(T) == 4) join_rest();
  const uint64_t minus = pair(-lse, -lse), log2e = pair(kLog2eF, kLog2eF);
  AnyLoad<T, kPer> any[U];
  uint4 plain[U] = {};
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = first + i * blockDim.x, c = out.column(v);
    const int n = !none && v < out.pieces && out.whole(v) ? kPer : 0;
    if constexpr (ANY)
      any[i].begin(x + c, n, lo, hi);
    else if (n)
      plain[i] = *reinterpret_cast<const uint4*>(x + c);
  }
  if (sizeof(T) == 2) join_rest();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = first + i * blockDim.x;
    if (v >= out.pieces) continue;
    const int c = out.column(v);
    Raw<T, kPer> u;
    u.w[0] = plain[i].x, u.w[1] = plain[i].y, u.w[2] = plain[i].z, u.w[3] = plain[i].w;
    if constexpr (ANY) u = any[i].end(x + c, !none && out.whole(v) ? kPer : 0);
    if (!none && !out.whole(v)) {
      // columns at a row's ends
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < out.cols) {
          if constexpr (sizeof(T) == 2)
            u.w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(x)[c + k] << (16 * (k % 2));
          else
            u.w[k] = reinterpret_cast<const uint32_t*>(x)[c + k];
        }
    }
    float f[kPer];
    to_floats(u, f);
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
          f[k] = -p * fmaf(dh_all, fmaxf(dp, -1e4f) + h_all, g_all);
          f[k + 1] = -q * fmaf(dh_all, fmaxf(dq, -1e4f) + h_all, g_all);
        } else {
          f[k] = -p * g_all;
          f[k + 1] = -q * g_all;
        }
      }
      const int64_t at = chosen - c;
      if (at >= 0 && at < kPer) {
        // 1 - p without the difference, which has no digits where p is near 1 (nor has d
        // there, if the rest of lse is not given)
        float d = load_logit(x + chosen) - lse;
        if (REST) d -= rest;
        const float p = exp2_fast(d * kLog2eF);
        float e = -g * expm1f(d);
        if (ENT) e -= p * dh * (fmaxf(d, -1e4f) + h);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (at == k) f[k] = e;
      }
    }
    T* p = dx + c;
    if (out.whole(v)) {
      store_piece(p, f);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k >= 0 && c + k < out.cols) p[k] = (T)f[k];
    }
  }
}

// ------------------------------------------------------------------ launches
// Pieces of the logits are pieces of the gradient.
bool same_places(const void* x, int64_t ldx, const void* dx, int64_t lddx, int elem) {
  return (reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(dx)) % 16 == 0 && (ldx - lddx) * elem % 16 == 0;
}

int threads_for(int64_t pieces, int most) {
  int t = most;
  while (t > 32 && pieces * 2 <= t) t /= 2;
  return t;
}
// How rows are held: blocks a row, threads and pieces a block.  cluster 0: not at all.
struct HeldPlan {
  int cluster, threads, pieces;
};
constexpr int64_t kSmBytes = 227 * 1024, kTopBytes = 211 * 1024;

HeldPlan held_plan(int64_t rows, int64_t vocab, int elem) {
  const int64_t per = 16 / elem, pieces = ceil_div(vocab + per - 1, per);
  for (int cluster = 1; cluster <= kMaxCluster; cluster *= 2) {
    const int64_t part = ceil_div(pieces, cluster), fit = kSmBytes / (part * 16 + 2048);
    // few rows are spread over the SMs; two blocks or more an SM
    if (cluster < kMaxCluster && ((rows * cluster * 2 <= sm_count() && part >= 2 * 512) || fit < 2)) continue;
    if (fit < 1) break;
    return {cluster, fit == 1 ? 1024 : fit == 2 ? 512 : fit == 3 ? 256 : 128, (int)part};
  }
  return {};
}
template <typename T, bool ENT, bool TOP>
cudaError_t run_rows(const Logprobs& a, cudaStream_t st) {
  const int64_t rows = a.targets.count, pieces = ceil_div(a.vocab + RowPieces<T>::kPer - 1, RowPieces<T>::kPer);
  // As many blocks a row as make the least of the rounds of blocks times a block's
  // batches, of which joining the sums is worth two and looking for alternatives four
  // more.
  int cluster = 0, threads = 0, smem = 0;
  int64_t batches = 0, least = 0;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    const int64_t part = ceil_div(pieces, c);
    const int t = threads_for(ceil_div(part, kUnroll), kTeam);
    const int64_t n = ceil_div(part, t * kUnroll);
    const int64_t bytes = (int64_t)kAhead * kUnroll * t * 16 + (TOP ? n * t * 4 : 0);
    if (bytes > kTopBytes) continue;
    const int64_t per_sm = std::min<int64_t>(std::min((TOP ? kBlocksTop : kBlocks) * kTeam / t, 32),
                                             kSmBytes / (bytes + (TOP ? 12800 : 2048)));
    const int64_t cost = ceil_div(rows * c, sm_count() * per_sm) * (n + (TOP ? 6 : 2));
    if (cluster && cost >= least) continue;
    cluster = c, threads = t, batches = n, smem = (int)bytes, least = cost;
  }
  if (!cluster || rows * cluster > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto* const kernel = logprobs_kernel<T, ENT, TOP>;
  if (smem > 32 * 1024) {  // with the static part, what a kernel may have unasked is 48 KB
    const cudaError_t e = allow_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, (unsigned)(rows * cluster), threads, smem, cluster > 1 ? cluster : 0, st, a,
                       (int)batches);
}
// Pieces a lane of a warp that holds a row, wherever it starts; 0: too many.
template <typename T>
int short_unroll(int64_t vocab) {
  const int64_t pieces = ceil_div(vocab + RowPieces<T>::kPer - 1, RowPieces<T>::kPer);
  return pieces <= 32 * 4 ? 4 : pieces <= 32 * 8 ? 8 : 0;
}
template <typename T, bool ENT, bool LOSS>
cudaError_t run_short(const Logprobs& a, int unroll, cudaStream_t st) {
  const int64_t blocks = ceil_div(a.targets.count, kShortWarps);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sm_count() * short_blocks(unroll));
  auto* const kernel = unroll == 4 ? short_rows_kernel<T, ENT, LOSS, 4> : short_rows_kernel<T, ENT, LOSS, 8>;
  return launch_kernel(kernel, grid, kShortWarps * 32, 0, 0, st, a);
}
template <typename T>
cudaError_t run_logprobs(const Logprobs& a, cudaStream_t st) {
  const int unroll = a.top ? 0 : short_unroll<T>(a.vocab);
  if (unroll) return a.entropy ? run_short<T, true, false>(a, unroll, st) : run_short<T, false, false>(a, unroll, st);
  if (a.top) return a.entropy ? run_rows<T, true, true>(a, st) : run_rows<T, false, true>(a, st);
  return a.entropy ? run_rows<T, true, false>(a, st) : run_rows<T, false, false>(a, st);
}

template <typename T>
cudaError_t run_logprobs_bwd(const LogprobsBwd& a, cudaStream_t st) {
  const int64_t pieces = ceil_div(a.vocab + RowPieces<T>::kPer - 1, RowPieces<T>::kPer);
  const bool same = same_places(a.x, a.ldx, a.dx, a.lddx, sizeof(T));
  const int unroll = same ? kBwdUnroll<false> : kBwdUnroll<true>;
  const int threads = threads_for(ceil_div(pieces, unroll), kBwdThreads);
  const bool many = threads == 32;
  const int64_t chunks = ceil_div(pieces, threads * unroll);
  const int64_t grid = many ? ceil_div(a.targets.count, kBwdRows) : a.targets.count * chunks;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto run = [&](auto kernel) {
    return launch_kernel(kernel, (unsigned)grid, dim3((unsigned)threads, many ? kBwdRows : 1), 0, 0, st, a,
                         (int)chunks, a.targets.count);
  };
  auto of = [&](auto ent, auto any, auto rest) {
    constexpr bool E = decltype(ent)::value, A = decltype(any)::value, R = decltype(rest)::value;
    return many ? run(logprobs_bwd_kernel<T, E, A, true, R>) : run(logprobs_bwd_kernel<T, E, A, false, R>);
  };
  auto with = [&](auto ent, auto any) {
    return a.rest ? of(ent, any, std::true_type()) : of(ent, any, std::false_type());
  };
  if (a.dentropy) return same ? with(std::true_type(), std::false_type()) : with(std::true_type(), std::true_type());
  return same ? with(std::false_type(), std::false_type()) : with(std::false_type(), std::true_type());
}

template <typename T>
cudaError_t run_token_loss(const TokenLoss& a, cudaStream_t st) {
  Logprobs f = {};
  f.x = a.x, f.ldx = a.ldx, f.targets = a.targets, f.vocab = a.vocab;
  f.logprob = a.loss, f.loss = true, f.weight = a.weight, f.weight_all = a.weight_all;
  if (same_places(a.x, a.ldx, a.dx, a.lddx, sizeof(T))) {
    const HeldPlan p = held_plan(a.targets.count, a.vocab, sizeof(T));
    if (p.cluster) {
      f.dx = a.dx, f.lddx = a.lddx;
      const int unroll = short_unroll<T>(a.vocab);
      if (unroll) return run_short<T, false, true>(f, unroll, st);
      const int smem = p.pieces * 16;
      if (smem > 32 * 1024) {  // with the static part, what a kernel may have unasked is 48 KB
        const cudaError_t e = allow_smem((const void*)token_loss_kernel<T>, smem);
        if (e != cudaSuccess) return e;
      }
      const int64_t grid = a.targets.count * p.cluster;
      if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
      return launch_kernel(token_loss_kernel<T>, (unsigned)grid, p.threads, smem, p.cluster > 1 ? p.cluster : 0, st, f);
    }
  }
  f.lse = a.lse, f.rest = a.rest;
  const cudaError_t e = run_logprobs<T>(f, st);
  if (e != cudaSuccess) return e;
  LogprobsBwd b = {};
  b.x = a.x, b.ldx = a.ldx, b.targets = a.targets, b.vocab = a.vocab;
  b.lse = a.lse, b.rest = a.rest, b.dlogprob = a.weight, b.dlogprob_all = a.weight_all, b.negate = true;
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
bool loss_on_chip(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t vocab, const void* dx, int64_t lddx) {
  const int elem = dtype == SCAPE_BF16 ? 2 : 4;
  return held_plan(rows, vocab, elem).cluster && same_places(x, ldx, dx, lddx, elem);
}
cudaError_t launch_token_loss(const TokenLoss& a, int dtype, cudaStream_t st) {
  return dtype == SCAPE_BF16 ? run_token_loss<bf16>(a, st) : run_token_loss<float>(a, st);
}

}  // namespace layer
}  // namespace scapek
