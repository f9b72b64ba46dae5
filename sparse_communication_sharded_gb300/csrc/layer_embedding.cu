// layer_embedding.cu -- rows of a table by token, and the table's gradient.
//
// Forward: y[i] = scale w[token i].  Bound by memory; a thread takes four pieces of 8
// columns so that their loads are in flight together (16384 x 1280 in bfloat16: 11.6
// us, 106% of the copy rate, where rows that come twice are in L2, 13.9 where none is).
// Where rows are on no 16-byte boundary one piece, whose aligned words are three loads
// (16381 x 1283 from float32: 20 us, with four pieces and their registers 38).
//
// Gradient: dw[v] = scale * sum of the dy rows of token v.  Atomics on dw would add
// in an order that changes, and in the output's type.  So the positions are sorted by
// token (stable: integers only), cut into tiles of kEmbedTile that blocks add up in
// 32 bits; a token with many positions leaves partial sums, joined in the tiles' order
// by blocks that are done last.  Most rows of a large table have no token, and writing
// their zeros is most of the bytes: that goes on beside the sums.
//
// 50304 x 1024 from 8192 tokens of a text, bfloat16: 27.9 to 29.3 us (sort 8, sums and
// zeros 22, each alone under ncu), its bytes at the copy rate 17.6; added to what is
// there, without zeros, 23.5.  The second launch waits for the first, which writes
// nothing but the order.
#include <algorithm>

#include "layer_tokens.h"

namespace scapek {
namespace layer {
namespace {

__device__ __forceinline__ int64_t load_token(const Tokens& t, int64_t i) {
  return t.bytes == 8 ? static_cast<const int64_t*>(t.p)[i] : (int64_t)static_cast<const int32_t*>(t.p)[i];
}
// Elements by which p lies past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// ------------------------------------------------------------------ forward
constexpr int kFwdThreads = 256;
template <bool ANY>
constexpr int kFwdUnroll = ANY ? 1 : 4;

// Items are (row, piece of 8 columns).  ANY: rows of w or y are not on 16 bytes;
// pieces then lie on y's boundaries, and the first of a row starts before it.
template <typename TW, typename TY, bool ANY>
__global__ __launch_bounds__(kFwdThreads) void embed_fwd_kernel(const __grid_constant__ EmbedFwd a, int pieces,
                                                                int64_t items) {
  start();
  constexpr int kPer = 16 / (int)sizeof(TY), U = kFwdUnroll<ANY>;
  const TW* w = static_cast<const TW*>(a.w);
  const TW* hi = w + (a.vocab - 1) * a.ldw + a.cols;
  const int64_t first = (int64_t)blockIdx.x * (kFwdThreads * U) + threadIdx.x;
  int64_t row[U], token[U];
  int c[U];
  int64_t r = items <= 0xFFFF0000ll ? (int64_t)((uint32_t)first / (uint32_t)pieces) : first / pieces;
  int piece = (int)(first - r * pieces);
  const int step_rows = kFwdThreads / pieces, step_pieces = kFwdThreads % pieces;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    row[u] = r;
    token[u] = r < a.tokens.count ? load_token(a.tokens, r) : -1;
    c[u] = piece * 8;
    piece += step_pieces, r += step_rows;
    if (piece >= pieces) piece -= pieces, ++r;
  }
  Raw<TW, 8> v[U];
  AnyLoad<TW, 8> any[U];
  const TW* from[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (ANY) c[u] -= phase_of(static_cast<const TY*>(a.y) + row[u] * a.ldy) % kPer;
    const bool in = token[u] >= 0 && token[u] < a.vocab;
    from[u] = w + (in ? token[u] : 0) * a.ldw + c[u];
    if constexpr (ANY)
      any[u].begin(from[u], in && c[u] >= 0 ? a.cols - c[u] : 0, w, hi);
    else
      v[u] = load_raw<8>(from[u], in ? a.cols - c[u] : 0);
  }
  if constexpr (ANY) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = token[u] >= 0 && token[u] < a.vocab;
      v[u] = any[u].end(from[u], in && c[u] >= 0 ? a.cols - c[u] : 0);
      if (in && c[u] < 0) {
        // a row's first elements, at the end of the piece
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c[u] + i >= 0 && c[u] + i < a.cols) {
            if constexpr (sizeof(TW) == 2)
              v[u].w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(from[u])[i] << (16 * (i % 2));
            else
              v[u].w[i] = reinterpret_cast<const uint32_t*>(from[u])[i];
          }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= a.tokens.count) continue;
    float f[8];
    to_floats(v[u], f);
    const float scale = token[u] < a.vocab ? a.scale : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = token[u] < 0 ? 0.0f : f[i] * scale;
    TY* y = static_cast<TY*>(a.y) + row[u] * a.ldy + c[u];
    if (c[u] >= 0) {
      store_part<8>(y, a.cols - c[u], f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c[u] + i >= 0 && c[u] + i < a.cols) y[i] = (TY)f[i];
    }
  }
}

// ------------------------------------------------------------------ sorting
// A block owns kSortRows tokens at most and reads all positions, counting how often
// each of its own occurs in each warp's share of them and how many tokens are below
// its first: that gives every one of its entries a place of its own, without waiting
// for another block.  All blocks reading all tokens is 152 x 8 bytes a token out of
// L2 for tables of up to 152 x kSortRows = 53504 rows, as much as a row of dy is out of
// memory; past that a block more for every kSortRows rows, and it is vocab / 44 bytes a
// token (alone, from 65536 tokens: 50304 rows 17 us, 131072 35, 262144 50; from 8192 8
// and 22).  Several passes of a radix sort would each be a launch.  What a warp finds it keeps, in order, up to kSortKept; only a warp
// that finds more (a very common token) reads its share again.
// (tokens is no __restrict__ pointer: the grid may start while an earlier kernel still
// writes them, so they are no data that stays as it is from start to end.)
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortUnroll = 16;
constexpr int kSortRows = 352, kSortKept = 256;  // 44 KB of counts, 64 KB
static_assert(kSortRows <= kSortThreads && kSortWarps <= 32, "a thread for each token, a lane for each warp");

template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_tokens_kernel(const I* tokens, int64_t count,
                                                                   int64_t vocab, int rows, int4* entries,
                                                                   int* starts, int* arrived, int64_t arrivals) {
  extern __shared__ __align__(8) int counts[];  // [kSortWarps][rows], rows even
  int2* const kept_of = reinterpret_cast<int2*>(counts + kSortWarps * rows);  // [kSortWarps][kSortKept]
  __shared__ int below_of[kSortWarps], sums[kSortWarps];
  __shared__ int2 range[kSortRows];  // of a token's entries
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = (int64_t)blockIdx.x * rows;
  const int mine = (int)min((int64_t)rows, vocab - lo);
  for (int i = threadIdx.x; i < kSortWarps * rows; i += kSortThreads) counts[i] = 0;
  start();
  const int64_t all = (int64_t)gridDim.x * kSortThreads;
  for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < arrivals; i += all) arrived[i] = 0;
  __syncthreads();
  const int64_t share = (count + kSortThreads - 1) / kSortThreads * 32;
  const int64_t begin = min(count, warp * share), end = min(count, begin + share);
  int* own = counts + warp * rows;
  int2* kept = kept_of + warp * kSortKept;
  int below = 0, found = 0;
  for (int64_t i = begin; i < end; i += 32 * kSortUnroll) {
    I t[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) t[u] = i + u * 32 + lane < end ? tokens[i + u * 32 + lane] : (I)-1;
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const bool valid = t[u] >= 0 && (int64_t)t[u] < vocab;
      const int d = (int)((uint32_t)t[u] - (uint32_t)lo);
      below += valid && d < 0;
      const bool in = valid && (uint32_t)d < (uint32_t)mine;
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, in);
      if (!all) continue;
      if (in) {
        atomicAdd(&own[d], 1);
        const int at = found + __popc(all & ((1u << lane) - 1));
        if (at < kSortKept) kept[at] = make_int2((int)(i + u * 32 + lane), d);
      }
      found += __popc(all);
    }
  }
  below = __reduce_add_sync(0xFFFFFFFFu, below);
  if (lane == 0) below_of[warp] = below;
  __syncthreads();
  // counts become offsets: within a token by warp, then by token
  int total = 0;
  if ((int)threadIdx.x < rows) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = counts[w * rows + threadIdx.x];
      counts[w * rows + threadIdx.x] = total;
      total += n;
    }
  }
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += n;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  const int before = __reduce_add_sync(0xFFFFFFFFu, lane < kSortWarps ? below_of[lane] : 0);
  const int base = before + scan - total + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[lane] : 0);
  if ((int)threadIdx.x < rows) range[threadIdx.x] = make_int2(base, base + total);
  if ((int)threadIdx.x < mine) starts[lo + threadIdx.x] = base;
  if (lo + mine == vocab && (int)threadIdx.x == mine - 1) starts[vocab] = base + total;
  __syncthreads();
  // 32 positions' entries, in their order; d: the place of its token, or -1
  auto place = [&](int position, int d) {
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
    const int rank = __popc(same & ((1u << lane) - 1));
    const int at = d >= 0 ? own[d] + rank : 0;
    __syncwarp();
    if (d >= 0) {
      const int2 r = range[d];
      entries[r.x + at] = make_int4(position, (int)(lo + d), r.x, r.y);
      if ((same >> lane) == 1u) own[d] = at + 1;
    }
    __syncwarp();
  };
  if (found <= kSortKept) {
    for (int k = 0; k < found; k += 32) {
      const int2 e = k + lane < found ? kept[k + lane] : make_int2(0, -1);
      place(e.x, e.y);
    }
    return;
  }
  constexpr int kAgain = 8;
  for (int64_t i = begin; i < end; i += 32 * kAgain) {
    I t[kAgain];
#pragma unroll
    for (int u = 0; u < kAgain; ++u) t[u] = i + u * 32 + lane < end ? tokens[i + u * 32 + lane] : (I)-1;
#pragma unroll
    for (int u = 0; u < kAgain; ++u) {
      const bool in = (int64_t)t[u] >= lo && (int64_t)t[u] < lo + mine;
      if (__any_sync(0xFFFFFFFFu, in)) place((int)(i + u * 32 + lane), in ? (int)((int64_t)t[u] - lo) : -1);
    }
  }
}

// ------------------------------------------------------------------ sums
template <typename T, int VEC>
__device__ __forceinline__ void put(T* p, int n, bool aligned, const float (&v)[VEC]) {
  if (n >= VEC && aligned) {
    if constexpr (VEC == 8) {
      store_vec<8>(p, v);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = (T)v[i];
  }
}

constexpr int kTileThreads = 160;  // at most: 16 x 161 x 16 bytes stay below 48 KB

// Zeros for one warp's row of any alignment.
template <typename T>
__device__ __forceinline__ void zero_row(T* p, int cols, int lane) {
  constexpr int kPer = 16 / (int)sizeof(T);
  const int head = min(cols, (kPer - phase_of(p)) % kPer);
  if (lane < head) p[lane] = (T)0.0f;
  const int body = (cols - head) / kPer;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int i = lane; i < body; i += 32) q[i] = make_uint4(0, 0, 0, 0);
  const int tail = cols - head - body * kPer;
  if (lane < tail) p[cols - tail + lane] = (T)0.0f;
}

// Blocks write rows of zeros, or add up some columns of a tile's entries: those of the
// tokens that start in it.  A long token, one that reaches over more than kPart tiles,
// is cut into parts of as many, from the tile where it starts on, each summed by the
// block of its first tile and left in `partial`; of every few parts the block that is
// done last (nobody waits) adds them up in their order, whichever it is.  So a common
// word is spread over blocks.  (Parts of 4 tiles: with 2 a padded batch's common token
// has more to join, 32000 x 1280 from 16384 tokens 45 -> 48 us, with 8 the sums take
// longer, 38 -> 45 for 50304 x 1024 from 8192.  A launch of its own to join them was
// 0.5 to 1.5 us slower for these and 5 for 50304 x 1024 in float32.  All of a token's
// parts by one block: 32000 x 512 from 65536 tokens 51 us, by eights 42.2, by sixteens
// 43.8; there a token of 9 to 16 parts needs one step less, 50304 x 1024 28.2 for 29.2.)
constexpr int kPart = 4, kStage = 8;
constexpr int kWindow = kPart * kEmbedTile;  // entries that a tile's block may go through
static_assert(kWindow == 64, "a bit for each, in words of 32");
constexpr int kGroup = 8, kLevels = kPart;  // of joining a long token's parts
// Of a token's entries [x, y).
__device__ __forceinline__ int parts_of(int2 e) { return ((e.y - 1) / kEmbedTile - e.x / kEmbedTile) / kPart + 1; }

template <typename TD, typename TG, bool ANY>
__global__ __launch_bounds__(kTileThreads) void embed_sum_kernel(const __grid_constant__ EmbedBwd a, int fill,
                                                                 int fill_rows, int chunks, bool dw16, uint32_t sms) {
  start();
  constexpr int VEC = 16 / (int)sizeof(TD);
  extern __shared__ __align__(16) uint4 staged[];  // [2][kStage][pitch]
  __shared__ uintptr_t address[kWindow];  // of the block's columns in an entry's row
  __shared__ int token[kWindow];
  __shared__ int2 ends[2];  // where the tile's first and last entry's tokens start and end
  __shared__ int is_last;
  TG* dw = static_cast<TG*>(a.dw);
  // tiles and rows of zeros in turn, as long as there are both: the ones wait for
  // loads, the others use what bandwidth is left.  (Blocks go round the SMs, of which
  // there is an even number: every round begins with the other kind.)
  const int sums = (int)gridDim.x - fill, both = 2 * min(sums, fill);
  const bool is_sum = (int)blockIdx.x < both ? (blockIdx.x + blockIdx.x / sms) % 2 == 0 : sums > fill;
  const int job = (int)blockIdx.x < both ? blockIdx.x / 2 : (int)blockIdx.x - both / 2;
  if (!is_sum) {
    const int lane = threadIdx.x & 31;
    const int64_t v0 = ((int64_t)job * (blockDim.x >> 5) + (threadIdx.x >> 5)) * fill_rows;
    const bool none = lane < fill_rows && v0 + lane < a.vocab && a.starts[v0 + lane] == a.starts[v0 + lane + 1];
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, none); left; left &= left - 1)
      zero_row(dw + (v0 + __ffs(left) - 1) * a.lddw, a.cols, lane);
    return;
  }
  const int tile = job / chunks, chunk = job % chunks;
  const int i0 = tile * kEmbedTile;
  const int cs = chunk * (int)blockDim.x * VEC;
  const TD* dy = static_cast<const TD*>(a.dy);
  const int valid = a.starts[a.vocab], last = min(valid - 1, i0 + kEmbedTile - 1) - i0;
  for (int i = threadIdx.x; i < kWindow; i += blockDim.x) {
    // (there are count entries, of which the first `valid` mean something)
    int4 e = i0 + i < a.tokens.count ? a.entries[i0 + i] : make_int4(0, -1, 0, 0);
    if (i0 + i >= valid) e.y = -1;
    address[i] = reinterpret_cast<uintptr_t>(dy + (int64_t)e.x * a.lddy + cs);
    token[i] = e.y;
    if (i == 0) ends[0] = make_int2(e.z, e.w);
    if (i == last) ends[1] = make_int2(e.z, e.w);
  }
  if (last < 0) return;
  __syncthreads();
  const int i1 = i0 + last + 1;
  const int2 head = ends[0], tail = ends[1];
  const int head_parts = parts_of(head), tail_parts = parts_of(tail);
  const bool head_long = head_parts > 1, tail_long = tail_parts > 1;
  // the first token: its part from here on, or nothing if it is another block's
  const bool head_here = head.x >= i0 || (head_long && (tile - head.x / kEmbedTile) % kPart == 0);
  const int begin = head_here ? i0 : min(head.y, i1);
  int end = tail.x >= i0 || begin < i1 ? min(tail.y, i0 + kWindow) : begin;
  if (tail.x < i0 && !head_here) end = begin;  // all of the tile is that token's
  // bit i: entry i0 + i is its token's last here
  uint64_t lasts = 0;
#pragma unroll
  for (int h = 0; h < kWindow; h += 32) {
    const int i = h + ((int)threadIdx.x & 31);
    lasts |= (uint64_t)__ballot_sync(0xFFFFFFFFu, i + 1 >= kWindow || token[i] != token[i + 1]) << h;
  }
  lasts |= 1ull << ((end - 1 - i0) & 63);
  const int c0 = cs + (int)threadIdx.x * VEC;
  const int mine = a.cols - c0;  // may be 0 or less
  // a row's columns from their sum
  auto write = [&](int v, float (&acc)[VEC]) {
    TG* p = dw + (int64_t)v * a.lddw + c0;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      acc[k] *= a.scale;
      if (a.accumulate && k < mine) acc[k] += (float)p[k];
    }
    put<TG, VEC>(p, mine, dw16, acc);
  };
  uint64_t sum[VEC / 2];  // pairs
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) sum[i] = 0;
  // kStage entries' rows are on their way while as many are added up, every thread's
  // piece at a place of its own.  ANY: the rows are on no 16-byte boundaries; what the
  // block's columns lie in is copied from the boundary before them on, a piece more
  // than there are threads, and a thread's values are put together from two pieces.
  const int pitch = (int)blockDim.x + (ANY ? 1 : 0);
  const uint32_t width = min(a.cols - cs, (int)blockDim.x * VEC) * (uint32_t)sizeof(TD);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(dy);
  const uintptr_t hi = reinterpret_cast<uintptr_t>(dy + (a.tokens.count - 1) * a.lddy + a.cols);
  auto copy = [&](const uint4* to, uintptr_t from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "r"(bytes)
                 : "memory");
  };
  auto stage = [&](int at, int half) {
    uint4* to = staged + half * kStage * pitch;
    const int n = min(kStage, end - at);
    for (int l = 0; l < n; ++l, to += pitch) {
      const uintptr_t row = address[at - i0 + l];
      if constexpr (!ANY) {
        if (mine > 0) copy(to + threadIdx.x, row + threadIdx.x * 16, min(mine, VEC) * (int)sizeof(TD));
      } else {
        const uint32_t off = (uint32_t)row & 15u;
        for (uint32_t j = threadIdx.x; j <= blockDim.x && j * 16 < off + width; j += blockDim.x) {
          const uintptr_t from = row - off + j * 16;
          if (from >= lo) {
            copy(to + j, from, (int)min((uint64_t)16, (uint64_t)(hi - from)));
          } else {
            // the matrix starts inside this piece
            for (int k = 0; k < VEC; ++k)
              if (from + k * sizeof(TD) >= lo && from + k * sizeof(TD) < hi)
                reinterpret_cast<TD*>(to + j)[k] = reinterpret_cast<const TD*>(from)[k];
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  stage(begin, 0);
  int half = 0;
  for (int at = begin; at < end; at += kStage, half ^= 1) {
    const int n = min(kStage, end - at);
    if (ANY) __syncthreads();  // the other half has been read
    stage(at + kStage, half ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (ANY) __syncthreads();
    const uint4* from = staged + half * kStage * pitch + threadIdx.x;
    for (int l = 0; l < n; ++l, from += pitch) {
      if (mine <= 0) break;
      const uint4 u = *from;
      Raw<TD, VEC> r;
      if constexpr (ANY) {
        const uint4 next = from[1];
        const uint32_t off = (uint32_t)address[at + l - i0] & 15u;
        uint32_t w[8] = {u.x, u.y, u.z, u.w, next.x, next.y, next.z, next.w};
        if (off & 8) {
#pragma unroll
          for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
        }
        if (off & 4) {
#pragma unroll
          for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r.w[j] = sizeof(TD) == 4 ? w[j] : __funnelshift_r(w[j], w[j + 1], (off & 2) * 8);
      } else {
        r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
      }
      float f[VEC];
      to_floats(r, f);
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) sum[i] = add2(sum[i], pair(f[2 * i], f[2 * i + 1]));
      const int i = at + l;
      if (!(lasts >> (i - i0) & 1)) continue;
      const int v = token[i - i0];
      float acc[VEC];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        unpair(sum[k], acc[2 * k], acc[2 * k + 1]);
        sum[k] = 0;
      }
      const bool of_head = i < head.y;
      if (of_head ? !head_long : i < tail.x || !tail_long) {
        write(v, acc);
      } else {
        // first the sum of what started before the tile, second of what starts in it
        float* p = a.partial + ((int64_t)tile * 2 + (of_head && head.x < i0 ? 0 : 1)) * a.partial_pitch + c0;
        put<float, VEC>(p, VEC, true, acc);
      }
    }
  }
  // A long token of which a part is done.  Parts are joined by eights, the eighths' sums
  // by eights again, and so on, each time by the block that comes last: its sum takes
  // the place of the first.  A group of two or more counts in its first part's first
  // tile, a level's at as many tiles further on: that part is not the token's last, so
  // its kPart tiles are all there and no other token counts in them.
  auto join = [&](int v, const int2& e, int units, int unit) {
    const int t0 = e.x / kEmbedTile;
    for (int level = 0, width = 1;; ++level, width *= kGroup) {
      const int first = level < kLevels - 1 ? unit / kGroup * kGroup : 0;
      const int count = level < kLevels - 1 ? min(kGroup, units - first) : units;
      unit /= kGroup;
      if (count == 1) {  // its sum stays where it is
        units = (units + kGroup - 1) / kGroup;
        continue;
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        is_last = atomicAdd(&a.arrived[((int64_t)t0 + (int64_t)first * width * kPart + level) * chunks + chunk], 1) ==
                  count - 1;
      __syncthreads();
      if (!is_last) return;
      __threadfence();
      float acc[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
      auto place = [&](int k) {  // of the k-th unit's sum
        return a.partial + (((int64_t)t0 + (int64_t)k * width * kPart) * 2 + (k == 0 ? 1 : 0)) * a.partial_pitch + c0;
      };
      if (mine > 0) {
#pragma unroll 8
        for (int k = first; k < first + count; ++k) {
          const float* p = place(k);
#pragma unroll
          for (int i = 0; i < VEC; i += 4) {
            const float4 q = __ldcg(reinterpret_cast<const float4*>(p + i));
            acc[i] += q.x, acc[i + 1] += q.y, acc[i + 2] += q.z, acc[i + 3] += q.w;
          }
        }
        if (count == units)
          write(v, acc);
        else
          put<float, VEC>(place(first), VEC, true, acc);
      }
      if (count == units) return;
      units = (units + kGroup - 1) / kGroup;
    }
  };
  if (head_long && head_here) join(token[0], head, head_parts, (tile - head.x / kEmbedTile) / kPart);
  if (tail_long && tail.x >= i0 && tail.x > head.x) join(token[last], tail, tail_parts, 0);
}

// ------------------------------------------------------------------ launches
template <typename TW, typename TY>
cudaError_t run_embedding(const EmbedFwd& a, cudaStream_t st) {
  const bool vec = rows16(a.w, a.ldw, sizeof(TW)) && rows16(a.y, a.ldy, sizeof(TY));
  // pieces of a row, with room for one that starts before it
  const int pieces = (int)(vec ? ceil_div(a.cols, 8) : ceil_div((int64_t)a.cols + 16 / (int)sizeof(TY) - 1, 8));
  const int64_t items = a.tokens.count * pieces, blocks = ceil_div(items, kFwdThreads * (vec ? kFwdUnroll<false> : kFwdUnroll<true>));
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(vec ? embed_fwd_kernel<TW, TY, false> : embed_fwd_kernel<TW, TY, true>, (unsigned)blocks,
                       kFwdThreads, 0, 0, st, a, pieces, items);
}

template <typename TD, typename TG>
cudaError_t run_embedding_bwd(const EmbedBwd& a, cudaStream_t st) {
  constexpr int VEC = 16 / (int)sizeof(TD);
  const int64_t vecs = ceil_div(a.cols, VEC), tiles = ceil_div(a.tokens.count, kEmbedTile);
  // equal chunks of at most kTileThreads pieces
  const int64_t parts = ceil_div(vecs, kTileThreads);
  const int threads = (int)(ceil_div(ceil_div(vecs, parts), 32) * 32);
  const int64_t chunks = ceil_div(vecs, threads);
  const int rows = (int)std::min<int64_t>(kSortRows, ceil_div(ceil_div(a.vocab, sm_count()), 2) * 2);
  const unsigned sorters = (unsigned)ceil_div(a.vocab, rows);
  const int bytes = kSortWarps * (rows * 4 + kSortKept * 8);
  auto sort = [&](auto* kernel, auto* tokens) {
    cudaError_t e = cudaSuccess;
    if (bytes > 44 * 1024) e = allow_smem((const void*)kernel, bytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, sorters, kSortThreads, (size_t)bytes, 0, st, tokens, a.tokens.count, a.vocab, rows,
                         a.entries, a.starts, a.arrived, tiles * chunks);
  };
  cudaError_t e = a.tokens.bytes == 8 ? sort(sort_tokens_kernel<int64_t>, static_cast<const int64_t*>(a.tokens.p))
                                      : sort(sort_tokens_kernel<int32_t>, static_cast<const int32_t*>(a.tokens.p));
  if (e != cudaSuccess) return e;
  // Rows of zeros a warp: enough to be worth a block's launch (77248 rows of 64 in
  // bfloat16 for 592 tokens: one a warp 86 us, 16 a warp 17; 50304 of 1024 for 8192 spread
  // evenly: one 28, two 25), and no more, as few warps have few stores in flight (32000 of 2048
  // for 1000: one 26, 32 a warp 58).
  const int fill_rows = (int)std::min<int64_t>(16, std::max<int64_t>(1, 4096 / ((int64_t)a.cols * (int)sizeof(TG))));
  const int64_t fill = a.accumulate ? 0 : ceil_div(a.vocab, fill_rows * (threads / 32));
  if (tiles * chunks + fill > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool any = !rows16(a.dy, a.lddy, sizeof(TD));
  const size_t smem = (size_t)2 * kStage * (threads + (any ? 1 : 0)) * 16;
  // whether VEC of the output's elements can be stored together
  const bool dw16 = aligned(a.dw, std::min<size_t>(16, VEC * sizeof(TG))) &&
                    (a.lddw * sizeof(TG)) % std::min<size_t>(16, VEC * sizeof(TG)) == 0;
  return launch_kernel(any ? embed_sum_kernel<TD, TG, true> : embed_sum_kernel<TD, TG, false>,
                       (unsigned)(tiles * chunks + fill), threads, smem, 0, st, a, (int)fill, fill_rows, (int)chunks,
                       dw16, (uint32_t)(sm_count() / 2 * 2));
}

}  // namespace

int64_t embed_partial_pitch(int64_t cols) { return ceil_div(cols, 8) * 8; }
// of pieces of 4 elements (float32 gradients; of 8, half as many)
int64_t embed_chunks_most(int64_t cols) { return ceil_div(ceil_div(cols, 4), kTileThreads); }

cudaError_t launch_embedding(const EmbedFwd& a, int w_dtype, int dtype, cudaStream_t st) {
  if (w_dtype == SCAPE_BF16)
    return dtype == SCAPE_BF16 ? run_embedding<bf16, bf16>(a, st) : run_embedding<bf16, float>(a, st);
  return dtype == SCAPE_BF16 ? run_embedding<float, bf16>(a, st) : run_embedding<float, float>(a, st);
}
cudaError_t launch_embedding_bwd(const EmbedBwd& a, int dtype, int dw_dtype, cudaStream_t st) {
  if (dtype == SCAPE_BF16)
    return dw_dtype == SCAPE_BF16 ? run_embedding_bwd<bf16, bf16>(a, st) : run_embedding_bwd<bf16, float>(a, st);
  return dw_dtype == SCAPE_BF16 ? run_embedding_bwd<float, bf16>(a, st) : run_embedding_bwd<float, float>(a, st);
}

}  // namespace layer
}  // namespace scapek
