// layer_embedding.cu -- rows of a table by token, and the table's gradient.
//
// Forward: y[i] = scale w[token i].  Bound by memory; a thread takes several pieces
// of 8 columns so that their loads are in flight together.
//
// Gradient: dw[v] = scale * sum of the dy rows of token v.  Atomics on dw would add
// in an order that changes, and in the output's type.  So the positions are sorted by
// token (stable: integers only), cut into tiles of kEmbedTile that blocks add up in
// 32 bits; a token whose positions reach over tiles leaves partial sums, joined in
// the tiles' order by a last launch.  Most rows of a large table have no token, and
// writing their zeros is most of the bytes: that goes on beside the sums.
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
constexpr int kFwdThreads = 256, kFwdUnroll = 4;

// Items are (row, piece of 8 columns).  ANY: rows of w or y are not on 16 bytes;
// pieces then lie on y's boundaries, and the first of a row starts before it.
template <typename TW, typename TY, bool ANY>
__global__ __launch_bounds__(kFwdThreads) void embed_fwd_kernel(const __grid_constant__ EmbedFwd a, int pieces,
                                                                int64_t items) {
  start();
  constexpr int kPer = 16 / (int)sizeof(TY);
  const TW* w = static_cast<const TW*>(a.w);
  const TW* hi = w + (a.vocab - 1) * a.ldw + a.cols;
  const int64_t first = (int64_t)blockIdx.x * (kFwdThreads * kFwdUnroll) + threadIdx.x;
  int64_t row[kFwdUnroll], token[kFwdUnroll];
  int c[kFwdUnroll];
  int64_t r = items <= 0xFFFFFFFFll ? (int64_t)((uint32_t)first / (uint32_t)pieces) : first / pieces;
  int piece = (int)(first - r * pieces);
  const int step_rows = kFwdThreads / pieces, step_pieces = kFwdThreads % pieces;
#pragma unroll
  for (int u = 0; u < kFwdUnroll; ++u) {
    row[u] = r;
    token[u] = r < a.tokens.count ? load_token(a.tokens, r) : -1;
    c[u] = piece * 8;
    piece += step_pieces, r += step_rows;
    if (piece >= pieces) piece -= pieces, ++r;
  }
  Raw<TW, 8> v[kFwdUnroll];
#pragma unroll
  for (int u = 0; u < kFwdUnroll; ++u) {
    if (ANY) c[u] -= phase_of(static_cast<const TY*>(a.y) + row[u] * a.ldy) % kPer;
    const bool in = token[u] >= 0 && token[u] < a.vocab;
    const TW* p = w + (in ? token[u] : 0) * a.ldw + c[u];
    if constexpr (ANY) {
      if (in && c[u] >= 0) {
        v[u] = load_any<8>(p, max(0, min(8, a.cols - c[u])), w, hi);
      } else {
        // a row's first elements, at the end of the piece
#pragma unroll
        for (int i = 0; i < Raw<TW, 8>::kWords; ++i) v[u].w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in && c[u] + i >= 0 && c[u] + i < a.cols) {
            if constexpr (sizeof(TW) == 2)
              v[u].w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
            else
              v[u].w[i] = reinterpret_cast<const uint32_t*>(p)[i];
          }
      }
    } else {
      v[u] = load_raw<8>(p, in ? a.cols - c[u] : 0);
    }
  }
#pragma unroll
  for (int u = 0; u < kFwdUnroll; ++u) {
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
// L2, as much as a row of dy is out of memory; several passes of a radix sort would
// each be a launch.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortUnroll = 16;
constexpr int kSortRows = 352;  // 44 KB of counts

template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_tokens_kernel(const I* __restrict__ tokens, int64_t count,
                                                                   int64_t vocab, int rows, int2* entries,
                                                                   int* starts) {
  extern __shared__ int counts[];  // [kSortWarps][rows]
  __shared__ int below_of[kSortWarps], sums[kSortWarps], first[kSortRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = (int64_t)blockIdx.x * rows;
  const int mine = (int)min((int64_t)rows, vocab - lo);
  for (int i = threadIdx.x; i < kSortWarps * rows; i += kSortThreads) counts[i] = 0;
  start();
  __syncthreads();
  const int64_t share = (count + kSortThreads - 1) / kSortThreads * 32;
  const int64_t begin = min(count, warp * share), end = min(count, begin + share);
  int* own = counts + warp * rows;
  int d[kSortUnroll];  // places of 32 x kSortUnroll tokens among this block's, or -1
  auto read = [&](int64_t i, int& below) {
    I t[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) t[u] = i + u * 32 + lane < end ? tokens[i + u * 32 + lane] : (I)-1;
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const int64_t at = (int64_t)t[u] - lo;
      below += t[u] >= 0 && at < 0;
      d[u] = at >= 0 && at < mine ? (int)at : -1;
    }
  };
  int below = 0;
  for (int64_t i = begin; i < end; i += 32 * kSortUnroll) {
    read(i, below);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u)
      if (d[u] >= 0) atomicAdd(&own[d[u]], 1);
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
  const int before = __reduce_add_sync(0xFFFFFFFFu, below_of[lane]);
  const int base = before + scan - total + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[lane] : 0);
  if ((int)threadIdx.x < rows) first[threadIdx.x] = base;
  if ((int)threadIdx.x < mine) starts[lo + threadIdx.x] = base;
  if (lo + mine == vocab && (int)threadIdx.x == mine - 1) starts[vocab] = base + total;
  __syncthreads();
  for (int64_t i = begin; i < end; i += 32 * kSortUnroll) {
    if (end - begin > 32 * kSortUnroll) read(i, below);  // else they are still there
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      if (!__any_sync(0xFFFFFFFFu, d[u] >= 0)) continue;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, d[u]);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int at = d[u] >= 0 ? own[d[u]] + rank : 0;
      __syncwarp();
      if (d[u] >= 0) {
        entries[first[d[u]] + at] = make_int2((int)(i + u * 32 + lane), (int)(lo + d[u]));
        if ((same >> lane) == 1u) own[d[u]] = at + 1;
      }
      __syncwarp();
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

constexpr int kTileThreads = 160;  // at most: 16 x 160 x 16 bytes stay below 48 KB

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

// The first blocks write zeros, the others each add up some columns of a tile's
// entries: those of the tokens that start in it, and, of a token with more than
// kLong entries, the tile's own part, which goes to `partial` for the join.  So a
// common word's entries are spread over blocks and few tokens need a join.
constexpr int kLong = 2 * kEmbedTile;

template <typename TD, typename TG, bool ANY>
__global__ __launch_bounds__(kTileThreads) void embed_sum_kernel(const __grid_constant__ EmbedBwd a, int fill,
                                                                 int chunks, bool dw16) {
  start();
  constexpr int VEC = 16 / (int)sizeof(TD);
  extern __shared__ __align__(16) uint4 staged[];  // [kEmbedTile][threads]
  __shared__ int position[kEmbedTile + kLong], token[kEmbedTile + kLong];
  __shared__ int ends[4];  // where the first and the last entry's tokens start and end
  TG* dw = static_cast<TG*>(a.dw);
  if ((int)blockIdx.x < fill) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t v0 = ((int64_t)blockIdx.x * warps + (threadIdx.x >> 5)) * 32;
    if (v0 >= a.vocab) return;
    const bool none = v0 + lane < a.vocab && a.starts[v0 + lane] == a.starts[v0 + lane + 1];
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, none); left; left &= left - 1)
      zero_row(dw + (v0 + __ffs(left) - 1) * a.lddw, a.cols, lane);
    return;
  }
  const int tile = ((int)blockIdx.x - fill) / chunks, chunk = ((int)blockIdx.x - fill) % chunks;
  const int valid = a.starts[a.vocab], i0 = tile * kEmbedTile;
  const int i1 = min(i0 + kEmbedTile, valid);
  if (i0 >= valid) {
    if (chunk == 0 && threadIdx.x == 0) a.crossing[tile] = -1;
    return;
  }
  for (int i = threadIdx.x; i < kEmbedTile + kLong; i += blockDim.x) {
    const int2 e = i0 + i < valid ? a.entries[i0 + i] : make_int2(0, -1);
    position[i] = e.x;
    token[i] = e.y;
  }
  if (threadIdx.x < 4) {
    const int64_t v = a.entries[threadIdx.x < 2 ? i0 : i1 - 1].y;
    ends[threadIdx.x] = a.starts[v + (threadIdx.x & 1)];
  }
  __syncthreads();
  // entries of a short token go with the tile where it starts
  const bool first_before = ends[0] < i0, first_long = ends[1] - ends[0] > kLong;
  const bool last_long = ends[3] - ends[2] > kLong;
  const int begin = first_before && !first_long ? min(ends[1], i1) : i0;
  const int end = last_long || ends[2] < i0 ? i1 : ends[3];
  if (chunk == 0 && threadIdx.x == 0) a.crossing[tile] = last_long && ends[2] >= i0 ? token[i1 - 1 - i0] : -1;
  const int c0 = (chunk * (int)blockDim.x + (int)threadIdx.x) * VEC;
  const int mine = a.cols - c0;
  if (mine <= 0) return;
  const TD* dy = static_cast<const TD*>(a.dy);
  const TD* hi = dy + (a.tokens.count - 1) * a.lddy + a.cols;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  for (int at = begin; at < end; at += kEmbedTile) {
    const int n = min(kEmbedTile, end - at);
    if constexpr (ANY) {
#pragma unroll 8
      for (int l = 0; l < n; ++l) {
        const Raw<TD, VEC> r =
            load_any<VEC>(dy + (int64_t)position[at - i0 + l] * a.lddy + c0, min(mine, VEC), dy, hi);
        staged[l * blockDim.x + threadIdx.x] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
      }
    } else {
      const int bytes = min(mine, VEC) * (int)sizeof(TD);
      for (int l = 0; l < n; ++l) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(&staged[l * blockDim.x + threadIdx.x]);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                     "l"(dy + (int64_t)position[at - i0 + l] * a.lddy + c0), "r"(bytes)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    }
    for (int l = 0; l < n; ++l) {
      const uint4 u = staged[l * blockDim.x + threadIdx.x];
      Raw<TD, VEC> r;
      r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
      float f[VEC];
      to_floats(r, f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += f[i];
      const int i = at + l, v = token[i - i0];
      if (i + 1 < end && token[i + 1 - i0] == v) continue;
      // a long token's sum is whole where it starts and ends in this tile's entries only
      const bool from_first = i < ends[1];
      const bool part = (from_first && first_long) || (i + 1 == end && last_long);
      if (!part) {
        TG* p = dw + (int64_t)v * a.lddw + c0;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          acc[k] *= a.scale;
          if (a.accumulate && k < mine) acc[k] += (float)p[k];
        }
        put<TG, VEC>(p, mine, dw16, acc);
      } else {
        // first the sum of what started before the tile, second of what starts in it
        float* p = a.partial + ((int64_t)tile * 2 + (from_first && first_before ? 0 : 1)) * a.partial_pitch + c0;
        put<float, VEC>(p, VEC, true, acc);
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] = 0.0f;
    }
  }
}

// ------------------------------------------------------------------ joining
// Item (tile, 128 columns): the sum of the long token that starts in the tile.  A
// block first looks at all its items' tiles.
constexpr int kJoinThreads = 256, kJoinCols = 128;

template <typename TG>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(const __grid_constant__ EmbedBwd a, int tiles,
                                                                  int chunks, bool dw8) {
  start();
  __shared__ float4 part[kJoinThreads / 32][32];
  __shared__ int found[kJoinThreads], found_tile[kJoinThreads], found_chunk[kJoinThreads];
  __shared__ int finds;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t items = (int64_t)tiles * chunks;
  TG* dw = static_cast<TG*>(a.dw);
  for (int64_t base = blockIdx.x; base < items; base += (int64_t)gridDim.x * kJoinThreads) {
    if (threadIdx.x == 0) finds = 0;
    __syncthreads();
    const int64_t my = base + (int64_t)threadIdx.x * gridDim.x;
    if (my < items) {
      const int tile = (int)(my / chunks), v = a.crossing[tile];
      if (v >= 0) {
        const int at = atomicAdd(&finds, 1);  // their order changes nothing
        found[at] = v, found_tile[at] = tile, found_chunk[at] = (int)(my % chunks);
      }
    }
    __syncthreads();
    for (int k = 0; k < finds; ++k) {
      const int v = found[k], tile = found_tile[k], c0 = found_chunk[k] * kJoinCols + lane * 4;
      const int last = (a.starts[v + 1] - 1) / kEmbedTile;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c0 < a.cols) {
#pragma unroll 4
        for (int t = tile + warp; t <= last; t += kJoinThreads / 32) {
          // its part of the tile where it starts is the tile's second sum
          const float4 p = *reinterpret_cast<const float4*>(
              a.partial + ((int64_t)t * 2 + (t == tile ? 1 : 0)) * a.partial_pitch + c0);
          s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
        }
      }
      part[warp][lane] = s;
      __syncthreads();
      if (warp == 0 && c0 < a.cols) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) {
          const float4 p = part[w][lane];
          f[0] += p.x, f[1] += p.y, f[2] += p.z, f[3] += p.w;
        }
        TG* p = dw + (int64_t)v * a.lddw + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] *= a.scale;
          if (a.accumulate && c0 + i < a.cols) f[i] += (float)p[i];
        }
        put<TG, 4>(p, a.cols - c0, dw8, f);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ launches
template <typename TW, typename TY>
cudaError_t run_embedding(const EmbedFwd& a, cudaStream_t st) {
  const bool vec = rows16(a.w, a.ldw, sizeof(TW)) && rows16(a.y, a.ldy, sizeof(TY));
  // pieces of a row, with room for one that starts before it
  const int pieces = (int)(vec ? ceil_div(a.cols, 8) : ceil_div((int64_t)a.cols + 16 / (int)sizeof(TY) - 1, 8));
  const int64_t items = a.tokens.count * pieces, blocks = ceil_div(items, kFwdThreads * kFwdUnroll);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(vec ? embed_fwd_kernel<TW, TY, false> : embed_fwd_kernel<TW, TY, true>, (unsigned)blocks,
                       kFwdThreads, 0, 0, st, a, pieces, items);
}

template <typename TD, typename TG>
cudaError_t run_embedding_bwd(const EmbedBwd& a, cudaStream_t st) {
  const int rows = (int)std::min<int64_t>(kSortRows, ceil_div(a.vocab, sm_count()));
  const unsigned sorters = (unsigned)ceil_div(a.vocab, rows);
  const size_t counts = (size_t)kSortWarps * rows * 4;
  cudaError_t e =
      a.tokens.bytes == 8
          ? launch_kernel(sort_tokens_kernel<int64_t>, sorters, kSortThreads, counts, 0, st,
                          static_cast<const int64_t*>(a.tokens.p), a.tokens.count, a.vocab, rows, a.entries, a.starts)
          : launch_kernel(sort_tokens_kernel<int32_t>, sorters, kSortThreads, counts, 0, st,
                          static_cast<const int32_t*>(a.tokens.p), a.tokens.count, a.vocab, rows, a.entries, a.starts);
  if (e != cudaSuccess) return e;
  constexpr int VEC = 16 / (int)sizeof(TD);
  const int64_t vecs = ceil_div(a.cols, VEC), tiles = ceil_div(a.tokens.count, kEmbedTile);
  // equal chunks of at most kTileThreads pieces
  const int64_t parts = ceil_div(vecs, kTileThreads);
  const int threads = (int)(ceil_div(ceil_div(vecs, parts), 32) * 32);
  const int64_t chunks = ceil_div(vecs, threads);
  const int64_t fill = a.accumulate ? 0 : ceil_div(a.vocab, 32 * (threads / 32));
  if (tiles * chunks + fill > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const size_t smem = (size_t)kEmbedTile * threads * 16;
  const bool any = !rows16(a.dy, a.lddy, sizeof(TD));
  // whether VEC of the output's elements can be stored together
  const bool dw16 = aligned(a.dw, std::min<size_t>(16, VEC * sizeof(TG))) &&
                    (a.lddw * sizeof(TG)) % std::min<size_t>(16, VEC * sizeof(TG)) == 0;
  e = launch_kernel(any ? embed_sum_kernel<TD, TG, true> : embed_sum_kernel<TD, TG, false>,
                    (unsigned)(tiles * chunks + fill), threads, smem, 0, st, a, (int)fill, (int)chunks, dw16);
  if (e != cudaSuccess) return e;
  const int64_t join = ceil_div(a.cols, kJoinCols);
  const bool dw8 = aligned(a.dw, 4 * sizeof(TG)) && (a.lddw * sizeof(TG)) % (4 * sizeof(TG)) == 0;
  return launch_kernel(embed_join_kernel<TG>, (unsigned)std::min<int64_t>(tiles * join, (int64_t)sm_count() * 4),
                       kJoinThreads, 0, 0, st, a, (int)tiles, (int)join, dw8);
}

}  // namespace

int64_t embed_partial_pitch(int64_t cols) { return ceil_div(cols, 8) * 8; }

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
