// layer_gemm.cuh -- bfloat16 matrix product D[M, N] = A B^T on the tensor cores
// (tcgen05, accumulators in tensor memory, operands staged by TMA), with the
// linear layer's epilogues.
//
// A and B are each either contraction-major (row i holds operand row i: [M, K])
// or transposed ([K, M]): the forward product, the input gradient and the weight
// gradient are the three combinations, none of which moves data to transpose it.
// Both forms are staged as 128-byte swizzled rows of 64 values; the difference is
// only in the matrix descriptors.
#pragma once

#include <cuda.h>

#include "layer_internal.cuh"

namespace scapek {
namespace layer {

// ------------------------------------------------------------------ what the host passes
enum GemmKind { kGemmForward = 0, kGemmInputGrad = 1, kGemmWeightGrad = 2 };

struct Epilogue {
  int act;
  // forward: z = acc + bias, q/scale = pack8(z), out = act(z) + res
  const bf16* bias;
  const bf16* res;
  int64_t ldres;
  uint8_t* q;
  int64_t ldq;
  uint8_t* scale;
  // input gradient: out = acc * act'(pre)
  const uint8_t* pre_q;
  int64_t ldpre;
  const uint8_t* pre_scale;
  int64_t blocks_per_row;
  void* out;
  int64_t ldo;
  int out_f32;
  int out_vec, res_vec, q_vec, pre_vec, bias_vec;  // rows (or the vector) aligned for 16 bytes
};

struct GemmOperand {
  const bf16* p;  // 16-byte aligned, ld a multiple of 8
  int64_t ld;
};

// D[m, n] over a contraction of k.  The operands' layouts go by the kind:
//   forward       A = a[m, k]   B = b[n, k]
//   input grad    A = a[m, k]   B = b[k, n]
//   weight grad   A = a[k, m]   B = b[k, n]
struct GemmCall {
  GemmOperand a, b;
  int64_t m, n, k;
  Epilogue e;
};
cudaError_t gemm_forward(const GemmCall& c, cudaStream_t st);
cudaError_t gemm_input_grad(const GemmCall& c, cudaStream_t st);
cudaError_t gemm_weight_grad(const GemmCall& c, cudaStream_t st);

// Where kernels record that they gave up a wait (one word a device).
cudaError_t gemm_status_word(unsigned int** word);

// 2-D tensor map of 64-column, `box_rows`-row boxes with 128-byte swizzle.
cudaError_t gemm_tensor_map(CUtensorMap* map, const bf16* p, int64_t rows, int64_t cols,
                            int64_t ld, int box_rows);

#ifdef __CUDACC__

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// ------------------------------------------------------------------ tiles
constexpr int kBM = 128;   // rows of a tile: the tensor core's 128 accumulator lanes
constexpr int kBK = 64;    // contraction a stage: one 128-byte swizzled row of bfloat16
constexpr int kChunk = 8192;  // bytes of 64 staged rows of 128 bytes
constexpr int kGemmThreads = 384;       // TMA, MMA, TMEM, one idle warp; 8 epilogue warps
constexpr int kEpilogueWarps = 8;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

template <int BN>
struct Tile {
  static constexpr int kABytes = kBM * kBK * 2;
  static constexpr int kBBytes = BN * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int kColumns = 2 * BN;  // two accumulators
  // column stride of the partial tile that split products exchange: odd, and 8
  // columns apart fall 8 banks apart
  static constexpr int kPartialLd = kBM + 1;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static_assert(kPartialLd * BN * 4 <= kStages * kStageBytes, "partial tile fits the stages");
};

// Matrix descriptor of a 128-byte swizzled operand.  Contraction-major: 8-row
// groups 1024 bytes apart (stride field).  Transposed: 8 contraction rows are
// 1024 bytes (stride field), the next 64 operand rows kChunk away (leading field).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool transposed) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(transposed ? kChunk >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of this architecture
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
template <int BN, bool TA, bool TB>
__device__ __forceinline__ constexpr uint32_t instr_desc() {
  return (1u << 4)            // 32-bit float accumulator
         | (1u << 7)          // A bfloat16
         | (1u << 10)         // B bfloat16
         | ((TA ? 1u : 0u) << 15) | ((TB ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)(kBM >> 4) << 24);
}

// ------------------------------------------------------------------ epilogue
// N neighbouring accumulators of one row from column c0 on; `left` = columns
// that exist from there.  N is a whole block of 32, or 8 of a block that lanes
// 8 and 16 apart share (all 32 lanes call it then, `live` or not).
template <int N>
__device__ __forceinline__ uint32_t block_top(uint32_t t) {
  if constexpr (N == 8) {
    t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
    t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
  }
  return t;
}

template <int N>
__device__ __forceinline__ void load_bf16_row(const bf16* p, int left, bool vec, float (&v)[N]) {
  if (vec && left >= N) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      float t[8];
      load_vec<8>(p + 8 * i, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * i + j] = t[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < left ? __bfloat162float(p[i]) : 0.0f;
  }
}

template <int N>
__device__ __forceinline__ void pack_row(float (&v)[N], int left, bool live, const Epilogue& e,
                                         int64_t row, int c0) {
  float z[N];
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = i < left ? v[i] : 0.0f;
  uint32_t top = block_top<N>(part_top<N>(z));
  const bool odd = top >= kInfBits;
  const uint32_t finite = block_top<N>(part_top_finite<N>(z));
  if (odd) top = finite;
  const uint32_t code = scale_code(top);
  uint32_t w[N / 4];
  to_e4m3<N>(z, scale_inverse(code), !odd, w);
  if (!live || left <= 0) return;
  uint8_t* q = e.q + row * e.ldq + c0;
  if (e.q_vec && left >= N) {
    if constexpr (N == 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 16; ++i)
        reinterpret_cast<uint4*>(q)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
  if (c0 % kBlock == 0) e.scale[row * e.blocks_per_row + c0 / kBlock] = (uint8_t)code;
}

template <int KIND, int N>
__device__ __forceinline__ void epilogue_row(float (&v)[N], bool live, int64_t row, int c0,
                                             int left, const Epilogue& e) {
  if constexpr (KIND == kGemmForward) {
    if (e.bias) {
      float b[N];
      load_bf16_row<N>(e.bias + c0, left, e.bias_vec, b);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += b[i];
    }
    if (e.q) pack_row<N>(v, left, live, e, row, c0);
    SCAPE_ACT_SWITCH(e.act, _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act_value<ACT>(v[i]));
    if (!live) return;
    if (e.res) {
      float r[N];
      load_bf16_row<N>(e.res + row * e.ldres + c0, left, e.res_vec, r);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += r[i];
    }
  }
  if (!live || left <= 0) return;
  if constexpr (KIND == kGemmInputGrad) {
    if (e.act != SCAPE_ACT_NONE) {
      const uint8_t* p = e.pre_q + row * e.ldpre + c0;
      const float s = scale_value(e.pre_scale[row * e.blocks_per_row + c0 / kBlock]);
      float z[N];
      if (e.pre_vec && left >= N) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const uint2 w = reinterpret_cast<const uint2*>(p)[i];
          from_e4m3(w.x, s, z + 8 * i);
          from_e4m3(w.y, s, z + 8 * i + 4);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = i < left ? from_e4m3_byte(p[i], s) : 0.0f;
      }
      SCAPE_ACT_SWITCH(e.act, _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] *= act_slope<ACT>(z[i]));
    }
  }
  if (KIND == kGemmWeightGrad && e.out_f32) {
    float* o = static_cast<float*>(e.out) + row * e.ldo + c0;
    if (e.out_vec && left >= N) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<float4*>(o)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) o[i] = v[i];
    }
  } else {
    bf16* o = static_cast<bf16*>(e.out) + row * e.ldo + c0;
    if (e.out_vec && left >= N) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
        reinterpret_cast<uint4*>(o)[i] =
            make_uint4(bf16_pair(v[8 * i], v[8 * i + 1]), bf16_pair(v[8 * i + 2], v[8 * i + 3]),
                       bf16_pair(v[8 * i + 4], v[8 * i + 5]), bf16_pair(v[8 * i + 6], v[8 * i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) o[i] = __float2bfloat16_rn(v[i]);
    }
  }
}

// ------------------------------------------------------------------ the kernel
struct GemmShape {
  int m, n;
  int tiles_m, tiles_n, ksteps;
  unsigned int* status;
};

template <int KIND, int BN, bool SPLIT>
__global__ __launch_bounds__(kGemmThreads, 1) void gemm_kernel(
    const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
    const GemmShape s, const __grid_constant__ Epilogue e) {
  using TL = Tile<BN>;
  constexpr bool TA = KIND == kGemmWeightGrad;
  constexpr bool TB = KIND != kGemmForward;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * TL::kStages + 5];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;

  // swizzled operands start on 1024-byte boundaries
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (TL::kStages + i); };
  auto acc_full = [&](int i) { return bar0 + 8 * (2 * TL::kStages + i); };
  auto acc_empty = [&](int i) { return bar0 + 8 * (2 * TL::kStages + 2 + i); };
  const uint32_t drain = bar0 + 8 * (2 * TL::kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < TL::kStages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(acc_full(i), 1), mbar_init(acc_empty(i), kEpilogueWarps);
    mbar_init(drain, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base)),
                 "n"(TL::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  // Every wait ends: after the limit the kernel records it and all its roles
  // stop (they look at gave_up while they wait).
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (;;) {
      for (int i = 0; i < 16; ++i)
        if (mbar_try(bar, parity)) return true;
      if (gave_up) return false;
      if (now_ns() - t0 > kWaitLimitNs) {
        gave_up = 1;
        atomicExch(s.status, 1u);
        return false;
      }
    }
  };

  // SPLIT: one tile a cluster, its contraction cut over the cluster's blocks.
  uint32_t rank = 0, ranks = 1;
  if constexpr (SPLIT) {
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %cluster_nctarank;" : "=r"(ranks));
  }
  const int tiles = s.tiles_m * s.tiles_n;
  const int first = SPLIT ? blockIdx.x / ranks : blockIdx.x;
  const int step = SPLIT ? tiles : gridDim.x;
  const int k0 = SPLIT ? (int)((int64_t)s.ksteps * rank / ranks) : 0;
  const int k1 = SPLIT ? (int)((int64_t)s.ksteps * (rank + 1) / ranks) : s.ksteps;
  // Tiles are taken down strips of 8 tile rows, so that the blocks at work at one
  // time share operand rows in L2.
  auto tile_at = [&](int t, int& tm, int& tn) {
    const int strip = t / (8 * s.tiles_n);
    const int base = strip * 8;
    const int high = min(8, s.tiles_m - base);
    const int r = t - strip * 8 * s.tiles_n;
    tm = base + r % high;
    tn = r / high;
  };

  if (warp == 0 && lane == 0) {
    // ---------------- producer
    int stage = 0, phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int tm, tn;
      tile_at(t, tm, tn);
      for (int k = k0; k < k1; ++k) {
        ok = wait(empty(stage), phase ^ 1);
        if (!ok) break;
        const uint32_t a = smem + stage * TL::kStageBytes, b = a + TL::kABytes;
        mbar_expect_tx(full(stage), TL::kStageBytes);
        if constexpr (TA) {
#pragma unroll
          for (int i = 0; i < kBM / 64; ++i)
            tma_load(a + i * kChunk, &map_a, tm * kBM + i * 64, k * kBK, full(stage));
        } else {
          tma_load(a, &map_a, k * kBK, tm * kBM, full(stage));
        }
        if constexpr (TB) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i)
            tma_load(b + i * kChunk, &map_b, tn * BN + i * 64, k * kBK, full(stage));
        } else {
          tma_load(b, &map_b, k * kBK, tn * BN, full(stage));
        }
        ++issued;
        if (++stage == TL::kStages) stage = 0, phase ^= 1;
      }
    }
    if (!ok) {
      // let the copies in flight land before the block's memory is given back
      const int64_t from = issued > TL::kStages ? issued - TL::kStages : 0;
      for (int64_t i = from; i < issued; ++i) {
        const uint64_t t0 = now_ns();
        while (!mbar_try(full((int)(i % TL::kStages)), (uint32_t)((i / TL::kStages) & 1)))
          if (now_ns() - t0 > kWaitLimitNs) break;
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------- tensor core
    constexpr uint32_t idesc = instr_desc<BN, TA, TB>();
    int stage = 0, phase = 0, acc = 0, acc_phase = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      ok = wait(acc_empty(acc), acc_phase ^ 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * BN;
      for (int k = k0; k < k1; ++k) {
        ok = wait(full(stage), phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem + stage * TL::kStageBytes, b = a + TL::kABytes;
#pragma unroll
        for (int i = 0; i < kBK / 16; ++i) {
          // 16 of the contraction: 32 bytes along a row, or 16 rows
          const uint64_t da = smem_desc(a + i * (TA ? 2048 : 32), TA);
          const uint64_t db = smem_desc(b + i * (TB ? 2048 : 32), TB);
          tc_mma(d, da, db, idesc, k > k0 || i > 0);
        }
        tc_commit(empty(stage));
        if (++stage == TL::kStages) stage = 0, phase ^= 1;
      }
      if (!ok) break;
      tc_commit(acc_full(acc));
      if (++acc == 2) acc = 0, acc_phase ^= 1;
    }
    if (!ok) {
      tc_commit(drain);
      const uint64_t t0 = now_ns();
      while (!mbar_try(drain, 0))
        if (now_ns() - t0 > kWaitLimitNs) break;
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: warp w reads the accumulator lanes of its quarter,
    // the two warps of a quarter take half of the columns each
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    int acc = 0, acc_phase = 0;
    for (int t = first; t < tiles; t += step) {
      int tm, tn;
      tile_at(t, tm, tn);
      if (!__all_sync(0xFFFFFFFFu, wait(acc_full(acc), acc_phase))) break;
      tc_fence_after();
      const uint32_t lanes = tmem + acc * BN + ((uint32_t)(quarter * 32) << 16);
      const int64_t row = (int64_t)tm * kBM + quarter * 32 + lane;
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
        uint32_t r[32];
        tmem_ld32(lanes + c, r);
        tmem_ld_wait();
        if constexpr (SPLIT) {
          const uint32_t p = smem + 4 * (quarter * 32 + lane);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            asm volatile("st.shared::cta.b32 [%0], %1;" ::"r"(p + 4 * TL::kPartialLd * (c + i)),
                         "r"(r[i])
                         : "memory");
        } else {
          const int c0 = tn * BN + c;
          if (c0 < s.n) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            epilogue_row<KIND, 32>(v, row < s.m, row, c0, s.n - c0, e);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(acc));
      if (++acc == 2) acc = 0, acc_phase ^= 1;
    }
  }

  __syncwarp();
  if constexpr (SPLIT) {
    // Each block adds up its share of the tile's rows over the cluster's partial
    // tiles, in rank order.
    cluster_sync();
    if (warp >= 4 && !gave_up) {
      int tm, tn;
      tile_at(first, tm, tn);
      const int rows = kBM / ranks;
      const int groups = rows / 8 * (BN / 32);
      for (int g = warp - 4; g < groups; g += kEpilogueWarps) {
        const int r = rank * rows + g % (rows / 8) * 8 + (lane & 7);
        const int c = g / (rows / 8) * 32 + (lane >> 3) * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        for (uint32_t q = 0; q < ranks; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] += cluster_load(smem + 4 * (TL::kPartialLd * (c + i) + r), q);
        const int64_t row = (int64_t)tm * kBM + r;
        const int c0 = tn * BN + c;
        epilogue_row<KIND, 8>(v, row < s.m, row, c0, s.n - c0, e);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(TL::kColumns));
  }
}

// ------------------------------------------------------------------ launch
template <int KIND, int BN, bool SPLIT>
cudaError_t gemm_launch(const GemmCall& c, int split, cudaStream_t st) {
  using TL = Tile<BN>;
  constexpr bool TA = KIND == kGemmWeightGrad;
  constexpr bool TB = KIND != kGemmForward;
  CUtensorMap ma, mb;
  cudaError_t err = TA ? gemm_tensor_map(&ma, c.a.p, c.k, c.m, c.a.ld, kBK)
                       : gemm_tensor_map(&ma, c.a.p, c.m, c.k, c.a.ld, kBM);
  if (err == cudaSuccess)
    err = TB ? gemm_tensor_map(&mb, c.b.p, c.k, c.n, c.b.ld, kBK)
             : gemm_tensor_map(&mb, c.b.p, c.n, c.k, c.b.ld, BN);
  GemmShape s;
  s.m = (int)c.m;
  s.n = (int)c.n;
  s.tiles_m = (int)ceil_div(c.m, kBM);
  s.tiles_n = (int)ceil_div(c.n, BN);
  s.ksteps = (int)ceil_div(c.k, kBK);
  if (err == cudaSuccess) err = gemm_status_word(&s.status);
  auto kernel = gemm_kernel<KIND, BN, SPLIT>;
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TL::kSmem);
  if (err != cudaSuccess) return err;
  const int64_t tiles = (int64_t)s.tiles_m * s.tiles_n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * split : std::min<int64_t>(tiles, sm_count())));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = TL::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (SPLIT) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, s, c.e);
}

// Tile width and split.  A wide tile reads the fewest bytes a product; a narrow
// one, or a contraction cut over a cluster of blocks, puts more of the SMs to
// work.  So: the widest tile that fills the SMs, else the narrowest, and of the
// contraction as many cuts (a power of two up to the portable cluster of 8) as
// the SMs have room for with four stages or more left in each.
template <int KIND>
cudaError_t gemm_run(const GemmCall& c, cudaStream_t st) {
  const int64_t sms = sm_count();
  const int64_t tm = ceil_div(c.m, kBM), ksteps = ceil_div(c.k, kBK);
  int bn = 64;
  if (tm * ceil_div(c.n, 256) * 5 >= sms * 4)
    bn = 256;
  else if (tm * ceil_div(c.n, 128) * 5 >= sms * 4)
    bn = 128;
  const int64_t tiles = tm * ceil_div(c.n, bn);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && ksteps / (split * 2) >= 4) split *= 2;
  if (split > 1) {
    if (bn == 64) return gemm_launch<KIND, 64, true>(c, split, st);
    if (bn == 128) return gemm_launch<KIND, 128, true>(c, split, st);
    return gemm_launch<KIND, 256, true>(c, split, st);
  }
  if (bn == 64) return gemm_launch<KIND, 64, false>(c, 1, st);
  if (bn == 128) return gemm_launch<KIND, 128, false>(c, 1, st);
  return gemm_launch<KIND, 256, false>(c, 1, st);
}

#endif  // __CUDACC__

}  // namespace layer
}  // namespace scapek
