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
#include "layer_limits.h"

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
  // rows aligned for 16 bytes (1; pre: 8 bytes) or for 32 (2)
  int out_vec, res_vec, q_vec, pre_vec;
  int out_align;  // bytes that rows of out are aligned for: 2, 4 or 8 (with out_vec: more)
};

struct GemmOperand {
  const bf16* p;  // 16-byte aligned, ld a multiple of 8 (skinny products: any)
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
// How a product is cut: tiles of 128 rows, each cut over a cluster of `cluster`
// blocks; tiles of 256 rows by pairs of blocks; or whole rounds of those, and the
// tiles left over in a split launch of 128 x 128 ones.
enum GemmHow { kPlanSplit, kPlanPairs, kPlanPairsAndRest };
struct GemmPlan {
  GemmHow how;
  int columns;  // of a tile
  int cluster;  // blocks that share a split tile
};
GemmPlan gemm_plan(int kind, int64_t m, int64_t n, int64_t k, bool packs);

cudaError_t gemm_forward(const GemmCall& c, cudaStream_t st);
cudaError_t gemm_input_grad(const GemmCall& c, cudaStream_t st);
cudaError_t gemm_weight_grad(const GemmCall& c, cudaStream_t st);

// The same products for up to kSkinnyRows rows (weight gradient:
// kSkinnyWeightRows), of operands of any alignment (layer_skinny.cu); m is the rows.
constexpr int kSkinnyRows = 4;
constexpr int kSkinnyWeightRows = 8;
cudaError_t skinny_forward(const GemmCall& c, cudaStream_t st);
cudaError_t skinny_input_grad(const GemmCall& c, cudaStream_t st);
struct SkinnyWeightGrad {
  const bf16 *dy, *x;
  int64_t lddy, ldx;
  const uint8_t *q, *scale;
  int64_t ldq;
  int act;
  int64_t rows, k, n;
  void *dw, *db;
  int64_t lddw;
  int out_f32;
};
cudaError_t skinny_weight_grad(const SkinnyWeightGrad& a, cudaStream_t st);

// Clusters of so many blocks, one block an SM, that are at work at one time (asked
// of CUDA once; clusters do not cross the GPU's processing clusters, so there are
// fewer than SMs / blocks: 15 of 8 blocks on 152 SMs, and a 16th waits for a whole
// one to end).
int64_t gemm_clusters(int blocks);
cudaError_t gemm_probe_clusters(int blocks, int* n);

// Where kernels count the waits that they gave up (one word a device, never cleared).
cudaError_t gemm_status_word(unsigned int** word);

// 2-D tensor map of box_rows x box_cols boxes, their rows (64 or 128 bytes)
// swizzled over that width.
cudaError_t gemm_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols,
                            int64_t ld, int box_rows, int box_cols);

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
// One try; the hardware may suspend the thread for up to the hinted millisecond.
// Without the hint the waiting warps' polls took enough of the SM to slow the
// products by 2 to 10% (8192^3: 562 against 550 us).
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// Every wait ends: after the limit the block records it (here and in the device's
// count) and all its roles stop, as they look at gave_up while they wait.
__device__ __forceinline__ bool limited_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                             volatile int* gave_up, unsigned int* count) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try(bar, parity)) return true;
    if (*gave_up) return false;
    if (now_ns() - t0 > limit_ns) {
      *gave_up = 1;
      atomicAdd(count, 1u);
      return false;
    }
  }
}
// PAIR: the copy signals a barrier of the pair's first block (bar is that one's
// address in the cluster).
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
  bulk_commit();
}
// At most N of this thread's stores still read shared memory.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// This thread's shared memory writes, before a bulk copy reads them.
__device__ __forceinline__ void fence_for_bulk() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
// Arrives on bar when the matrix instructions issued so far are done; PAIR: on
// the barrier at that address in both blocks.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  }
}
// The same on this block's own barrier only.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_own(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  else
    tc_commit<false>(bar);
}
template <bool PAIR>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, int columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(where)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(where)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem, int columns) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  return remote;
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float4 block_load(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cta.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 cluster_load(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(addr, rank)));
  return v;
}

// ------------------------------------------------------------------ tiles
constexpr int kBM = 128;  // rows of a block's tile: the tensor core's 128 accumulator lanes
constexpr int kBK = 64;   // contraction a stage: one 128-byte swizzled row of bfloat16
constexpr int kChunk = 8192;       // bytes of 64 staged rows of 128 bytes
constexpr int kBoxBytes = 2048;    // 32 x 32 bfloat16 on their way out
constexpr int kTileCost = 500;     // clocks a tile costs besides its stages
// Clocks that a tile wider than 256 columns is read out with nothing beside it,
// without and with an 8-bit output.
constexpr int kWideCost = 3000, kWidePackCost = 6000;
// A second, split launch: clocks a stage of a 128 x 128 tile, and besides.
constexpr int kSmallStage = 600;
constexpr int kSmallLaunch = 9000;

// How a product is laid over the blocks.
enum GemmMode {
  // One tile a cluster of 1 to 8 blocks, the contraction cut over them.
  kModeSplit = 0,
  // Persistent pairs of blocks on neighbouring SMs: the pair's 256-row tile is
  // one tensor-core instruction stream, each block holding half of either
  // operand, so a byte read feeds twice the work it does in a single block.
  // The tile's width is chosen at run time (a multiple of 32 up to BN).  BN = 256
  // keeps two accumulators; BN = 384 has one, written by two instructions: the
  // first 256 columns and the others.
  kModePair = 1
};

// FULL: an epilogue with an activation or an 8-bit output; without, a bias and a
// residual at most.
template <int KIND, int BN, int MODE, bool FULL>
struct Tile {
  static constexpr bool kPair = MODE == kModePair;
  // 8 warps, 2 a scheduler; with an activation to compute 12, whose latencies
  // overlap more.  8192 x 4096, contraction 1024, in us with 8 / 12 / 16 warps:
  // forward 40.0 / 41.3 / 53, with gelu 46.5 / 44.9 / 54, input gradient through
  // gelu 51.9 / 47.5 / 48.3.  More warps crowd the one thread that issues the
  // matrix instructions; at 16 their output boxes take a stage as well.
  static constexpr int kEpilogueWarps = kPair && FULL ? 12 : 8;
  static constexpr int kThreads = 128 + 32 * kEpilogueWarps;  // + TMA, MMA, TMEM, an idle warp
  static constexpr int kGroups = kEpilogueWarps / 4;  // warps that share a quarter of the rows
  static constexpr int kWarpChunks = (BN / 32 + kGroups - 1) / kGroups;  // 32-column chunks a warp, at most
  static constexpr int kBRows = kPair ? BN / 2 : BN;  // operand B rows a block stages, at most
  static constexpr int kABytes = kBM * kBK * 2;
  static constexpr int kBBytes = kBRows * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // as many stages as fit beside the output boxes and the bias
  static constexpr int kStages = kStageBytes > 32768 ? 4 : kStageBytes > 24576 ? 5 : 6;
  static constexpr bool kWide = BN > 256;
  static constexpr int kColumns = kWide ? 512 : 2 * BN;  // two accumulators
  static constexpr int kBoxAt = kStages * kStageBytes;
  static constexpr int kBiasAt = kBoxAt + (kPair ? kEpilogueWarps * 2 * kBoxBytes : 0);
  static constexpr int kSmem =
      kBiasAt + (kPair ? kEpilogueWarps * kWarpChunks * 128 : 0) + 1024;
  // row stride of the partial tile that split products exchange: 16-byte
  // accesses of 8 neighbouring rows fall on different banks
  static constexpr int kPartialLd = BN + 4;
  static_assert(kPair || kPartialLd * kBM * 4 <= kStages * kStageBytes, "partial tile fits");
  static_assert(kSmem <= 232448, "shared memory of a block");
  static_assert(kBRows % 64 == 0, "transposed operands are staged 64 rows at a time");
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
template <int ROWS, bool TA, bool TB>
__device__ __forceinline__ uint32_t instr_desc(int bn) {
  return (1u << 4)            // 32-bit float accumulator
         | (1u << 7)          // A bfloat16
         | (1u << 10)         // B bfloat16
         | ((TA ? 1u : 0u) << 15) | ((TB ? 1u : 0u) << 16) | ((uint32_t)(bn >> 3) << 17) |
         ((uint32_t)(ROWS >> 4) << 24);
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

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

template <int N>
__device__ __forceinline__ void pack_row(const float (&v)[N], int left, bool live,
                                         const Epilogue& e, int64_t row, int c0) {
  float z[N];
  if (left >= N) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = i < left ? v[i] : 0.0f;
  }
  uint32_t top = block_top<N>(part_top<N>(z));
  if (__any_sync(0xFFFFFFFFu, top >= kInfBits)) {
    top = block_top<N>(part_top_finite<N>(z));
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = nan_unless_finite(z[i]);
  }
  const uint32_t code = scale_code(top);
  uint32_t w[N / 4];
  to_e4m3<N>(z, scale_inverse(code), w);
  if (!live || left <= 0) return;
  uint8_t* q = e.q + row * e.ldq + c0;
  if (left >= N && e.q_vec) {
    if constexpr (N == 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    } else if (e.q_vec == 2) {
      store32(q, w);
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

// What the epilogue reads of its row from memory: N bfloat16 of the residual,
// or N 8-bit values and their scale.
template <int KIND, int N>
struct Beside {
  uint32_t w[KIND == kGemmForward ? N / 2 : KIND == kGemmInputGrad ? N / 4 : 1];
  uint32_t code;
};
template <int KIND, bool FULL, int N>
__device__ __forceinline__ void load_beside(Beside<KIND, N>& b, bool live, int64_t row, int c0,
                                            int left, const Epilogue& e) {
  if constexpr (KIND == kGemmForward) {
    if (!e.res || !live || left <= 0) return;
    const bf16* p = e.res + row * e.ldres + c0;
    if (left >= N && e.res_vec) {
      if (N == 32 && e.res_vec == 2) {
        load32(p, b.w);
        load32(p + 16, b.w + 8 % (N / 2));
      } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const uint4 u = reinterpret_cast<const uint4*>(p)[i];
          b.w[4 * i] = u.x, b.w[4 * i + 1] = u.y, b.w[4 * i + 2] = u.z, b.w[4 * i + 3] = u.w;
        }
      }
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        b.w[i] = (2 * i < left ? s[2 * i] : 0u) |
                 ((uint32_t)(2 * i + 1 < left ? s[2 * i + 1] : 0u) << 16);
    }
  } else if constexpr (KIND == kGemmInputGrad && FULL) {
    if (e.act == SCAPE_ACT_NONE || !live || left <= 0) return;
    const uint8_t* p = e.pre_q + row * e.ldpre + c0;
    b.code = e.pre_scale[row * e.blocks_per_row + c0 / kBlock];
    if (left >= N && e.pre_vec) {
      if (N == 32 && e.pre_vec == 2) {
        load32(p, b.w);
      } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const uint2 u = reinterpret_cast<const uint2*>(p)[i];
          b.w[2 * i] = u.x, b.w[2 * i + 1] = u.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        b.w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * i + j < left) b.w[i] |= (uint32_t)p[4 * i + j] << (8 * j);
      }
    }
  }
}

// v *= act'(z), four z at a time from their 8-bit words.
template <int ACT, int N, int W>
__device__ __forceinline__ void times_slopes(float (&v)[N], const uint32_t (&w)[W], float scale) {
  const Slope<ACT> f(scale);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    uint64_t lo, hi;
    e4m3_pairs(w[i], lo, hi);
    unpair(mul2(f.slope(lo), pair(v[4 * i], v[4 * i + 1])), v[4 * i], v[4 * i + 1]);
    unpair(mul2(f.slope(hi), pair(v[4 * i + 2], v[4 * i + 3])), v[4 * i + 2], v[4 * i + 3]);
  }
}

// The accumulators become the values to store; the 8-bit form is stored here.
// All 32 lanes call it.
template <int KIND, bool FULL, int N>
__device__ __forceinline__ void epilogue_math(float (&v)[N], const Beside<KIND, N>& b, bool live,
                                              int64_t row, int c0, int left, const Epilogue& e) {
  if constexpr (KIND == kGemmForward) {
    if constexpr (FULL) {
      if (e.q) pack_row<N>(v, left, live, e, row, c0);
      SCAPE_ACT_SWITCH(e.act, act_values<ACT>(v));
    }
    if (e.res && live && left > 0) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        v[2 * i] += __uint_as_float(b.w[i] << 16);
        v[2 * i + 1] += __uint_as_float(b.w[i] & 0xFFFF0000u);
      }
    }
  } else if constexpr (KIND == kGemmInputGrad && FULL) {
    if (e.act != SCAPE_ACT_NONE && live && left > 0) {
      SCAPE_ACT_SWITCH(e.act, times_slopes<ACT>(v, b.w, scale_value(b.code)));
    }
  }
}

// Stores N values of a row straight from registers.
template <int KIND, int N>
__device__ __forceinline__ void store_row(const float (&v)[N], int64_t row, int c0, int left,
                                          const Epilogue& e) {
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

// Rows of a box in shared memory, written out G bytes a lane (the rows' alignment).
template <int G>
__device__ __forceinline__ void store_box_rows(uint32_t box, int lane, char* out, int64_t pitch, int rows,
                                               int left) {
  constexpr int kLanes = 64 / G, kRows = 32 / kLanes;  // lanes a row, rows at a time
  const int at = lane % kLanes * G, r0 = lane / kLanes;
#pragma unroll 8
  for (int r = r0; r < 32; r += kRows) {
    const uint32_t from = box + r * 64 + (((at >> 4) ^ ((r >> 1) & 3)) << 4) + (at & 15);
    char* to = out + r * pitch + at;
    if constexpr (G == 8) {
      uint32_t x, y;
      asm volatile("ld.shared::cta.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(from) : "memory");
      if (r < rows && at + 8 <= 2 * left) {
        *reinterpret_cast<uint2*>(to) = make_uint2(x, y);
      } else if (r < rows) {
        if (at < 2 * left) reinterpret_cast<uint16_t*>(to)[0] = (uint16_t)x;
        if (at + 2 < 2 * left) reinterpret_cast<uint16_t*>(to)[1] = (uint16_t)(x >> 16);
        if (at + 4 < 2 * left) reinterpret_cast<uint16_t*>(to)[2] = (uint16_t)y;
      }
    } else if constexpr (G == 4) {
      uint32_t x;
      asm volatile("ld.shared::cta.b32 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
      if (r < rows && at + 4 <= 2 * left)
        *reinterpret_cast<uint32_t*>(to) = x;
      else if (r < rows && at < 2 * left)
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)x;
    } else {
      uint16_t x;
      asm volatile("ld.shared::cta.u16 %0, [%1];" : "=h"(x) : "r"(from) : "memory");
      if (r < rows && at < 2 * left) *reinterpret_cast<uint16_t*>(to) = x;
    }
  }
}

// A warp's 32 x 32 values, one row a lane, through shared memory: 64-byte rows
// whose 16-byte quarters are swizzled as the output's tensor map has them, so
// neither side meets a bank twice.  Aligned outputs leave as one bulk copy, which
// cuts what is past the matrix, but of a row in whole pieces of 16 bytes: a last box
// that ends inside one goes row by row, as outputs of any alignment do, or the copy
// would write past the row's end into whatever lies beside the output.
__device__ __forceinline__ void store_box(const float (&v)[32], uint32_t box, int lane,
                                          const CUtensorMap* map, int64_t row0, int c0, int rows,
                                          int left, const Epilogue& e) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared::cta.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                     box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                 "r"(bf16_pair(v[8 * j], v[8 * j + 1])), "r"(bf16_pair(v[8 * j + 2], v[8 * j + 3])),
                 "r"(bf16_pair(v[8 * j + 4], v[8 * j + 5])), "r"(bf16_pair(v[8 * j + 6], v[8 * j + 7]))
                 : "memory");
  if (e.out_vec && (left >= 32 || left % 8 == 0)) {
    fence_for_bulk();
    __syncwarp();
    if (lane == 0) tma_store(map, c0, (int)row0, box);
  } else {
    __syncwarp();
    // one group a store, so that groups count boxes
    if (e.out_vec && lane == 0) bulk_commit();
    char* out = static_cast<char*>(e.out) + (row0 * e.ldo + c0) * 2;
    if (e.out_align == 8)
      store_box_rows<8>(box, lane, out, e.ldo * 2, rows, left);
    else if (e.out_align == 4)
      store_box_rows<4>(box, lane, out, e.ldo * 2, rows, left);
    else
      store_box_rows<2>(box, lane, out, e.ldo * 2, rows, left);
  }
}

// ------------------------------------------------------------------ the kernel
struct GemmShape {
  int m, n;
  int bn;       // columns of a tile
  int a_bytes;  // of operand A a block copies for a stage
  int tiles_m, tiles_n, ksteps;
  int tiles;  // this launch's
  // a split launch for the tiles that pairs left over: pair tiles from tile_base
  // on, each cut into 2 x sub_n of this launch's (sub_n 0: tiles of its own)
  int tile_base, sub_n;
  uint64_t product_ns;  // limit of the wait for an accumulator
  unsigned int* status;
};

// Split tiles: a warp's part of the sum over the cluster's partial tiles, in rank
// order, and the epilogue: 8 rows of 32 columns at a time, two such groups
// together.  A block does this once, so its time is latency: groups in flight
// together, no division, and a block's own part from its own shared memory.
template <int KIND, int BN, bool FULL>
__device__ __forceinline__ void join_parts(const Epilogue& e, uint32_t smem, int tm, int tn, int m, int n,
                                           uint32_t rank, uint32_t ranks) {
  using TL = Tile<KIND, BN, kModeSplit, FULL>;
  const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
  const int log_rows8 = 4 - (__ffs(ranks) - 1);  // 16 / ranks groups of 8 rows
  const int groups = (BN / 32) << log_rows8;
#pragma unroll 1
  for (int g0 = warp; g0 < groups; g0 += 2 * TL::kEpilogueWarps) {
    float v[2][8];
    Beside<KIND, 8> beside[2];
    int r[2], c[2];
    bool live[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int g = g0 + k * TL::kEpilogueWarps;
      r[k] = ((rank << log_rows8) + (g & ((1 << log_rows8) - 1))) * 8 + (lane & 7);
      c[k] = (g >> log_rows8) * 32 + (lane >> 3) * 8;
      live[k] = g < groups && tm * kBM + r[k] < m;
      if (g >= groups) r[k] = c[k] = 0;
      load_beside<KIND, FULL, 8>(beside[k], live[k], (int64_t)tm * kBM + r[k], tn * BN + c[k],
                                 n - tn * BN - c[k], e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
    }
#pragma unroll 1
    for (uint32_t q = 0; q < ranks; q += 2) {
      float4 part[2][2][2];
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (q + i < ranks) {
            const uint32_t at = smem + 4 * (TL::kPartialLd * r[k] + c[k]);
            if (q + i == rank) {
              part[i][k][0] = block_load(at), part[i][k][1] = block_load(at + 16);
            } else {
              part[i][k][0] = cluster_load(at, q + i), part[i][k][1] = cluster_load(at + 16, q + i);
            }
          }
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (q + i < ranks) {
            const float4 a = part[i][k][0], b = part[i][k][1];
            v[k][0] += a.x, v[k][1] += a.y, v[k][2] += a.z, v[k][3] += a.w;
            v[k][4] += b.x, v[k][5] += b.y, v[k][6] += b.z, v[k][7] += b.w;
          }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t row = (int64_t)tm * kBM + r[k];
      const int c0 = tn * BN + c[k], left = n - c0;
      if (KIND == kGemmForward && e.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] += i < left ? __bfloat162float(e.bias[c0 + i]) : 0.0f;
      }
      epilogue_math<KIND, FULL, 8>(v[k], beside[k], live[k], row, c0, left, e);
      if (live[k] && left > 0) store_row<KIND, 8>(v[k], row, c0, left, e);
    }
  }
}

template <int KIND, int BN, int MODE, bool FULL>
__global__ __launch_bounds__(Tile<KIND, BN, MODE, FULL>::kThreads, 1) void gemm_kernel(
    const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
    const __grid_constant__ CUtensorMap map_out, const GemmShape s,
    const __grid_constant__ Epilogue e) {
  using TL = Tile<KIND, BN, MODE, FULL>;
  constexpr bool PAIR = MODE == kModePair;
  constexpr bool TA = KIND == kGemmWeightGrad;
  constexpr bool TB = KIND != kGemmForward;
  constexpr int kTileRows = PAIR ? 2 * kBM : kBM;
  constexpr bool WIDE = TL::kWide;
  let_next_start();
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
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));

  if (threadIdx.x == 0) {
    for (int i = 0; i < TL::kStages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(acc_full(i), 1), mbar_init(acc_empty(i), TL::kEpilogueWarps * (PAIR ? 2 : 1));
    mbar_init(drain, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 96) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    if constexpr (PAIR) prefetch_map(&map_out);
  }
  if (warp == 2) tmem_alloc<PAIR>(&tmem_base, TL::kColumns);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  wait_for_earlier();  // all of the above is this kernel's own

  auto wait = [&](uint32_t bar, uint32_t parity, uint64_t limit = kWaitLimitNs) -> bool {
    return limited_wait(bar, parity, limit, &gave_up, s.status);
  };

  const int bn = PAIR ? s.bn : BN;
  const int b_rows = WIDE ? 128 : PAIR ? bn / 2 : BN;  // operand B rows this block stages
  // WIDE: beside those of the first 256 columns, its half of the others
  const int b_more = WIDE ? bn / 2 - 128 : 0;
  const int tiles = s.tiles;
  const int first = blockIdx.x / ranks;
  const int step = PAIR ? gridDim.x / 2 : tiles;
  const int k0 = PAIR ? 0 : (int)((int64_t)s.ksteps * rank / ranks);
  const int k1 = PAIR ? s.ksteps : (int)((int64_t)s.ksteps * (rank + 1) / ranks);
  // Tiles are taken down strips of 8 tile rows, so that the blocks at work at one
  // time share operand rows in L2.
  auto tile_at = [&](int t, int& tm, int& tn) {
    int part = 0;
    if (!PAIR && s.sub_n) {
      part = t % (2 * s.sub_n);
      t = s.tile_base + t / (2 * s.sub_n);
    }
    const int strip = t / (8 * s.tiles_n);
    const int base = strip * 8;
    const int high = min(8, s.tiles_m - base);
    const int r = t - strip * 8 * s.tiles_n;
    tm = base + r % high;
    tn = r / high;
    if (!PAIR && s.sub_n) {
      tm = 2 * tm + part / s.sub_n;
      tn = tn * s.sub_n + part % s.sub_n;
    }
  };

  if (warp == 0 && lane == 0) {
    // ---------------- producer: this block's rows of A and of B.  In a pair both
    // blocks' copies count on the first block's barrier, which expects them all.
    const int b_boxes = TB || WIDE ? (b_rows + 63) / 64 + (b_more + 63) / 64 : 1;
    const uint32_t bytes = s.a_bytes + (TB || WIDE ? b_boxes * kChunk : b_rows * kBK * 2);
    const uint32_t lead = PAIR ? cluster_addr(bar0, 0) - bar0 : 0;
    int stage = 0, phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int tm, tn;
      tile_at(t, tm, tn);
      const int row_a = tm * kTileRows + (PAIR ? rank * kBM : 0);
      const int row_b = tn * bn + (PAIR ? rank * b_rows : 0);
      const int row_b2 = tn * bn + 256 + (int)rank * b_more;
      for (int k = k0; k < k1; ++k) {
        ok = wait(empty(stage), phase ^ 1);
        if (!ok) break;
        const uint32_t a = smem + stage * TL::kStageBytes, b = a + TL::kABytes;
        const uint32_t bar = full(stage) + lead;
        if (!PAIR || rank == 0) mbar_expect_tx(full(stage), bytes * (PAIR ? 2 : 1));
        if constexpr (TA) {
#pragma unroll
          for (int i = 0; i < kBM / 64; ++i)
            tma_load<PAIR>(a + i * kChunk, &map_a, row_a + i * 64, k * kBK, bar);
        } else {
          tma_load<PAIR>(a, &map_a, k * kBK, row_a, bar);
        }
        if constexpr (TB || WIDE) {
          for (int i = 0; i < b_boxes; ++i) {
            const int r = WIDE && i == 2 ? row_b2 : row_b + i * 64;
            tma_load<PAIR>(b + i * kChunk, &map_b, TB ? r : k * kBK, TB ? k * kBK : r, bar);
          }
        } else {
          tma_load<PAIR>(b, &map_b, k * kBK, row_b, bar);
        }
        ++issued;
        if (++stage == TL::kStages) stage = 0, phase ^= 1;
      }
    }
    if (!ok) {
      // let the copies in flight land before the block's memory is given back
      const uint64_t t0 = now_ns();
      if (!PAIR) {
        const int64_t from = issued > TL::kStages ? issued - TL::kStages : 0;
        for (int64_t i = from; i < issued; ++i)
          while (!mbar_try(full((int)(i % TL::kStages)), (uint32_t)((i / TL::kStages) & 1)))
            if (now_ns() - t0 > kWaitLimitNs) break;
      } else {
        // the barrier that counts them may be the other block's: wait a time
        // that is long for a copy instead
        while (now_ns() - t0 < kWaitLimitNs / 100) __nanosleep(1000);
      }
    }
  } else if (warp == 1 && lane == 0 && (!PAIR || rank == 0)) {
    // ---------------- tensor core
    const uint32_t idesc = instr_desc<kTileRows, TA, TB>(WIDE ? 256 : bn);
    const uint32_t idesc2 = WIDE ? instr_desc<kTileRows, TA, TB>(bn - 256) : 0;
    const uint64_t desc_a = smem_desc(smem, TA), desc_b = smem_desc(smem + TL::kABytes, TB);
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
        // 16 of the contraction: 32 bytes along a row, or 16 rows (addresses count
        // 16 bytes; a block's shared memory ends below where they would carry)
        const uint64_t da = desc_a + ((stage * TL::kStageBytes) >> 4);
        const uint64_t db = desc_b + ((stage * TL::kStageBytes) >> 4);
#pragma unroll
        for (int i = 0; i < kBK / 16; ++i)
          tc_mma<PAIR>(d, da + i * (TA ? 128 : 2), db + i * (TB ? 128 : 2), idesc, k > k0 || i > 0);
        if constexpr (WIDE) {
#pragma unroll
          for (int i = 0; i < kBK / 16; ++i)
            tc_mma<PAIR>(d + 256, da + i * (TA ? 128 : 2), db + ((2 * kChunk) >> 4) + i * (TB ? 128 : 2), idesc2,
                         k > k0 || i > 0);
        }
        tc_commit<PAIR>(empty(stage));
        if (++stage == TL::kStages) stage = 0, phase ^= 1;
      }
      if (!ok) break;
      tc_commit<PAIR>(acc_full(acc));
      if (WIDE || ++acc == 2) acc = 0, acc_phase ^= 1;
    }
    // Tensor memory is given back when all matrix instructions are done, also where
    // the epilogue gave up before they were.  (On this block's barrier alone: the
    // pair's other block does not wait for it and may be gone when it is signalled.)
    tc_commit_own<PAIR>(drain);
    const uint64_t t0 = now_ns();
    while (!mbar_try(drain, 0))
      if (now_ns() - t0 > kWaitLimitNs) break;
    // Having given up itself, it also lets the copies land that it has not waited for
    // (a pair's are all counted here): the producer may have issued its last and gone.
    // Stages that were not issued cost the limit, once.  (A wait of the producer's in
    // every run, for its stages to be free, took 0.3 us of a product of 7.)
    for (int i = 0; !ok && i < TL::kStages; ++i) {
      while (!mbar_try(full(stage), phase))
        if (now_ns() - t0 > 2 * kWaitLimitNs) break;
      if (++stage == TL::kStages) stage = 0, phase ^= 1;
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: warp w reads the accumulator lanes of its quarter;
    // the warps of a quarter take 32-column chunks in turn, and go on with it in the
    // next tile: eight chunks are 3, 3 and 2 for three warps, and with two
    // accumulators the one with 2 need not wait for the others (8192 x 4096 x 1024
    // with gelu and 8 bits kept: 53.7 us, from the same warp on in every tile 55.1)
    const int quarter = warp & 3, group = (warp - 4) >> 2;
    const uint32_t box = smem + TL::kBoxAt + (warp - 4) * 2 * kBoxBytes;
    const uint32_t bias_at = smem + TL::kBiasAt + (warp - 4) * TL::kWarpChunks * 128;
    const bool through_box = KIND != kGemmWeightGrad || !e.out_f32;
    int acc = 0, acc_phase = 0, boxes = 0;
    int turn = group;  // this warp's first chunk of the tile
    for (int t = first; t < tiles; t += step) {
      int tm, tn;
      tile_at(t, tm, tn);
      const int64_t row0 = (int64_t)tm * kTileRows + (PAIR ? rank * kBM : 0) + quarter * 32;
      const int64_t row = row0 + lane;
      const bool live = row < s.m;
      const int col0 = tn * bn + turn * 32;
      Beside<KIND, 32> next;
      if constexpr (PAIR) {
        // before the accumulator is ready: this tile's bias, the first chunk's
        // residual or 8-bit values
        if (KIND == kGemmForward && e.bias) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < TL::kWarpChunks; ++j) {
            const int c = col0 + j * TL::kGroups * 32 + lane;
            asm volatile("st.shared::cta.f32 [%0], %1;" ::"r"(bias_at + j * 128 + lane * 4),
                         "f"(c < s.n ? __bfloat162float(e.bias[c]) : 0.0f)
                         : "memory");
          }
          __syncwarp();
        }
        load_beside<KIND, FULL, 32>(next, live, row, col0, turn * 32 < bn ? s.n - col0 : 0, e);
      }
      if (!__all_sync(0xFFFFFFFFu, wait(acc_full(acc), acc_phase, s.product_ns))) break;
      tc_fence_after();
      const uint32_t lanes = tmem + acc * BN + ((uint32_t)(quarter * 32) << 16) + turn * 32;
#pragma unroll 1
      for (int j = 0; j < TL::kWarpChunks; ++j) {
        const int c = j * TL::kGroups * 32;  // from this warp's first column
        if (turn * 32 + c >= bn) break;
        uint32_t r[32];
        tmem_ld32(lanes + c, r);
        if constexpr (!PAIR) {
          tmem_ld_wait();
          const uint32_t p = smem + 4 * (TL::kPartialLd * (quarter * 32 + lane) + turn * 32 + c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared::cta.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p + 16 * i),
                         "r"(r[4 * i]), "r"(r[4 * i + 1]), "r"(r[4 * i + 2]), "r"(r[4 * i + 3])
                         : "memory");
        } else {
          const int c0 = col0 + c, left = s.n - c0;
          const Beside<KIND, 32> beside = next;
          if (j + 1 < TL::kWarpChunks && turn * 32 + c + TL::kGroups * 32 < bn)
            load_beside<KIND, FULL, 32>(next, live, row, c0 + TL::kGroups * 32,
                                  left - TL::kGroups * 32, e);
          tmem_ld_wait();
          if (left > 0) {
            float v[32];
            if (KIND == kGemmForward && e.bias) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float b0, b1, b2, b3;
                asm volatile("ld.shared::cta.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(b0), "=f"(b1), "=f"(b2), "=f"(b3)
                             : "r"(bias_at + j * 128 + 16 * i)
                             : "memory");
                unpair(add2(pair(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), pair(b0, b1)),
                       v[4 * i], v[4 * i + 1]);
                unpair(add2(pair(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), pair(b2, b3)),
                       v[4 * i + 2], v[4 * i + 3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            }
            epilogue_math<KIND, FULL, 32>(v, beside, live, row, c0, left, e);
            if (through_box) {
              if (e.out_vec) {
                // the box two stores ago has been read
                if (lane == 0) tma_store_wait_read<1>();
              }
              __syncwarp();
              if (row0 < s.m) {
                store_box(v, box + (boxes & 1) * kBoxBytes, lane, &map_out, row0, c0,
                          (int)min((int64_t)32, s.m - row0), left, e);
                ++boxes;  // counts stores: two in a row never use one box
              }
            } else if (live) {
              store_row<KIND, 32>(v, row, c0, left, e);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          cluster_arrive(cluster_addr(acc_empty(acc), 0));
        else
          mbar_arrive(acc_empty(acc));
      }
      if (WIDE || ++acc == 2) acc = 0, acc_phase ^= 1;
      turn = (turn + TL::kGroups * 8 - bn / 32) % TL::kGroups;
    }
    if (lane == 0) tma_store_wait_all();
  }

  __syncwarp();
  if constexpr (PAIR) {
    cluster_sync();
  } else {
    auto sync_parts = [&] {
      if (ranks > 1)
        cluster_sync();
      else
        __syncthreads();
    };
    sync_parts();
    if (warp >= 4 && !gave_up) {
      int tm, tn;
      tile_at(first, tm, tn);
      join_parts<KIND, BN, FULL>(e, smem, tm, tn, s.m, s.n, rank, ranks);
    }
    __syncwarp();
    if (ranks > 1) cluster_sync();  // the parts have been read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<PAIR>(tmem, TL::kColumns);
  }
}

// ------------------------------------------------------------------ launch
// The tiles of a launch, where they are not all there are: pairs take the first
// `count`; a split launch takes what is left of a grid of pair tiles of `of_bn`
// columns, from `base` on.
struct TileRange {
  int64_t count = 0, base = 0;
  int of_bn = 0;
};

template <int KIND, int BN, int MODE, bool FULL>
cudaError_t gemm_launch(const GemmCall& c, int bn, int split, cudaStream_t st, TileRange range = {}) {
  using TL = Tile<KIND, BN, MODE, FULL>;
  constexpr bool PAIR = MODE == kModePair;
  constexpr bool TA = KIND == kGemmWeightGrad;
  constexpr bool TB = KIND != kGemmForward;
  CUtensorMap ma, mb, mo;
  // fewer rows than a tile's: copy those only (what lies in the others' place
  // reaches accumulator rows that nobody reads)
  const int a_rows = (int)std::min<int64_t>(kBM, (c.m + 7) / 8 * 8);
  cudaError_t err = TA ? gemm_tensor_map(&ma, c.a.p, c.k, c.m, c.a.ld, kBK, kBK)
                       : gemm_tensor_map(&ma, c.a.p, c.m, c.k, c.a.ld, a_rows, kBK);
  if (err == cudaSuccess)
    err = TB ? gemm_tensor_map(&mb, c.b.p, c.k, c.n, c.b.ld, kBK, kBK)
             : gemm_tensor_map(&mb, c.b.p, c.n, c.k, c.b.ld, TL::kWide ? 64 : PAIR ? bn / 2 : bn, kBK);
  if (PAIR && c.e.out_vec && !c.e.out_f32) {
    if (err == cudaSuccess) err = gemm_tensor_map(&mo, c.e.out, c.m, c.n, c.e.ldo, 32, 32);
  } else {
    mo = ma;  // not used
  }
  GemmShape s;
  s.m = (int)c.m;
  s.n = (int)c.n;
  s.bn = bn;
  s.a_bytes = TA ? TL::kABytes : a_rows * kBK * 2;
  const bool rest = range.of_bn != 0;
  s.tiles_m = (int)ceil_div(c.m, PAIR || rest ? 2 * kBM : kBM);
  s.tiles_n = (int)ceil_div(c.n, rest ? range.of_bn : bn);
  s.sub_n = rest ? range.of_bn / bn : 0;
  s.tile_base = (int)range.base;
  s.tiles = rest ? (int)((s.tiles_m * (int64_t)s.tiles_n - range.base) * 2 * s.sub_n)
                 : range.count ? (int)range.count : s.tiles_m * s.tiles_n;
  s.ksteps = (int)ceil_div(c.k, kBK);
  s.product_ns = product_wait_ns(ceil_div(s.ksteps, PAIR ? 1 : split));
  if (err == cudaSuccess) err = gemm_status_word(&s.status);
  auto kernel = gemm_kernel<KIND, BN, MODE, FULL>;
  if (err == cudaSuccess) err = allow_smem((const void*)kernel, TL::kSmem);
  if (err != cudaSuccess) return err;
  const int64_t tiles = s.tiles;
  const int cluster = PAIR ? 2 : split;
  const int64_t grid = PAIR ? 2 * std::min<int64_t>(tiles, sm_count() / 2) : tiles * split;
  return launch_kernel(kernel, (unsigned)grid, TL::kThreads, TL::kSmem, cluster, st, ma, mb, mo, s, c.e);
}

template <int KIND>
cudaError_t gemm_pairs(const GemmCall& c, int bn, cudaStream_t st, TileRange range) {
  if constexpr (KIND != kGemmWeightGrad) {
    if (c.e.act != SCAPE_ACT_NONE || c.e.q)
      return bn > 256 ? gemm_launch<KIND, 384, kModePair, true>(c, bn, 2, st, range)
                      : gemm_launch<KIND, 256, kModePair, true>(c, bn, 2, st, range);
  }
  if (bn > 256) return gemm_launch<KIND, 384, kModePair, false>(c, bn, 2, st, range);
  return gemm_launch<KIND, 256, kModePair, false>(c, bn, 2, st, range);
}

template <int KIND>
cudaError_t gemm_run(const GemmCall& c, cudaStream_t st) {
  const GemmPlan plan = gemm_plan(KIND, c.m, c.n, c.k, c.e.q != nullptr);
  switch (plan.how) {
    case kPlanPairs: return gemm_pairs<KIND>(c, plan.columns, st, {});
    case kPlanPairsAndRest: {
      const int64_t pairs = sm_count() / 2;
      const int64_t whole = ceil_div(c.m, 2 * kBM) * ceil_div(c.n, plan.columns) / pairs * pairs;
      TileRange first, rest;
      first.count = rest.base = whole;
      rest.of_bn = plan.columns;
      const cudaError_t e = gemm_pairs<KIND>(c, plan.columns, st, first);
      return e != cudaSuccess ? e : gemm_launch<KIND, 128, kModeSplit, true>(c, 128, plan.cluster, st, rest);
    }
    default:
      return plan.columns == 64 ? gemm_launch<KIND, 64, kModeSplit, true>(c, 64, plan.cluster, st)
                                : gemm_launch<KIND, 128, kModeSplit, true>(c, 128, plan.cluster, st);
  }
}

#endif  // __CUDACC__

}  // namespace layer
}  // namespace scapek
