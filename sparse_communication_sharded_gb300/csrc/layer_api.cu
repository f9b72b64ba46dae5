// layer_api.cu -- host side of the training-layer operators (include/scape_layers.h):
// checks of the arguments, workspaces and launches.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "layer_checks.h"
#include "layer_gemm.cuh"
#include "layer_limits.h"

namespace scapek {
namespace layer {
namespace {

__device__ unsigned int g_status;  // waits that kernels gave up

constexpr int kMaxDevices = RaisedLimits::kDevices;
std::atomic<unsigned int*> g_status_word[kMaxDevices];
LastSeen g_status_seen[kMaxDevices];

thread_local char g_error[kErrorBytes];

struct Matrix {
  const void* p;
  int64_t ld, rows, cols;
};

// Up to two matrices (blockIdx.z) of any alignment copied to 16-byte aligned
// rows, eight values a thread.  (Eight 2-byte loads a thread took 42 us for two
// passes over 10384 x 3114, bound by their instructions.)
struct AlignCopy {
  const bf16* src;
  int64_t ld, rows, cols;
  bf16* dst;
  int64_t ldd;
};
struct AlignCopies {
  AlignCopy m[2];
};
constexpr int kCopyRows = 4;
__global__ __launch_bounds__(256) void align_rows_kernel(const __grid_constant__ AlignCopies a) {
  start();
  const AlignCopy& m = a.m[blockIdx.z];
  // a block covers 8 rows of 32 vectors at a time, a thread kCopyRows of them
  const int64_t c = ((int64_t)blockIdx.x * 32 + (threadIdx.x & 31)) * 8;
  if (c >= m.ldd) return;
  const bf16* end = m.src + (m.rows - 1) * m.ld + m.cols;
  const int n = (int)min((int64_t)8, m.cols - c);
  for (int64_t row = (int64_t)blockIdx.y * 8 * kCopyRows + (threadIdx.x >> 5); row < m.rows;
       row += (int64_t)gridDim.y * 8 * kCopyRows) {
    Raw<bf16, 8> v[kCopyRows];
#pragma unroll
    for (int i = 0; i < kCopyRows; ++i)
      v[i] = load_any<8>(m.src + (row + 8 * i) * m.ld + c, row + 8 * i < m.rows ? n : 0, m.src, end);
#pragma unroll
    for (int i = 0; i < kCopyRows; ++i)
      if (row + 8 * i < m.rows)
        *reinterpret_cast<uint4*>(m.dst + (row + 8 * i) * m.ldd + c) =
            make_uint4(v[i].w[0], v[i].w[1], v[i].w[2], v[i].w[3]);
  }
}

// A wait that runs out: nothing arrives at the barrier.
__global__ void probe_wait_kernel(uint64_t limit_ns, unsigned int* count) {
  start();
  __shared__ __align__(8) uint64_t bar;
  __shared__ volatile int gave_up;
  if (threadIdx.x != 0) return;
  mbar_init(smem_addr(&bar), 1);
  gave_up = 0;
  limited_wait(smem_addr(&bar), 0, limit_ns, &gave_up, count);
}

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
size_t copy_bytes(int64_t rows, int64_t cols) { return round256((size_t)rows * round8(cols) * 2); }

bool rows32(const void* p, int64_t ld, size_t elem) {
  return aligned(p, 32) && (ld * (int64_t)elem) % 32 == 0;
}

// Bytes (up to 8) that every row starts on a multiple of.
int row_alignment(const void* p, int64_t pitch) {
  const uint64_t all = reinterpret_cast<uintptr_t>(p) | (uint64_t)pitch;
  return all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

// TMA reads rows that start on 16-byte boundaries; other operands are first
// copied to such rows in the workspace.
bool tma_rows(const void* p, int64_t ld) { return rows16(p, ld, 2); }
size_t operand_bytes(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  return tma_rows(p, ld) ? 0 : copy_bytes(rows, cols);
}
cudaError_t operands(const Matrix& a, const Matrix& b, bool any_rows, uint8_t* ws, GemmCall* call,
                     cudaStream_t st) {
  const Matrix* in[2] = {&a, &b};
  GemmOperand* out[2] = {&call->a, &call->b};
  AlignCopies copies = {};
  int n = 0;
  int64_t x = 1, y = 1;
  for (int i = 0; i < 2; ++i) {
    const Matrix& m = *in[i];
    if (any_rows || tma_rows(m.p, m.ld)) {
      *out[i] = {static_cast<const bf16*>(m.p), m.ld};
      continue;
    }
    AlignCopy& c = copies.m[n++];
    c = {static_cast<const bf16*>(m.p), m.ld, m.rows, m.cols, reinterpret_cast<bf16*>(ws), round8(m.cols)};
    ws += copy_bytes(m.rows, m.cols);
    *out[i] = {c.dst, c.ldd};
    x = std::max(x, ceil_div(c.ldd, 256));
    y = std::max(y, ceil_div(c.rows, 8 * kCopyRows));
  }
  if (n == 0) return cudaSuccess;
  return launch_kernel(align_rows_kernel, dim3((unsigned)x, (unsigned)std::min<int64_t>(y, 32768), (unsigned)n),
                       256, 0, 0, st, copies);
}

}  // namespace

char* error_text() { return g_error; }

cudaError_t gemm_status_word(unsigned int** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  unsigned int* p = g_status_word[dev].load(std::memory_order_acquire);
  if (!p) {
    void* v = nullptr;
    e = cudaGetSymbolAddress(&v, g_status);
    if (e != cudaSuccess) return e;
    p = static_cast<unsigned int*>(v);
    g_status_word[dev].store(p, std::memory_order_release);
  }
  *word = p;
  return cudaSuccess;
}

int64_t gemm_clusters(int blocks) {
  static std::atomic<int> known[kMaxDevices][4];  // 1, 2, 4, 8 blocks
  const int i = blocks == 1 ? 0 : blocks == 2 ? 1 : blocks == 4 ? 2 : 3;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev][i].load(std::memory_order_relaxed);
  if (n == 0) {
    // an answer that is not to be had counts as no cluster, i.e. no cut
    if (gemm_probe_clusters(blocks, &n) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = -1;
    }
    known[dev][i].store(n, std::memory_order_relaxed);
  }
  return n < 0 ? 0 : n;
}

// Pairs do the most work a byte read and keep the tensor cores
// busy through the epilogue; they take whole tiles, so their time goes by the
// number of tiles the busiest pair gets times a tile's.  A stage of a tile takes
// 2 clocks a column on the tensor cores, or 18 a kilobyte that comes into the SM
// (measured: 590 clocks for 32 KB, whatever the width), whichever is more.  The
// width with the least time is taken, or whole rounds of pairs with a second
// launch for the tiles left over, or one round of wider tiles (4096 x 1280,
// contraction 3584: 80 tiles for 76 pairs, 42 us in two rounds, 34.5 with 4 left
// over, 26.1 as 64 of 320 columns; contraction 1280: 23.0 left over, 13.3 wide;
// 5120 x 1024, 4096: 37.4, 31.8).  Pairs want at least 3/4 of the SMs at
// work.  Below that, narrow tiles, each cut over a cluster as far as there are
// SMs and at least four stages of the contraction for every block.
GemmPlan gemm_plan(int kind, int64_t m, int64_t n, int64_t k, bool packs) {
  const int64_t sms = sm_count(), pairs = sms / 2;
  const int64_t tp = ceil_div(m, 2 * kBM), ksteps = ceil_div(k, kBK);
  int best = 0, best_split = 0;
  int64_t least = 0;
  for (int bn = 256; bn >= 128; bn -= 32) {
    const int64_t tiles = tp * ceil_div(n, bn);
    const int64_t kb = 16 + (kind == kGemmForward ? bn / 16 : ceil_div(bn, 128) * 8);
    const int64_t tile = ksteps * std::max<int64_t>(2 * bn, 18 * kb) + kTileCost;
    const int64_t cost = ceil_div(tiles, pairs) * tile;
    if (tiles * 4 >= pairs * 3 && (best == 0 || cost < least)) best = bn, best_split = 0, least = cost;
    // whole rounds of pairs, and the tiles left over as 128 x 128 ones cut over
    // clusters, all at one time
    const int64_t rest = tiles % pairs;
    if (bn % 128 != 0 || tiles < pairs || rest == 0) continue;
    const int64_t small = rest * 2 * (bn / 128);
    int split = 1;
    while (split < 8 && small <= gemm_clusters(split * 2) && ksteps / (split * 2) >= 4) split *= 2;
    const int64_t both_cost = tiles / pairs * tile + ceil_div(ksteps, split) * kSmallStage + kSmallLaunch;
    if (small <= gemm_clusters(split) && both_cost < least) best = bn, best_split = split, least = both_cost;
  }
  // One round of tiles of 320 or 384 columns, where that is less.  They are read
  // out after their products, not beside them, so further rounds would wait, and
  // a short contraction is better off with two rounds of narrow ones (forward,
  // 4096 x 1280: 9.9 against 8.9 us at 512).
  for (int bn = 384; bn > 256; bn -= 64) {
    const int64_t tiles = tp * ceil_div(n, bn);
    const int64_t cost = ksteps * std::max<int64_t>(2 * bn, 18 * 40) + kTileCost + (packs ? kWidePackCost : kWideCost);
    if (tiles <= pairs && tiles * 4 >= pairs * 3 && best && cost < least) best = bn, best_split = 0, least = cost;
  }
  if (best) return {best_split ? kPlanPairsAndRest : kPlanPairs, best, best_split};
  const int64_t tm = ceil_div(m, kBM);
  const int bn = tm * ceil_div(n, 64) <= sms ? 64 : 128;
  const int64_t tiles = tm * ceil_div(n, bn);
  int split = 1;
  while (split < 8 && tiles <= gemm_clusters(split * 2) && ksteps / (split * 2) >= 4) split *= 2;
  return {kPlanSplit, bn, split};
}

cudaError_t allow_smem(const void* kernel, int bytes) {
  static RaisedLimits limits;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  return limits.raise(dev, kernel, bytes, cudaErrorMemoryAllocation, [&](int b) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, b);
  });
}

cudaError_t gemm_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols,
                            int64_t ld, int box_rows, int box_cols) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> encode{nullptr};
  Encode f = encode.load(std::memory_order_acquire);
  if (!f) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    f = reinterpret_cast<Encode>(fn);
    encode.store(f, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t ones[2] = {1, 1};
  const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims,
                       strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace layer
}  // namespace scapek

using namespace scapek::layer;

extern "C" const char* scape_layer_last_error(void) { return g_error; }

extern "C" int scape_layer_status(int* host_status, void* stream) {
  if (!host_status) return fail(SCAPE_EINVAL, "host_status is NULL");
  *host_status = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned int* word = nullptr;
  unsigned int v = 0;
  int dev = 0;
  cudaError_t e = gemm_status_word(&word);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof v, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) *host_status = g_status_seen[dev].news(v);
  return cuda_result(e, "scape_layer_status");
}

extern "C" int scape_layer_probe_wait(int64_t limit_ns, void* stream) {
  if (limit_ns < 1 || limit_ns > (int64_t)kWaitLimitNs)
    return fail(SCAPE_EINVAL, "limit_ns must be from 1 to two seconds");
  unsigned int* word = nullptr;
  cudaError_t e = gemm_status_word(&word);
  if (e == cudaSuccess)
    e = launch_kernel(probe_wait_kernel, dim3(1), 32, 0, 0, static_cast<cudaStream_t>(stream), (uint64_t)limit_ns, word);
  return cuda_result(e, "scape_layer_probe_wait");
}

extern "C" int scape_layer_pack8(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                                 uint8_t* q, int64_t ldq, uint8_t* scale, void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  if (rows == 0 || cols == 0) return SCAPE_OK;
  int rc = check_matrix(x, ldx, cols, dtype, "x is NULL or misaligned");
  if (!rc) rc = check_packed(q, ldq, scale, cols);
  if (!rc)
    rc = check_apart({matrix_span(q, ldq, rows, cols, 1), scale_span(scale, rows, cols)},
                     {{matrix_span(x, ldx, rows, cols, elem_size(dtype))}});
  if (rc) return rc;
  return cuda_result(launch_pack8(x, ldx, dtype, rows, cols, q, ldq, scale,
                                  static_cast<cudaStream_t>(stream)),
                     "scape_layer_pack8");
}

extern "C" int scape_layer_unpack8(const uint8_t* q, int64_t ldq, const uint8_t* scale,
                                   int64_t rows, int64_t cols, int activation, void* y,
                                   int64_t ldy, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!act_ok(activation)) return fail(SCAPE_EINVAL, "unknown activation");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  if (rows == 0 || cols == 0) return SCAPE_OK;
  int rc = check_packed(q, ldq, scale, cols);
  if (!rc) rc = check_matrix(y, ldy, cols, dtype, "y is NULL or misaligned");
  if (!rc)
    rc = check_apart({matrix_span(y, ldy, rows, cols, elem_size(dtype))},
                     {{matrix_span(q, ldq, rows, cols, 1)}, {scale_span(scale, rows, cols)}});
  if (rc) return rc;
  return cuda_result(launch_unpack8(q, ldq, scale, rows, cols, activation, y, ldy, dtype,
                                    static_cast<cudaStream_t>(stream)),
                     "scape_layer_unpack8");
}

extern "C" int scape_layer_act_grad(const void* dy, int64_t lddy, const uint8_t* q, int64_t ldq,
                                    const uint8_t* scale, int64_t rows, int64_t cols,
                                    int activation, void* dz, int64_t lddz, int dtype,
                                    void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!act_ok(activation)) return fail(SCAPE_EINVAL, "unknown activation");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  if (rows == 0 || cols == 0) return SCAPE_OK;
  int rc = check_matrix(dy, lddy, cols, dtype, "dy is NULL or misaligned");
  if (!rc) rc = check_packed(q, ldq, scale, cols);
  if (!rc) rc = check_matrix(dz, lddz, cols, dtype, "dz is NULL or misaligned");
  if (!rc)
    rc = check_apart({matrix_span(dz, lddz, rows, cols, elem_size(dtype))},
                     {{matrix_span(dy, lddy, rows, cols, elem_size(dtype)), true},
                      {matrix_span(q, ldq, rows, cols, 1)},
                      {scale_span(scale, rows, cols)}});
  if (rc) return rc;
  return cuda_result(launch_act_grad(dy, lddy, q, ldq, scale, rows, cols, activation, dz, lddz,
                                     dtype, static_cast<cudaStream_t>(stream)),
                     "scape_layer_act_grad");
}

extern "C" int scape_layer_add_rmsnorm(const void* x, int64_t ldx, const void* residual,
                                       int64_t ldres, const void* weight, int weight_dtype,
                                       int64_t rows, int64_t cols, float eps, int dtype, void* y,
                                       int64_t ldy, void* h, int64_t ldh, float* rstd, uint8_t* q,
                                       int64_t ldq, uint8_t* scale, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SCAPE_EINVAL, "eps must be finite and >= 0");
  if (rows == 0 || cols == 0) return SCAPE_OK;
  int rc = check_matrix(x, ldx, cols, dtype, "x is NULL or misaligned");
  if (!rc && residual) rc = check_matrix(residual, ldres, cols, dtype, "residual is misaligned");
  if (!rc) rc = check_matrix(y, ldy, cols, dtype, "y is NULL or misaligned");
  if (!rc && h) rc = check_matrix(h, ldh, cols, dtype, "h is misaligned");
  if (!rc && !elem_ok(weight, weight_dtype)) rc = fail(SCAPE_EINVAL, "weight is NULL or misaligned");
  if (!rc && rstd && !aligned(rstd, 4)) rc = fail(SCAPE_EINVAL, "rstd is misaligned");
  if (!rc && (q || scale)) rc = check_packed(q, ldq, scale, cols);
  if (!rc) {
    const size_t e = elem_size(dtype);
    rc = check_apart({matrix_span(h, ldh, rows, cols, e), matrix_span(y, ldy, rows, cols, e), vector_span(rstd, rows, 4),
                      matrix_span(q, ldq, rows, cols, 1), scale_span(scale, rows, cols)},
                     {{matrix_span(x, ldx, rows, cols, e), true},
                      {matrix_span(residual, ldres, rows, cols, e), true},
                      {vector_span(weight, cols, elem_size(weight_dtype))}});
  }
  if (rc) return rc;
  NormFwd a;
  a.x = x, a.res = residual, a.w = weight;
  a.ldx = ldx, a.ldres = ldres, a.ldy = ldy, a.ldh = ldh, a.ldq = ldq;
  a.w_bf16 = weight_dtype == SCAPE_BF16;
  a.rows = rows, a.cols = (int)cols, a.eps = eps;
  a.y = y, a.h = h, a.rstd = rstd, a.q = q, a.scale = scale, a.q16 = false;
  return cuda_result(launch_norm_fwd(a, dtype, static_cast<cudaStream_t>(stream)),
                     "scape_layer_add_rmsnorm");
}

extern "C" int scape_layer_add_rmsnorm_bwd_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  *bytes = rows && cols ? round256((size_t)norm_bwd_partials(rows, cols) * cols * 4) : 0;
  return SCAPE_OK;
}

extern "C" int scape_layer_add_rmsnorm_bwd(const void* dy, int64_t lddy, const void* h,
                                           int64_t ldh, const void* weight, int weight_dtype,
                                           const float* rstd, const void* dh, int64_t lddh,
                                           int64_t rows, int64_t cols, int dtype, void* dx,
                                           int64_t lddx, void* dweight, int dweight_dtype,
                                           void* workspace, size_t ws_bytes, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || !dtype_ok(dweight_dtype))
    return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !size_ok(cols)) return fail(SCAPE_EINVAL, "rows or cols out of range");
  if (cols == 0) return SCAPE_OK;
  if (dweight && !elem_ok(dweight, dweight_dtype)) return fail(SCAPE_EINVAL, "dweight is misaligned");
  if (rows == 0) {
    if (!dweight) return SCAPE_OK;
    return cuda_result(cudaMemsetAsync(dweight, 0, cols * (dweight_dtype == SCAPE_BF16 ? 2 : 4), st),
                       "scape_layer_add_rmsnorm_bwd");
  }
  int rc = check_matrix(dy, lddy, cols, dtype, "dy is NULL or misaligned");
  if (!rc) rc = check_matrix(h, ldh, cols, dtype, "h is NULL or misaligned");
  if (!rc && dh) rc = check_matrix(dh, lddh, cols, dtype, "dh is misaligned");
  if (!rc) rc = check_matrix(dx, lddx, cols, dtype, "dx is NULL or misaligned");
  if (!rc && !elem_ok(weight, weight_dtype)) rc = fail(SCAPE_EINVAL, "weight is NULL or misaligned");
  if (!rc && (!rstd || !aligned(rstd, 4))) rc = fail(SCAPE_EINVAL, "rstd is NULL or misaligned");
  size_t need = 0;
  if (!rc && dweight) rc = scape_layer_add_rmsnorm_bwd_workspace(rows, cols, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  if (!rc) {
    const size_t e = elem_size(dtype);
    rc = check_apart({matrix_span(dx, lddx, rows, cols, e), vector_span(dweight, cols, elem_size(dweight_dtype)),
                      vector_span(workspace, need, 1)},
                     {{matrix_span(dy, lddy, rows, cols, e), true},
                      {matrix_span(h, ldh, rows, cols, e)},
                      {vector_span(weight, cols, elem_size(weight_dtype))},
                      {vector_span(rstd, rows, 4)},
                      {matrix_span(dh, lddh, rows, cols, e), true}});
  }
  if (rc) return rc;
  NormBwd a;
  a.dy = dy, a.h = h, a.w = weight, a.dh = dh;
  a.lddy = lddy, a.ldh = ldh, a.lddh = lddh, a.lddx = lddx;
  a.rstd = rstd, a.w_bf16 = weight_dtype == SCAPE_BF16, a.dw_bf16 = dweight_dtype == SCAPE_BF16;
  a.rows = rows, a.cols = (int)cols, a.dx = dx, a.dw = dweight;
  a.partial = static_cast<float*>(workspace);
  return cuda_result(launch_norm_bwd(a, dtype, st), "scape_layer_add_rmsnorm_bwd");
}

// ---------------------------------------------------------------------- linear
extern "C" int scape_layer_linear_workspace(const void* x, int64_t ldx, const void* weight,
                                            int64_t ldw, int64_t rows, int64_t k, int64_t n,
                                            size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  *bytes = rows > kSkinnyRows && n ? operand_bytes(x, ldx, rows, k) + operand_bytes(weight, ldw, n, k) : 0;
  return SCAPE_OK;
}

extern "C" int scape_layer_linear(const void* x, int64_t ldx, const void* weight, int64_t ldw,
                                  const void* bias, const void* residual, int64_t ldres,
                                  int64_t rows, int64_t k, int64_t n, int activation, void* y,
                                  int64_t ldy, uint8_t* q, int64_t ldq, uint8_t* scale,
                                  void* workspace, size_t ws_bytes, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!act_ok(activation)) return fail(SCAPE_EINVAL, "unknown activation");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  if (k == 0) return fail(SCAPE_EINVAL, "k must be at least 1");
  if (rows == 0 || n == 0) return SCAPE_OK;
  int rc = check_matrix(x, ldx, k, SCAPE_BF16, "x is NULL or misaligned");
  if (!rc) rc = check_matrix(weight, ldw, k, SCAPE_BF16, "weight is NULL or misaligned");
  if (!rc && bias && !aligned(bias, 2)) rc = fail(SCAPE_EINVAL, "bias is misaligned");
  if (!rc && residual) rc = check_matrix(residual, ldres, n, SCAPE_BF16, "residual is misaligned");
  if (!rc) rc = check_matrix(y, ldy, n, SCAPE_BF16, "y is NULL or misaligned");
  if (!rc && (q || scale)) rc = check_packed(q, ldq, scale, n);
  size_t need = 0;
  if (!rc) rc = scape_layer_linear_workspace(x, ldx, weight, ldw, rows, k, n, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  if (!rc)
    rc = check_apart({matrix_span(y, ldy, rows, n, 2), matrix_span(q, ldq, rows, n, 1), scale_span(scale, rows, n),
                      vector_span(workspace, need, 1)},
                     {{matrix_span(x, ldx, rows, k, 2)},
                      {matrix_span(weight, ldw, n, k, 2)},
                      {vector_span(bias, n, 2)},
                      {matrix_span(residual, ldres, rows, n, 2), true}});
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GemmCall c = {};
  const bool skinny = rows <= kSkinnyRows;
  cudaError_t e = operands({x, ldx, rows, k}, {weight, ldw, n, k}, skinny, ws, &c, st);
  c.m = rows, c.n = n, c.k = k;
  c.e.act = activation;
  c.e.bias = static_cast<const bf16*>(bias);
  c.e.res = static_cast<const bf16*>(residual);
  c.e.ldres = ldres;
  c.e.res_vec = rows16(residual, ldres, 2) + rows32(residual, ldres, 2);
  c.e.q = q, c.e.ldq = ldq, c.e.scale = scale;
  c.e.q_vec = rows16(q, ldq, 1) + rows32(q, ldq, 1);
  c.e.blocks_per_row = ceil_div(n, kBlock);
  c.e.out = y, c.e.ldo = ldy;
  c.e.out_vec = rows16(y, ldy, 2);
  c.e.out_align = row_alignment(y, ldy * 2);
  if (e == cudaSuccess) e = skinny ? skinny_forward(c, st) : gemm_forward(c, st);
  return cuda_result(e, "scape_layer_linear");
}

extern "C" int scape_layer_linear_bwd_input_workspace(const void* dy, int64_t lddy,
                                                      const void* weight, int64_t ldw,
                                                      int64_t rows, int64_t k, int64_t n,
                                                      size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  *bytes = rows > kSkinnyRows && k ? operand_bytes(dy, lddy, rows, n) + operand_bytes(weight, ldw, n, k) : 0;
  return SCAPE_OK;
}

extern "C" int scape_layer_linear_bwd_input(const void* dy, int64_t lddy, const void* weight,
                                            int64_t ldw, const uint8_t* q, int64_t ldq,
                                            const uint8_t* scale, int activation, int64_t rows,
                                            int64_t k, int64_t n, void* dx, int64_t lddx,
                                            void* workspace, size_t ws_bytes, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!act_ok(activation)) return fail(SCAPE_EINVAL, "unknown activation");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  if (n == 0) return fail(SCAPE_EINVAL, "n must be at least 1");
  if (rows == 0 || k == 0) return SCAPE_OK;
  int rc = check_matrix(dy, lddy, n, SCAPE_BF16, "dy is NULL or misaligned");
  if (!rc) rc = check_matrix(weight, ldw, k, SCAPE_BF16, "weight is NULL or misaligned");
  if (!rc) rc = check_matrix(dx, lddx, k, SCAPE_BF16, "dx is NULL or misaligned");
  if (!rc && activation != SCAPE_ACT_NONE) rc = check_packed(q, ldq, scale, k);
  size_t need = 0;
  if (!rc) rc = scape_layer_linear_bwd_input_workspace(dy, lddy, weight, ldw, rows, k, n, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  if (!rc) {
    const int64_t pre = activation != SCAPE_ACT_NONE ? rows : 0;
    rc = check_apart({matrix_span(dx, lddx, rows, k, 2), vector_span(workspace, need, 1)},
                     {{matrix_span(dy, lddy, rows, n, 2)},
                      {matrix_span(weight, ldw, n, k, 2)},
                      {matrix_span(q, ldq, pre, k, 1)},
                      {scale_span(scale, pre, k)}});
  }
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GemmCall c = {};
  const bool skinny = rows <= kSkinnyRows;
  cudaError_t e = operands({dy, lddy, rows, n}, {weight, ldw, n, k}, skinny, ws, &c, st);
  c.m = rows, c.n = k, c.k = n;
  c.e.act = activation;
  c.e.pre_q = q, c.e.ldpre = ldq, c.e.pre_scale = scale;
  c.e.pre_vec = rows8(q, ldq) + rows32(q, ldq, 1);
  c.e.blocks_per_row = ceil_div(k, kBlock);
  c.e.out = dx, c.e.ldo = lddx;
  c.e.out_vec = rows16(dx, lddx, 2);
  c.e.out_align = row_alignment(dx, lddx * 2);
  if (e == cudaSuccess) e = skinny ? skinny_input_grad(c, st) : gemm_input_grad(c, st);
  return cuda_result(e, "scape_layer_linear_bwd_input");
}

extern "C" int scape_layer_linear_plan(int product, int64_t rows, int64_t k, int64_t n, int keeps_8bit, int* kernel,
                                       int* columns, int* cluster) {
  if (product < SCAPE_LINEAR_FORWARD || product > SCAPE_LINEAR_WEIGHT_GRAD) return fail(SCAPE_EINVAL, "unknown product");
  if (!kernel || !columns || !cluster) return fail(SCAPE_EINVAL, "kernel, columns and cluster must be given");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n) || !rows || !k || !n) return fail(SCAPE_EINVAL, "a size is out of range");
  *columns = *cluster = 0;
  if (rows <= (product == SCAPE_LINEAR_WEIGHT_GRAD ? kSkinnyWeightRows : kSkinnyRows)) {
    *kernel = SCAPE_PLAN_FEW_ROWS;
    return SCAPE_OK;
  }
  const GemmPlan p = product == SCAPE_LINEAR_FORWARD      ? gemm_plan(kGemmForward, rows, n, k, keeps_8bit != 0)
                     : product == SCAPE_LINEAR_INPUT_GRAD ? gemm_plan(kGemmInputGrad, rows, k, n, false)
                                                          : gemm_plan(kGemmWeightGrad, n, k, rows, false);
  *kernel = p.how == kPlanSplit ? SCAPE_PLAN_SPLIT : p.how == kPlanPairs ? SCAPE_PLAN_PAIRS : SCAPE_PLAN_PAIRS_AND_SPLIT;
  *columns = p.columns;
  *cluster = p.cluster;
  return SCAPE_OK;
}

// Whether the bias sums go into the launch that unpacks the input.  That spares a
// launch (us with them there / in one of their own; dy n wide, the input k):
//   64 x 256, n 256   6.4 / 8.0      4096 x 1280, n 3584   36.1 / 41.1
//   2048 x 1024, n 4096   20.4 / 25.8     8192 x 4096, n 4096   189 / 194
// But a block of the sums takes an eighth of the rows, however little else there is
// to do, and of the blocks beside the unpacking fewer are in flight.  Where the bytes
// of a row, 3 k + 2 n, are few that is the longer part, the more so the more rows:
//   rows            12000        16384        24576        65536        131072
//   k 64, n 64    17.2 / 17.4  20.5 / 19.9  25.9 / 24.6     -          98 / 89
//   k 256, n 256  19.7 / 20.1  22.8 / 23.6  29.4 / 29.7  64.3 / 58.8   134 / 115
//   k 64, n 1024  20.4 / 21.2  23.5 / 23.9  33.0 / 30.0  77.6 / 70.0   141 / 123
//   k 256, n 1024 24.6 / 26.1  31.1 / 31.2  42.5 / 42.0  107 / 98      195 / 182
// while rows of 3200 bytes and more hide it at any length:
//   k 1024, n 64  24.4 / 27.5  29.8 / 33.5  40.8 / 45.7     -          205 / 214
//   k 256, n 2048 33.8 / 35.9  44.4 / 48.5  64.2 / 68.9     -          316 / 345
static bool sums_beside(const void* dy, int64_t lddy, int64_t rows, int64_t k, int64_t n) {
  return rows16(dy, lddy, 2) && (rows <= 12288 || 3 * k + 2 * n >= 3200);
}

extern "C" int scape_layer_linear_bwd_weight_workspace(const void* dy, int64_t lddy, const void* x,
                                                       int64_t ldx, int64_t rows, int64_t k,
                                                       int64_t n, size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  *bytes = 0;
  if (rows <= kSkinnyWeightRows || n == 0) return SCAPE_OK;
  *bytes = operand_bytes(dy, lddy, rows, n) +
           (x ? operand_bytes(x, ldx, rows, k) : copy_bytes(rows, k));
  return SCAPE_OK;
}

extern "C" int scape_layer_linear_bwd_weight(const void* dy, int64_t lddy, const void* x,
                                             int64_t ldx, const uint8_t* q, int64_t ldq,
                                             const uint8_t* scale, int activation, int64_t rows,
                                             int64_t k, int64_t n, void* dweight, int64_t lddw,
                                             void* dbias, int grad_dtype, void* workspace,
                                             size_t ws_bytes, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const char* const who = "scape_layer_linear_bwd_weight";
  if (!act_ok(activation)) return fail(SCAPE_EINVAL, "unknown activation");
  if (!dtype_ok(grad_dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !size_ok(k) || !size_ok(n)) return fail(SCAPE_EINVAL, "a size is out of range");
  if (x && q) return fail(SCAPE_EINVAL, "x and q are both given");
  if (x && activation != SCAPE_ACT_NONE)
    return fail(SCAPE_EINVAL, "an activation is applied to an 8-bit input only");
  if (n == 0) return SCAPE_OK;
  const size_t ge = grad_dtype == SCAPE_BF16 ? 2 : 4;
  if (dbias && !elem_ok(dbias, grad_dtype)) return fail(SCAPE_EINVAL, "dbias is misaligned");
  int rc = SCAPE_OK;
  if (k) rc = check_matrix(dweight, lddw, k, grad_dtype, "dweight is NULL or misaligned");
  if (rc) return rc;
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    if (k) e = cudaMemset2DAsync(dweight, lddw * ge, 0, k * ge, n, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, n * ge, st);
    return cuda_result(e, who);
  }
  rc = check_matrix(dy, lddy, n, SCAPE_BF16, "dy is NULL or misaligned");
  if (!rc && k) rc = x ? check_matrix(x, ldx, k, SCAPE_BF16, "x is misaligned") : check_packed(q, ldq, scale, k);
  size_t need = 0;
  if (!rc) rc = scape_layer_linear_bwd_weight_workspace(dy, lddy, x, ldx, rows, k, n, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  if (!rc)
    rc = check_apart({matrix_span(dweight, lddw, n, k, ge), vector_span(dbias, n, ge), vector_span(workspace, need, 1)},
                     {{matrix_span(dy, lddy, rows, n, 2)},
                      {matrix_span(x, ldx, rows, k, 2)},
                      {matrix_span(q, ldq, rows, k, 1)},
                      {scale_span(q ? scale : nullptr, rows, k)}});
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (k && rows <= kSkinnyWeightRows) {
    SkinnyWeightGrad a;
    a.dy = static_cast<const bf16*>(dy), a.x = static_cast<const bf16*>(x);
    a.lddy = lddy, a.ldx = ldx, a.q = q, a.scale = scale, a.ldq = ldq, a.act = activation;
    a.rows = rows, a.k = k, a.n = n;
    a.dw = dweight, a.db = dbias, a.lddw = lddw, a.out_f32 = grad_dtype == SCAPE_F32;
    return cuda_result(skinny_weight_grad(a, st), who);
  }
  if (k) {
    GemmCall c = {};
    if (x) {
      e = operands({dy, lddy, rows, n}, {x, ldx, rows, k}, false, ws, &c, st);
    } else {
      // The tensor cores multiply bfloat16, so an activation's value is rounded to it,
      // as the forward product took it: 8192 x 4096 through gelu against 1024 columns
      // of dy has an error of 0.0018 of the gradient so, 0.0017 with 32-bit values.
      // Without an activation the values are exact.
      bf16* a = reinterpret_cast<bf16*>(ws);
      ws += copy_bytes(rows, k);
      if (dbias && sums_beside(dy, lddy, rows, k, n)) {
        e = launch_unpack8_sums(q, ldq, scale, rows, k, activation, a, round8(k),
                                {static_cast<const bf16*>(dy), lddy, rows, n, dbias, grad_dtype == SCAPE_BF16}, st);
        dbias = nullptr;
      } else {
        e = launch_unpack8(q, ldq, scale, rows, k, activation, a, round8(k), SCAPE_BF16, st);
      }
      if (e == cudaSuccess) e = operands({dy, lddy, rows, n}, {a, round8(k), rows, k}, false, ws, &c, st);
    }
    c.m = n, c.n = k, c.k = rows;
    c.e.out = dweight, c.e.ldo = lddw, c.e.out_f32 = grad_dtype == SCAPE_F32;
    c.e.out_vec = rows16(dweight, lddw, ge);
    c.e.out_align = row_alignment(dweight, lddw * ge);
    if (e == cudaSuccess) e = gemm_weight_grad(c, st);
    // from aligned rows, if they had to be made
    dy = c.a.p, lddy = c.a.ld;
  }
  if (e == cudaSuccess && dbias)
    e = launch_colsum({static_cast<const bf16*>(dy), lddy, rows, n, dbias, grad_dtype == SCAPE_BF16}, st);
  return cuda_result(e, who);
}
