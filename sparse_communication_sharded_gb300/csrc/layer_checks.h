// layer_checks.h -- what the C entry points of the training-layer operators share:
// the calling thread's message, checks of sizes, matrices and workspaces, and of
// outputs that would share memory with what the call reads.
#pragma once

#include <cstdio>
#include <initializer_list>

#include "layer_internal.cuh"
#include "layer_overlap.h"

namespace scapek {
namespace layer {

// The calling thread's last message (scape_layer_last_error()).
constexpr int kErrorBytes = 256;
char* error_text();

inline int fail(int code, const char* what) {
  std::snprintf(error_text(), kErrorBytes, "%s", what);
  return code;
}
inline int cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SCAPE_OK;
  // told here: CUDA's own record of it would fail the next scape_* call, whose
  // launches are checked by that record
  (void)cudaGetLastError();
  std::snprintf(error_text(), kErrorBytes, "%s: %s", what, cudaGetErrorString(e));
  return SCAPE_ECUDA;
}

// Sizes stay below this so that column numbers and tile coordinates fit an int.
constexpr int64_t kMaxSize = (int64_t{1} << 31) - 1024;

inline bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }
inline bool dtype_ok(int d) { return d == SCAPE_F32 || d == SCAPE_BF16; }
inline bool act_ok(int a) { return a >= SCAPE_ACT_NONE && a <= SCAPE_ACT_SILU; }
inline bool elem_ok(const void* p, int dtype) { return p && aligned(p, dtype == SCAPE_BF16 ? 2 : 4); }


inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SCAPE_OK;
  if (!ws || !aligned(ws, 256)) return fail(SCAPE_EINVAL, "workspace is NULL or not 256-byte aligned");
  if (have < need) return fail(SCAPE_EINVAL, "workspace is too small");
  return SCAPE_OK;
}

inline int check_packed(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t cols) {
  if (!q || !scale) return fail(SCAPE_EINVAL, "q and scale must both be given");
  if (ldq < cols) return fail(SCAPE_EINVAL, "row stride of q is below its columns");
  return SCAPE_OK;
}
inline int check_matrix(const void* p, int64_t ld, int64_t cols, int dtype, const char* what) {
  if (!elem_ok(p, dtype)) return fail(SCAPE_EINVAL, what);
  if (ld < cols) return fail(SCAPE_EINVAL, "a row stride is below the number of columns");
  return SCAPE_OK;
}

inline size_t elem_size(int dtype) { return dtype == SCAPE_BF16 ? 2 : 4; }
inline Span matrix_span(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t elem) {
  return Span(p, ld * (int64_t)elem, cols * (int64_t)elem, rows);
}
inline Span vector_span(const void* p, int64_t n, size_t elem) { return Span(p, n * (int64_t)elem, n * (int64_t)elem, 1); }
inline Span scale_span(const void* p, int64_t rows, int64_t cols) { return vector_span(p, rows * ceil_div(cols, kBlock), 1); }

// An input, and whether the call's first output may take its place.
struct Input {
  Span s;
  bool may_be_first = false;
};
// No output shares memory with an input or another output, but where the header
// says that one may be the other.
inline int check_apart(std::initializer_list<Span> outs, std::initializer_list<Input> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Input& i : ins)
      if (overlap(*o, i.s) && !(i.may_be_first && o == outs.begin() && o->same(i.s)))
        return fail(SCAPE_EINVAL, "an output overlaps an input");
    for (const Span* p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return fail(SCAPE_EINVAL, "two outputs overlap");
  }
  return SCAPE_OK;
}

}  // namespace layer
}  // namespace scapek
