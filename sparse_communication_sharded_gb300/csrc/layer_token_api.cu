// layer_token_api.cu -- host side of the operators on tokens, logits and sets of
// gradients (include/scape_layers.h): checks of the arguments, workspaces, launches.
#include <algorithm>
#include <cmath>
#include <vector>

#include "layer_checks.h"
#include "layer_tokens.h"

using namespace scapek::layer;

namespace {

int check_tokens(const void* tokens, int token_bytes, const char* what) {
  if (token_bytes != 4 && token_bytes != 8) return fail(SCAPE_EINVAL, "token_bytes must be 4 or 8");
  if (!tokens || !aligned(tokens, token_bytes)) return fail(SCAPE_EINVAL, what);
  return SCAPE_OK;
}
int check_floats(const float* p, const char* what) {
  return p && aligned(p, 4) ? (int)SCAPE_OK : fail(SCAPE_EINVAL, what);
}

// Columns of a row: column numbers, rounded up to a block's, stay in an int.
constexpr int64_t kMaxCols = int64_t{1} << 30;
bool cols_ok(int64_t n) { return n >= 0 && n <= kMaxCols; }

// Where the parts of embedding_bwd's workspace lie.
struct EmbedSpace {
  size_t entries, starts, arrived, partial, bytes;
};
EmbedSpace embed_space(int64_t count, int64_t vocab, int64_t cols) {
  EmbedSpace s;
  const int64_t tiles = ceil_div(count, kEmbedTile);
  s.entries = 0;
  s.starts = round256((size_t)count * sizeof(int4));
  s.arrived = s.starts + round256((size_t)(vocab + 1) * 4);
  s.partial = s.arrived + round256((size_t)tiles * embed_chunks_most(cols) * 4);
  s.bytes = s.partial + round256((size_t)tiles * 2 * embed_partial_pitch(cols) * 4);
  return s;
}

constexpr int64_t kMaxTensor = int64_t{1} << 38;  // elements

struct Bytes {
  uintptr_t from, to;
  int index;
};

}  // namespace

extern "C" int scape_layer_embedding(const void* tokens, int token_bytes, int64_t count, const void* weight,
                                     int64_t ldw, int weight_dtype, int64_t vocab, int64_t cols, float scale, void* y,
                                     int64_t ldy, int dtype, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(count) || !size_ok(vocab) || !cols_ok(cols)) return fail(SCAPE_EINVAL, "a size is out of range");
  if (vocab == 0) return fail(SCAPE_EINVAL, "vocab must be at least 1");
  if (count == 0 || cols == 0) return SCAPE_OK;
  int rc = check_tokens(tokens, token_bytes, "tokens is NULL or misaligned");
  if (!rc) rc = check_matrix(weight, ldw, cols, weight_dtype, "weight is NULL or misaligned");
  if (!rc) rc = check_matrix(y, ldy, cols, dtype, "y is NULL or misaligned");
  if (!rc)
    rc = check_apart({matrix_span(y, ldy, count, cols, elem_size(dtype))},
                     {{vector_span(tokens, count, token_bytes)},
                      {matrix_span(weight, ldw, vocab, cols, elem_size(weight_dtype))}});
  if (rc) return rc;
  const EmbedFwd a = {{tokens, token_bytes, count}, weight, ldw, vocab, (int)cols, scale, y, ldy};
  return cuda_result(launch_embedding(a, weight_dtype, dtype, static_cast<cudaStream_t>(stream)),
                     "scape_layer_embedding");
}

extern "C" int scape_layer_embedding_bwd_workspace(int64_t count, int64_t vocab, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!size_ok(count) || !size_ok(vocab) || !cols_ok(cols)) return fail(SCAPE_EINVAL, "a size is out of range");
  *bytes = count && vocab && cols ? embed_space(count, vocab, cols).bytes : 0;
  return SCAPE_OK;
}

extern "C" int scape_layer_embedding_bwd(const void* dy, int64_t lddy, int dtype, const void* tokens, int token_bytes,
                                         int64_t count, int64_t vocab, int64_t cols, float scale, int accumulate,
                                         void* dweight, int64_t lddw, int dweight_dtype, void* workspace,
                                         size_t ws_bytes, void* stream) {
  const char* const who = "scape_layer_embedding_bwd";
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!dtype_ok(dtype) || !dtype_ok(dweight_dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(count) || !size_ok(vocab) || !cols_ok(cols)) return fail(SCAPE_EINVAL, "a size is out of range");
  if (vocab == 0) return fail(SCAPE_EINVAL, "vocab must be at least 1");
  if (cols == 0) return SCAPE_OK;
  const size_t ge = elem_size(dweight_dtype);
  int rc = check_matrix(dweight, lddw, cols, dweight_dtype, "dweight is NULL or misaligned");
  if (rc) return rc;
  if (count == 0) {
    if (accumulate) return SCAPE_OK;
    return cuda_result(cudaMemset2DAsync(dweight, lddw * ge, 0, cols * ge, vocab, st), who);
  }
  rc = check_tokens(tokens, token_bytes, "tokens is NULL or misaligned");
  if (!rc) rc = check_matrix(dy, lddy, cols, dtype, "dy is NULL or misaligned");
  const EmbedSpace s = embed_space(count, vocab, cols);
  if (!rc) rc = check_workspace(workspace, ws_bytes, s.bytes);
  if (!rc)
    rc = check_apart({matrix_span(dweight, lddw, vocab, cols, ge), vector_span(workspace, s.bytes, 1)},
                     {{vector_span(tokens, count, token_bytes)},
                      {matrix_span(dy, lddy, count, cols, elem_size(dtype))}});
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  EmbedBwd a;
  a.dy = dy, a.lddy = lddy, a.tokens = {tokens, token_bytes, count};
  a.vocab = vocab, a.cols = (int)cols, a.scale = scale, a.accumulate = accumulate != 0;
  a.dw = dweight, a.lddw = lddw;
  a.entries = reinterpret_cast<int4*>(ws + s.entries);
  a.starts = reinterpret_cast<int*>(ws + s.starts);
  a.arrived = reinterpret_cast<int*>(ws + s.arrived);
  a.partial = reinterpret_cast<float*>(ws + s.partial);
  a.partial_pitch = embed_partial_pitch(cols);
  return cuda_result(launch_embedding_bwd(a, dtype, dweight_dtype, st), who);
}

// ---------------------------------------------------------------------- logits
static int check_logits(const void* logits, int64_t ldx, int dtype, const void* targets, int token_bytes,
                        int64_t vocab) {
  int rc = check_matrix(logits, ldx, vocab, dtype, "logits is NULL or misaligned");
  if (!rc) rc = check_tokens(targets, token_bytes, "targets is NULL or misaligned");
  return rc;
}

extern "C" int scape_layer_token_logprobs(const void* logits, int64_t ldx, int dtype, const void* targets,
                                          int token_bytes, int64_t rows, int64_t vocab, int top, float* logprob,
                                          float* lse, float* entropy, float* top_logprob, int64_t* top_token,
                                          void* stream) {
  return scape_layer_token_logprobs_rest(logits, ldx, dtype, targets, token_bytes, rows, vocab, top, logprob, lse,
                                         nullptr, entropy, top_logprob, top_token, stream);
}

extern "C" int scape_layer_token_logprobs_rest(const void* logits, int64_t ldx, int dtype, const void* targets,
                                               int token_bytes, int64_t rows, int64_t vocab, int top, float* logprob,
                                               float* lse, float* lse_rest, float* entropy, float* top_logprob,
                                               int64_t* top_token, void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !cols_ok(vocab)) return fail(SCAPE_EINVAL, "rows or vocab out of range");
  if (vocab == 0) return fail(SCAPE_EINVAL, "vocab must be at least 1");
  if (top < 0 || top > SCAPE_TOP_MAX || top > vocab) return fail(SCAPE_EINVAL, "top must be 0 to 32, and at most vocab");
  if (top && vocab > SCAPE_TOP_VOCAB_MAX) return fail(SCAPE_EINVAL, "vocab is too large for alternatives");
  if (rows == 0) return SCAPE_OK;
  int rc = check_logits(logits, ldx, dtype, targets, token_bytes, vocab);
  if (!rc) rc = check_floats(logprob, "logprob is NULL or misaligned");
  if (!rc) rc = check_floats(lse, "lse is NULL or misaligned");
  if (!rc && lse_rest) rc = check_floats(lse_rest, "lse_rest is misaligned");
  if (!rc && entropy) rc = check_floats(entropy, "entropy is misaligned");
  if (!rc && top) rc = check_floats(top_logprob, "top_logprob is NULL or misaligned");
  if (!rc && top && (!top_token || !aligned(top_token, 8))) rc = fail(SCAPE_EINVAL, "top_token is NULL or misaligned");
  if (!rc)
    rc = check_apart({vector_span(logprob, rows, 4), vector_span(lse, rows, 4), vector_span(lse_rest, rows, 4),
                      vector_span(entropy, rows, 4), vector_span(top ? top_logprob : nullptr, rows * top, 4),
                      vector_span(top ? top_token : nullptr, rows * top, 8)},
                     {{matrix_span(logits, ldx, rows, vocab, elem_size(dtype))},
                      {vector_span(targets, rows, token_bytes)}});
  if (rc) return rc;
  Logprobs a = {};
  a.x = logits, a.ldx = ldx, a.targets = {targets, token_bytes, rows}, a.vocab = vocab, a.top = top;
  a.logprob = logprob, a.lse = lse, a.rest = lse_rest, a.entropy = entropy;
  a.top_logprob = top_logprob, a.top_token = top_token;
  return cuda_result(launch_logprobs(a, dtype, static_cast<cudaStream_t>(stream)), "scape_layer_token_logprobs");
}

extern "C" int scape_layer_token_logprobs_bwd(const void* logits, int64_t ldx, int dtype, const void* targets,
                                              int token_bytes, int64_t rows, int64_t vocab, const float* lse,
                                              const float* dlogprob, const float* entropy, const float* dentropy,
                                              void* dlogits, int64_t lddx, void* stream) {
  return scape_layer_token_logprobs_rest_bwd(logits, ldx, dtype, targets, token_bytes, rows, vocab, lse, nullptr,
                                             dlogprob, entropy, dentropy, dlogits, lddx, stream);
}

extern "C" int scape_layer_token_logprobs_rest_bwd(const void* logits, int64_t ldx, int dtype, const void* targets,
                                                   int token_bytes, int64_t rows, int64_t vocab, const float* lse,
                                                   const float* lse_rest, const float* dlogprob, const float* entropy,
                                                   const float* dentropy, void* dlogits, int64_t lddx, void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !cols_ok(vocab)) return fail(SCAPE_EINVAL, "rows or vocab out of range");
  if (vocab == 0) return fail(SCAPE_EINVAL, "vocab must be at least 1");
  if (rows == 0) return SCAPE_OK;
  int rc = check_logits(logits, ldx, dtype, targets, token_bytes, vocab);
  if (!rc) rc = check_floats(lse, "lse is NULL or misaligned");
  if (!rc && lse_rest) rc = check_floats(lse_rest, "lse_rest is misaligned");
  if (!rc) rc = check_floats(dlogprob, "dlogprob is NULL or misaligned");
  if (!rc && dentropy) rc = check_floats(dentropy, "dentropy is misaligned");
  if (!rc && dentropy) rc = check_floats(entropy, "entropy is NULL or misaligned");
  if (!rc) rc = check_matrix(dlogits, lddx, vocab, dtype, "dlogits is NULL or misaligned");
  const size_t e = elem_size(dtype);
  if (!rc)
    rc = check_apart({matrix_span(dlogits, lddx, rows, vocab, e)},
                     {{matrix_span(logits, ldx, rows, vocab, e), true},
                      {vector_span(targets, rows, token_bytes)},
                      {vector_span(lse, rows, 4)},
                      {vector_span(lse_rest, rows, 4)},
                      {vector_span(dlogprob, rows, 4)},
                      {vector_span(dentropy ? entropy : nullptr, rows, 4)},
                      {vector_span(dentropy, rows, 4)}});
  if (rc) return rc;
  LogprobsBwd a = {};
  a.x = logits, a.ldx = ldx, a.targets = {targets, token_bytes, rows}, a.vocab = vocab;
  a.lse = lse, a.rest = lse_rest, a.dlogprob = dlogprob, a.entropy = entropy, a.dentropy = dentropy;
  a.dx = dlogits, a.lddx = lddx;
  return cuda_result(launch_logprobs_bwd(a, dtype, static_cast<cudaStream_t>(stream)),
                     "scape_layer_token_logprobs_bwd");
}

extern "C" int scape_layer_token_loss_workspace(const void* logits, int64_t ldx, int dtype, int64_t rows,
                                                int64_t vocab, const void* dlogits, int64_t lddx, size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !cols_ok(vocab)) return fail(SCAPE_EINVAL, "rows or vocab out of range");
  const bool none = !rows || !vocab || loss_on_chip(logits, ldx, dtype, rows, vocab, dlogits, lddx);
  *bytes = none ? 0 : round256((size_t)rows * 8);  // lse in two numbers
  return SCAPE_OK;
}

extern "C" int scape_layer_token_loss(const void* logits, int64_t ldx, int dtype, const void* targets,
                                      int token_bytes, int64_t rows, int64_t vocab, const float* weight,
                                      float weight_all, float* loss, void* dlogits, int64_t lddx, void* workspace,
                                      size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype)) return fail(SCAPE_EINVAL, "unknown dtype");
  if (!size_ok(rows) || !cols_ok(vocab)) return fail(SCAPE_EINVAL, "rows or vocab out of range");
  if (vocab == 0) return fail(SCAPE_EINVAL, "vocab must be at least 1");
  if (rows == 0) return SCAPE_OK;
  int rc = check_logits(logits, ldx, dtype, targets, token_bytes, vocab);
  if (!rc && weight) rc = check_floats(weight, "weight is misaligned");
  if (!rc) rc = check_floats(loss, "loss is NULL or misaligned");
  if (!rc) rc = check_matrix(dlogits, lddx, vocab, dtype, "dlogits is NULL or misaligned");
  size_t need = 0;
  if (!rc) rc = scape_layer_token_loss_workspace(logits, ldx, dtype, rows, vocab, dlogits, lddx, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  const size_t e = elem_size(dtype);
  if (!rc)
    rc = check_apart({matrix_span(dlogits, lddx, rows, vocab, e), vector_span(loss, rows, 4),
                      vector_span(need ? workspace : nullptr, need, 1)},
                     {{matrix_span(logits, ldx, rows, vocab, e), true},
                      {vector_span(targets, rows, token_bytes)},
                      {vector_span(weight, rows, 4)}});
  if (rc) return rc;
  TokenLoss a = {};
  a.x = logits, a.ldx = ldx, a.targets = {targets, token_bytes, rows}, a.vocab = vocab;
  a.weight = weight, a.weight_all = weight_all, a.loss = loss, a.dx = dlogits, a.lddx = lddx;
  a.lse = static_cast<float*>(workspace), a.rest = need ? a.lse + rows : nullptr;
  return cuda_result(launch_token_loss(a, dtype, static_cast<cudaStream_t>(stream)), "scape_layer_token_loss");
}

// ---------------------------------------------------------------------- gradients
static int check_set(int n, const void* const* grads, const int64_t* numel, const int* dtype, const char* what) {
  if (n < 0) return fail(SCAPE_EINVAL, "n is below 0");
  if (n && (!grads || !numel || !dtype)) return fail(SCAPE_EINVAL, "an array of the set is NULL");
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > kMaxTensor) return fail(SCAPE_EINVAL, "a tensor's size is out of range");
    if (!dtype_ok(dtype[i])) return fail(SCAPE_EINVAL, "unknown dtype");
    if (numel[i] && !elem_ok(grads[i], dtype[i])) return fail(SCAPE_EINVAL, what);
  }
  return SCAPE_OK;
}

// Outputs share no memory with one another or with another tensor that is read; one
// may be its own input.  `other`: the norm and the workspace.
static int check_set_apart(const GradSet& a, std::initializer_list<Bytes> other) {
  auto bytes_of = [](const void* p, int64_t n, int dtype, int i) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return Bytes{at, at + (uintptr_t)n * elem_size(dtype), i};
  };
  std::vector<Bytes> outs;
  outs.reserve(a.n + other.size());
  for (int i = 0; a.out && i < a.n; ++i)
    if (a.numel[i]) outs.push_back(bytes_of(a.out[i], a.numel[i], a.out_dtype[i], i));
  for (const Bytes& b : other)
    if (b.to > b.from) outs.push_back(b);
  const auto before = [](const Bytes& x, const Bytes& y) { return x.from < y.from; };
  if (!std::is_sorted(outs.begin(), outs.end(), before)) std::sort(outs.begin(), outs.end(), before);
  for (size_t i = 1; i < outs.size(); ++i)
    if (outs[i].from < outs[i - 1].to) return fail(SCAPE_EINVAL, "two outputs overlap");
  for (int i = 0; i < a.n; ++i) {
    if (!a.numel[i]) continue;
    const Bytes g = bytes_of(a.grads[i], a.numel[i], a.dtype[i], i);
    // the outputs are apart, so the first that ends after g's start is the only one to
    // look at, and those that start before g's end
    auto o = std::partition_point(outs.begin(), outs.end(), [&](const Bytes& x) { return x.to <= g.from; });
    for (; o != outs.end() && o->from < g.to; ++o)
      if (!(o->index == i && o->from == g.from && o->to == g.to && a.out_dtype[i] == a.dtype[i]))
        return fail(SCAPE_EINVAL, "an output overlaps an input");
  }
  return SCAPE_OK;
}

static int run_set(const GradSet& a, void* workspace, size_t ws_bytes, cudaStream_t st, const char* who) {
  if (!a.norm || !aligned(a.norm, 4)) return fail(SCAPE_EINVAL, "norm is NULL or misaligned");
  size_t need = 0;
  int rc = scape_layer_grad_norm_workspace(a.n, a.numel, &need);
  if (!rc) rc = check_workspace(workspace, ws_bytes, need);
  if (rc) return rc;
  const uintptr_t norm = reinterpret_cast<uintptr_t>(a.norm), ws = reinterpret_cast<uintptr_t>(workspace);
  try {
    rc = check_set_apart(a, {{norm, norm + 4, -1}, {ws, ws + need, -1}});
  } catch (...) {  // memory for the list of places
    return fail(SCAPE_EINVAL, "out of host memory");
  }
  if (rc) return rc;
  GradSet b = a;
  b.partial = static_cast<double*>(workspace);
  b.partials = (int64_t)(need / sizeof(double));
  return cuda_result(launch_grad_norm(b, st), who);
}

extern "C" int scape_layer_grad_norm_workspace(int n, const int64_t* host_numel, size_t* bytes) {
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  if (n < 0 || (n && !host_numel)) return fail(SCAPE_EINVAL, "n is below 0, or host_numel NULL");
  for (int i = 0; i < n; ++i)
    if (host_numel[i] < 0 || host_numel[i] > kMaxTensor)
      return fail(SCAPE_EINVAL, "a tensor's size is out of range");
  *bytes = round256((size_t)grad_norm_partials(n, host_numel) * sizeof(double));
  return SCAPE_OK;
}

extern "C" int scape_layer_grad_norm(int n, const void* const* host_grads, const int64_t* host_numel,
                                     const int* host_dtype, float* norm, void* workspace, size_t ws_bytes,
                                     void* stream) {
  const int rc = check_set(n, host_grads, host_numel, host_dtype, "a tensor is NULL or misaligned");
  if (rc) return rc;
  GradSet a = {};
  a.n = n, a.grads = host_grads, a.numel = host_numel, a.dtype = host_dtype, a.norm = norm;
  return run_set(a, workspace, ws_bytes, static_cast<cudaStream_t>(stream), "scape_layer_grad_norm");
}

extern "C" int scape_layer_clip_grads(int n, const void* const* host_grads, const int64_t* host_numel,
                                      const int* host_dtype, void* const* host_out, const int* host_out_dtype,
                                      float max_norm, float eps, float* norm, void* workspace, size_t ws_bytes,
                                      void* stream) {
  if (!(max_norm >= 0.0f)) return fail(SCAPE_EINVAL, "max_norm must be >= 0");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SCAPE_EINVAL, "eps must be finite and >= 0");
  int rc = check_set(n, host_grads, host_numel, host_dtype, "a tensor is NULL or misaligned");
  GradSet a = {};
  a.n = n, a.grads = host_grads, a.numel = host_numel, a.dtype = host_dtype, a.norm = norm;
  a.max_norm = max_norm, a.eps = eps;
  // in place: the tensors themselves
  a.out = host_out ? host_out : const_cast<void* const*>(host_grads);
  a.out_dtype = host_out ? host_out_dtype : host_dtype;
  if (!rc && host_out)
    rc = check_set(n, const_cast<const void* const*>(host_out), host_numel, host_out_dtype,
                   "an output is NULL or misaligned");
  if (rc) return rc;
  return run_set(a, workspace, ws_bytes, static_cast<cudaStream_t>(stream), "scape_layer_clip_grads");
}
