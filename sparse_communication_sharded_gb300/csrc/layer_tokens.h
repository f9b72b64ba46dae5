// layer_tokens.h -- launchers of the operators on tokens, logits and whole sets of
// gradients (layer_embedding.cu, layer_logprobs.cu, layer_gradnorm.cu).
#pragma once

#include "layer_internal.cuh"

namespace scapek {
namespace layer {

struct Tokens {
  const void* p;
  int bytes;  // 4 or 8 a token
  int64_t count;
};

struct EmbedFwd {
  Tokens tokens;
  const void* w;
  int64_t ldw, vocab;
  int cols;
  float scale;
  void* y;
  int64_t ldy;
};
cudaError_t launch_embedding(const EmbedFwd& a, int w_dtype, int dtype, cudaStream_t st);

struct EmbedBwd {
  const void* dy;
  int64_t lddy;
  Tokens tokens;
  int64_t vocab;
  int cols;
  float scale;
  bool accumulate;
  void* dw;
  int64_t lddw;
  // workspace
  int4* entries;   // of the tokens in range, by token, then position: position, token, and
                   // where the token's entries start and end
  int* starts;     // [vocab + 1]: where a token's entries start
  int* arrived;    // [tiles][embed_chunks_most()] at most: parts done of the long token that starts
                   // in a tile, for a block's columns
  float* partial;  // [tiles][2][partial_pitch]: sums of long tokens' parts
  int64_t partial_pitch;
};
constexpr int kEmbedTile = 16;
int64_t embed_partial_pitch(int64_t cols);
int64_t embed_chunks_most(int64_t cols);
cudaError_t launch_embedding_bwd(const EmbedBwd& a, int dtype, int dw_dtype, cudaStream_t st);

struct Logprobs {
  const void* x;
  int64_t ldx;
  Tokens targets;
  int64_t vocab;
  int top;
  float *logprob, *lse, *entropy, *top_logprob;
  int64_t* top_token;
  float* rest;  // what lse's rounding leaves of it, or NULL
  // a loss: logprob receives -w times it, w = weight[row] or weight_all, and dx (in the
  // logits' places modulo 16 bytes), where it is given, the gradient
  bool loss;
  const float* weight;
  float weight_all;
  void* dx;
  int64_t lddx;
};
cudaError_t launch_logprobs(const Logprobs& a, int dtype, cudaStream_t st);

struct LogprobsBwd {
  const void* x;
  int64_t ldx;
  Tokens targets;
  int64_t vocab;
  const float *lse, *dlogprob, *entropy, *dentropy;
  const float* rest;   // of lse, or NULL
  float dlogprob_all;  // for every row where dlogprob is NULL
  bool negate;         // of dlogprob (a loss's weights)
  void* dx;
  int64_t lddx;
};
cudaError_t launch_logprobs_bwd(const LogprobsBwd& a, int dtype, cudaStream_t st);

struct TokenLoss {
  const void* x;
  int64_t ldx;
  Tokens targets;
  int64_t vocab;
  const float* weight;
  float weight_all;
  float* loss;
  void* dx;
  int64_t lddx;
  float *lse, *rest;  // workspace, where the row does not stay on chip
};
// Whether token_loss keeps a row of these on chip between its two passes.
bool loss_on_chip(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t vocab, const void* dx, int64_t lddx);
cudaError_t launch_token_loss(const TokenLoss& a, int dtype, cudaStream_t st);

struct GradSet {
  int n;
  const void* const* grads;
  const int64_t* numel;
  const int* dtype;
  void* const* out;  // NULL: the norm alone
  const int* out_dtype;
  float max_norm, eps;
  float* norm;
  double* partial;  // workspace: room for this many
  int64_t partials;
};
int64_t grad_norm_partials(int n, const int64_t* numel);
cudaError_t launch_grad_norm(const GradSet& a, cudaStream_t st);

}  // namespace layer
}  // namespace scapek
