// layer_gemm_weight_grad.cu -- the matrix product of layer_gemm.cuh for the linear layer's
// weight gradient.
#include <algorithm>

#include "layer_gemm.cuh"

namespace scapek {
namespace layer {

cudaError_t gemm_weight_grad(const GemmCall& c, cudaStream_t st) { return gemm_run<kGemmWeightGrad>(c, st); }

}  // namespace layer
}  // namespace scapek
