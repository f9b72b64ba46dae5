// layer_gemm_input_grad.cu -- the matrix product of layer_gemm.cuh for the linear layer's
// input gradient.
#include <algorithm>

#include "layer_gemm.cuh"

namespace scapek {
namespace layer {

cudaError_t gemm_input_grad(const GemmCall& c, cudaStream_t st) { return gemm_run<kGemmInputGrad>(c, st); }

}  // namespace layer
}  // namespace scapek
