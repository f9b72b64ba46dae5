// layer_gemm_forward.cu -- the matrix product of layer_gemm.cuh for the linear layer's
// forward pass.
#include <algorithm>

#include "layer_gemm.cuh"

namespace scapek {
namespace layer {

cudaError_t gemm_forward(const GemmCall& c, cudaStream_t st) { return gemm_run<kGemmForward>(c, st); }

}  // namespace layer
}  // namespace scapek
