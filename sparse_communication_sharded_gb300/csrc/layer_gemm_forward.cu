// layer_gemm_forward.cu -- the matrix product of layer_gemm.cuh for the linear layer's
// forward pass.
#include <algorithm>

#include "layer_gemm.cuh"

namespace scapek {
namespace layer {

cudaError_t gemm_probe_clusters(int blocks, int* n) {
  using TL = Tile<kGemmForward, 64, kModeSplit, true>;
  auto kernel = gemm_kernel<kGemmForward, 64, kModeSplit, true>;
  const cudaError_t e = allow_smem((const void*)kernel, TL::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(TL::kThreads);
  cfg.dynamicSmemBytes = TL::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
}

cudaError_t gemm_forward(const GemmCall& c, cudaStream_t st) { return gemm_run<kGemmForward>(c, st); }

}  // namespace layer
}  // namespace scapek
