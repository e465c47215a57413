// The experts' pair product DX (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_dx(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream) {
  return launch_expert<EXPERT_DX, 2>(maps, args, pairs, stream);
}

}  // namespace tgemm
