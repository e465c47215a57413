// The experts' pair product DOWN (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_down(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream) {
  return launch_expert<EXPERT_DOWN, 2>(maps, args, pairs, stream);
}

}  // namespace tgemm
