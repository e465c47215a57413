// The experts' pair product DH (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_dh(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream) {
  return launch_expert<EXPERT_DH, 4>(maps, args, pairs, stream);
}

}  // namespace tgemm
