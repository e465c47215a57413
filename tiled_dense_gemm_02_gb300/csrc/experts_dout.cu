// The experts' pair product DOUT (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_dout(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const ExpertArgs& args,
                           int pairs, cudaStream_t stream) {
  return launch_expert<EXPERT_DOUT>(a, b, c, args, pairs, stream);
}

}  // namespace tgemm
