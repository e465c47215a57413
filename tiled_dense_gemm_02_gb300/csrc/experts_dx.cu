// The experts' pair product DX (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_dx(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const ExpertArgs& args,
                           int pairs, cudaStream_t stream) {
  return launch_expert<EXPERT_DX>(a, b, c, args, pairs, stream);
}

}  // namespace tgemm
