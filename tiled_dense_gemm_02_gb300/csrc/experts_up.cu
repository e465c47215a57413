// The experts' pair product UP (experts_gemm.cuh).
#include "experts_gemm.cuh"

namespace tgemm {

cudaError_t launch_expert_up(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream) {
  if (args.gu) return launch_expert<EXPERT_UP, 4>(maps, args, pairs, stream);
  return args.gather ? launch_expert<EXPERT_UP, 2, true>(maps, args, pairs, stream)
                     : launch_expert<EXPERT_UP, 2>(maps, args, pairs, stream);
}

}  // namespace tgemm
