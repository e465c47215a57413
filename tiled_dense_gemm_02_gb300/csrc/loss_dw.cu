// The pair product of the vocabulary-head losses: gradient of the weight (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_dw(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  if (planes == 3)
    return args.k_blocks > args.chunk ? launch<HEAD_DW, 3, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DW, 3, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  if (planes == 2) return launch<HEAD_DW, 2, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  return launch<HEAD_DW, 1, 2, false>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
