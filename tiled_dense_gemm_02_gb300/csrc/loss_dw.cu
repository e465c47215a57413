// The pair product of the vocabulary-head losses: gradient of the weight (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_dw(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  const bool chunks = args.k_blocks > args.chunk;
  if (planes == 3)
    return chunks ? launch<HEAD_DW, 3, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DW, 3, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  if (planes == 2) return launch<HEAD_DW, 2, 2, false>(mapA, mapB, mapC, args, pairs, stream);  // few rows: one stage
  return chunks ? launch<HEAD_DW, 1, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                : launch<HEAD_DW, 1, 2, false>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
