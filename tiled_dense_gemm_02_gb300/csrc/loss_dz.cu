// The pair product of the vocabulary-head losses: gradient of the logits (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_dz(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  const bool chunks = args.k_blocks > args.chunk;
  if (planes == 3)
    return chunks ? launch<HEAD_DZ, 3, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DZ, 3, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  if (planes == 2)
    return chunks ? launch<HEAD_DZ, 2, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DZ, 2, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  return chunks ? launch<HEAD_DZ, 1, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                : launch<HEAD_DZ, 1, 2, false>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
