// The pair product of the vocabulary-head losses: gradient of the hidden states (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_dh(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  const bool chunks = args.k_per_split > args.chunk;
  if (planes == 3)
    return chunks ? launch<HEAD_DH, 3, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DH, 3, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  if (planes == 2)
    return chunks ? launch<HEAD_DH, 2, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                  : launch<HEAD_DH, 2, 2, false>(mapA, mapB, mapC, args, pairs, stream);
  return chunks ? launch<HEAD_DH, 1, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                : launch<HEAD_DH, 1, 2, false>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
