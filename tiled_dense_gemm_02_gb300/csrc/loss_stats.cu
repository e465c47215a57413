// The pair product of the vocabulary-head losses: row statistics of the logits (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_stats(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  const bool chunks = args.k_blocks > args.chunk;
  if (planes == 3) return chunks ? launch<HEAD_STATS, 3, 2, true>(mapA, mapB, mapC, args, pairs, stream)
                                 : launch<HEAD_STATS, 3, 1, false>(mapA, mapB, mapC, args, pairs, stream);
  if (chunks) return launch<HEAD_STATS, 1, 2, true>(mapA, mapB, mapC, args, pairs, stream);
  return args.parts == 2 ? launch<HEAD_STATS, 1, 2, false>(mapA, mapB, mapC, args, pairs, stream)
                         : launch<HEAD_STATS, 1, 1, false>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
