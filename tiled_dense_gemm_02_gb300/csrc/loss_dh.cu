// The pair product of the vocabulary-head losses: gradient of the hidden states (loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace tgemm {

cudaError_t launch_head_dh(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                          const HeadArgs& args, int pairs, cudaStream_t stream) {
  if (planes == 3) return launch<HEAD_DH, 3, 2>(mapA, mapB, mapC, args, pairs, stream);
  if (planes == 2) return launch<HEAD_DH, 2, 2>(mapA, mapB, mapC, args, pairs, stream);
  return launch<HEAD_DH, 1, 2>(mapA, mapB, mapC, args, pairs, stream);
}

}  // namespace tgemm
