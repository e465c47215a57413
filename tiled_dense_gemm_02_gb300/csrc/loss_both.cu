// The two gradient products of the vocabulary-head losses in one launch
// (loss_gemm.cuh): the first pairs compute dH, the others dW.  For calls so
// short that a second launch, its set-up and the first one's tail cost more than
// the products.
#include "loss_gemm.cuh"

namespace tgemm {
namespace {

template <int PLANES>
__global__ void __launch_bounds__(head_threads(2), 1) head_both_kernel(const __grid_constant__ HeadLaunch dh,
                                                                       const __grid_constant__ HeadLaunch dw,
                                                                       const int dh_pairs) {
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (pair < dh_pairs)
    head_product<HEAD_DH, PLANES, 2, PLANES == 3>(dh.a, dh.b, dh.c, dh.args, pair, dh_pairs);
  else
    head_product<HEAD_DW, PLANES, 2, PLANES == 3>(dw.a, dw.b, dw.c, dw.args, pair - dh_pairs, pairs - dh_pairs);
}

template <int PLANES>
cudaError_t launch_both(const HeadLaunch& dh, int dh_pairs, const HeadLaunch& dw, int dw_pairs, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  static_assert(head_smem(HEAD_DH, 2) == head_smem(HEAD_DW, 2), "one shared-memory size");
  return launch_pairs(head_both_kernel<PLANES>, head_smem(HEAD_DH, 2), head_threads(2), done_mask, dh_pairs + dw_pairs,
                      stream, dh, dw, dh_pairs);
}

}  // namespace

cudaError_t launch_head_both(int planes, const HeadLaunch& dh, int dh_pairs, const HeadLaunch& dw, int dw_pairs,
                             cudaStream_t stream) {
  if (planes == 3) return launch_both<3>(dh, dh_pairs, dw, dw_pairs, stream);
  if (planes == 2) return launch_both<2>(dh, dh_pairs, dw, dw_pairs, stream);
  return launch_both<1>(dh, dh_pairs, dw, dw_pairs, stream);
}

}  // namespace tgemm
