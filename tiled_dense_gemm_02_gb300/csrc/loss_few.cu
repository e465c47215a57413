// Forward of the vocabulary-head losses for a few rows (loss_few.cuh).
#include "loss_few.cuh"

namespace tgemm {
namespace {

template <typename E, int G>
cudaError_t launch_rows(const FewArgs& a, int blocks, cudaStream_t stream) {
  if (a.T <= 1) return launch_logits<E, 1, G, false>(a, blocks, stream);
  if constexpr (sizeof(E) == 4 || G < 16) {
    if (a.T <= 2) return launch_logits<E, 2, G, false>(a, blocks, stream);
    if (a.T <= 4) return launch_logits<E, 4, G, false>(a, blocks, stream);
    return launch_logits<E, 8, G, false>(a, blocks, stream);
  }
  return cudaErrorInvalidValue;  // aligned 16-bit rows from two on take the tensor cores
}

template <typename E>
cudaError_t launch_type(const FewArgs& a, int granule, int blocks, cudaStream_t stream) {
  if (granule == 16) return launch_rows<E, 16>(a, blocks, stream);
  if constexpr (sizeof(E) == 4)
    return launch_rows<E, 4>(a, blocks, stream);
  else
    return granule >= 4 ? launch_rows<E, 4>(a, blocks, stream) : launch_rows<E, 2>(a, blocks, stream);
}

}  // namespace

// As far as it is faster than the tensor cores (loss_few.cuh, loss_few_grad.cu have
// both sides), and the rows of H fit shared memory.
bool few_rows(bool backward, int64_t T, int64_t V, int64_t D, bool f32, bool aligned) {
  int64_t most = kFewRows;
  if (f32) {
    // below kFewSimtV entries passes of eight rows beat the tiles of loss_simt.cu too
    if (!backward && V < kFewSimtV) most = kHeadSimtRows;
  } else if (backward) {
    most = aligned ? 2 : 0;
  } else if (aligned) {
    most = 1;
  }
  return T <= most && rows_held(T) * (D + 8) * 4 <= kFewSmem;
}

int few_blocks(int64_t T, int64_t V) {
  // the blocks that fit the SMs at once, each warp with at least one entry
  const int tn = rows_held(T), warps = few_threads(tn) / 32;
  return static_cast<int>(std::min<int64_t>((V + warps - 1) / warps, int64_t(kFewSms) * few_per_sm(tn)));
}

cudaError_t launch_few_stats(const FewArgs& args, int type, int granule, int blocks, cudaStream_t stream) {
  // eight rows at a time; every pass leaves its statistics in the same number of parts
  for (int t0 = 0; t0 < args.T; t0 += kFewRows) {
    FewArgs a = args;
    a.T = std::min(kFewRows, args.T - t0);
    a.H = static_cast<const char*>(args.H) + t0 * args.ldh * (type == 2 ? 4 : 2);
    if (a.targets) a.targets += t0;
    if (a.ids) {
      a.ids += static_cast<int64_t>(t0) * a.K;
      a.q += static_cast<int64_t>(t0) * a.K;
    }
    a.ms += t0;
    a.dot += t0;
    const cudaError_t e = type == 0   ? launch_type<__nv_bfloat16>(a, granule, blocks, stream)
                          : type == 1 ? launch_type<__half>(a, granule, blocks, stream)
                                      : launch_type<float>(a, granule, blocks, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tgemm
