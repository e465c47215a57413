// The gated activation and its gradient (experts_gemm.cuh, experts_rows.cu).
#pragma once

namespace tgemm {
namespace {

__device__ __forceinline__ float fast_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// h = g s u, dg = wv u s (1 + g (1 - s)), du = wv g s, with s = sigmoid(g) and wv the weight times
// the gradient of h.
struct GatedGradient {
  float h, dg, du;
};
__device__ __forceinline__ GatedGradient gated_gradient(float g, float u, float wv) {
  const float s = fast_sigmoid(g), silu = g * s;
  return {silu * u, wv * u * fmaf(silu, 1.0f - s, s), wv * silu};
}

}  // namespace
}  // namespace tgemm
