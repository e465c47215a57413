// What the row kernels of the vocabulary-head losses share.
#pragma once

#include "loss_internal.h"
#include "ptx.cuh"

namespace tgemm {
namespace {

__device__ __forceinline__ unsigned char row_flag(const RowRule& a, int t) {
  if (!a.targets) return a.flags[t];
  const int64_t y = a.targets[t];
  if (y == a.ignore_index) return kRowIgnored;
  return (y >= 0 && y < a.V) ? kRowCounts : kRowBad;
}

// Joins two {maximum, sum of 2^(y - maximum)}.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.0f : top;
  s = s * exp2f(m - ref) + s2 * exp2f(m2 - ref);
  m = top;
}

}  // namespace
}  // namespace tgemm
