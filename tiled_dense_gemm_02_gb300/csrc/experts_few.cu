// The experts' products for a few places (a decoding step of one or two tokens), on
// the CUDA cores: every place reads its expert's weights once, a warp a row.
//
// Bound by the weights' bytes, 3 D F elements a place.  The tensor-core products need
// the places sorted first, four launches, and hold at most 112 KB of a weight in flight
// on 128 of 152 SMs; here two launches and eight or more 16-byte loads a lane stream
// them (one token, eight experts of 2048 x 1024: UP 24 and DOWN 12 us there, 13 and 8
// here).  Places that share an expert read its weights again, from L2, so only so few
// take this way (experts_api.cu).
//
// h stays fp32, and a token's sum over its experts stays in its warp: only the
// result is rounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts_internal.h"
#include "ptx.cuh"

namespace tgemm {
namespace {

constexpr int kFewWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float2 pair_values(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ float value(uint16_t w) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
  return __half2float(__ushort_as_half(w));
}

// acc += the eight products of two words of 16-bit values.
template <bool BF16>
__device__ __forceinline__ void dot_words(const uint4& a, const uint4& b, float2& acc) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __ffma2_rn(pair_values<BF16>(p[i]), pair_values<BF16>(q[i]), acc);
}
template <bool BF16>
__device__ __forceinline__ void dot_floats(const uint4& a, const float4& lo, const float4& hi, float2& acc) {
  acc = __ffma2_rn(pair_values<BF16>(a.x), make_float2(lo.x, lo.y), acc);
  acc = __ffma2_rn(pair_values<BF16>(a.y), make_float2(lo.z, lo.w), acc);
  acc = __ffma2_rn(pair_values<BF16>(a.z), make_float2(hi.x, hi.y), acc);
  acc = __ffma2_rn(pair_values<BF16>(a.w), make_float2(hi.z, hi.w), acc);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// A warp: place blockIdx.y, one feature's gate and up.
template <bool BF16>
__global__ void __launch_bounds__(kFewWarps * 32) few_up_kernel(const __grid_constant__ ExpertFewArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, f = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  const int place = blockIdx.y;
  const int64_t id = __ldg(a.ids + place);
  if (f >= a.F || id < 0 || id >= a.E) return;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + place / a.k * a.ldx;
  const uint16_t* gate = static_cast<const uint16_t*>(a.w_in) + (id * 2 * a.F + f) * a.ld_in;
  const uint16_t* up = gate + a.F * a.ld_in;
  const uint4 *x4 = reinterpret_cast<const uint4*>(x), *g4 = reinterpret_cast<const uint4*>(gate),
              *u4 = reinterpret_cast<const uint4*>(up);
  const int words = a.D / 8;
  float2 g = make_float2(0.0f, 0.0f), u = g;
  int i = lane;
  for (; i + 96 < words; i += 128) {
    uint4 vg[4], vu[4], vx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vg[j] = __ldcs(g4 + i + 32 * j);
      vu[j] = __ldcs(u4 + i + 32 * j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) vx[j] = __ldg(x4 + i + 32 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dot_words<BF16>(vg[j], vx[j], g);
      dot_words<BF16>(vu[j], vx[j], u);
    }
  }
  for (; i < words; i += 32) {
    const uint4 vx = __ldg(x4 + i);
    dot_words<BF16>(__ldcs(g4 + i), vx, g);
    dot_words<BF16>(__ldcs(u4 + i), vx, u);
  }
  for (int d = words * 8 + lane; d < a.D; d += 32) {
    const float v = value<BF16>(__ldg(x + d));
    g.x = fmaf(value<BF16>(__ldg(gate + d)), v, g.x);
    u.x = fmaf(value<BF16>(__ldg(up + d)), v, u.x);
  }
  const float gs = warp_sum(g.x + g.y), us = warp_sum(u.x + u.y);
  if (lane == 0) a.h[place * a.ldh + f] = gs / (1.0f + expf(-gs)) * us;
}

// A block: token blockIdx.y, kDownRows elements of out; a warp takes every kDownWarps-th of
// the token's places, so that all of them are read at once.
constexpr int kDownRows = 4, kDownWarps = 8;

template <bool BF16>
__global__ void __launch_bounds__(kDownWarps * 32) few_down_kernel(const __grid_constant__ ExpertFewArgs a) {
  __shared__ float sums[kDownWarps][kDownRows];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int t = blockIdx.y, d0 = blockIdx.x * kDownRows;
  const int words = a.F / 8;
  float sum[kDownRows];
#pragma unroll
  for (int r = 0; r < kDownRows; ++r) sum[r] = 0.0f;
  for (int j = warp; j < a.k; j += warps) {
    const int64_t id = __ldg(a.ids + t * a.k + j);
    if (id < 0) continue;
    if (id >= a.E) {
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) sum[r] = NAN;
      continue;
    }
    const float w = __ldg(a.weights + t * a.k + j);
    const uint16_t* rows[kDownRows];  // past the last element: the last row again, which is not stored
#pragma unroll
    for (int r = 0; r < kDownRows; ++r)
      rows[r] = static_cast<const uint16_t*>(a.w_out) + (id * a.D + min(d0 + r, a.D - 1)) * a.ld_out;
    const float* h = a.h + (t * a.k + j) * a.ldh;
    const float4* h4 = reinterpret_cast<const float4*>(h);
    float2 acc[kDownRows];
#pragma unroll
    for (int r = 0; r < kDownRows; ++r) acc[r] = make_float2(0.0f, 0.0f);
    int i = lane;
    for (; i + 32 < words; i += 64) {
      uint4 v[2][kDownRows];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int r = 0; r < kDownRows; ++r) v[q][r] = __ldcs(reinterpret_cast<const uint4*>(rows[r]) + i + 32 * q);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 lo = __ldcg(h4 + 2 * (i + 32 * q)), hi = __ldcg(h4 + 2 * (i + 32 * q) + 1);
#pragma unroll
        for (int r = 0; r < kDownRows; ++r) dot_floats<BF16>(v[q][r], lo, hi, acc[r]);
      }
    }
    for (; i < words; i += 32) {
      const float4 lo = __ldcg(h4 + 2 * i), hi = __ldcg(h4 + 2 * i + 1);
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) dot_floats<BF16>(__ldcs(reinterpret_cast<const uint4*>(rows[r]) + i), lo, hi, acc[r]);
    }
    for (int f = words * 8 + lane; f < a.F; f += 32) {
      const float v = __ldcg(h + f);
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) acc[r].x = fmaf(value<BF16>(__ldg(rows[r] + f)), v, acc[r].x);
    }
#pragma unroll
    for (int r = 0; r < kDownRows; ++r) sum[r] = fmaf(w, acc[r].x + acc[r].y, sum[r]);
  }
#pragma unroll
  for (int r = 0; r < kDownRows; ++r) {
    const float s = warp_sum(sum[r]);
    if (lane == 0) sums[warp][r] = s;
  }
  __syncthreads();
  const int d = d0 + threadIdx.x;
  if (threadIdx.x >= kDownRows || d >= a.D) return;
  float total = 0.0f;
  for (int w = 0; w < warps; ++w) total += sums[w][threadIdx.x];
  static_cast<uint16_t*>(a.out)[t * a.ldo + d] =
      BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(total)) : __half_as_ushort(__float2half_rn(total));
}

template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_experts_few(const ExpertFewArgs& a, bool bf16, cudaStream_t stream) {
  const dim3 up((a.F + kFewWarps - 1) / kFewWarps, a.T * a.k), down((a.D + kDownRows - 1) / kDownRows, a.T);
  const int threads = 32 * (a.k < kDownWarps ? a.k : kDownWarps);
  const cudaError_t e = launch_next(bf16 ? few_up_kernel<true> : few_up_kernel<false>, up, kFewWarps * 32, stream, a);
  if (e != cudaSuccess) return e;
  return launch_next(bf16 ? few_down_kernel<true> : few_down_kernel<false>, down, threads, stream, a);
}

}  // namespace tgemm
