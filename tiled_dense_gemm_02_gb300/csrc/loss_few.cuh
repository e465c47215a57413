// Row statistics, and the logits' gradient, of the vocabulary-head losses for a
// few rows on the CUDA cores: the scoring of single tokens and of up to eight where
// rows of W are off the 16-byte grid or fp32; steps on one or two tokens, and on up
// to eight in fp32 (loss_few_grad.cu).
//
// The work is one pass over W: 2 T V D operations against V D elements read.  Each
// warp takes four entries of W at a time, lane by lane in 16-byte pieces,
// multiplies them with the rows of H held in shared memory as fp32 (exact for
// 16-bit inputs), and keeps the running maximum and sum of a softmax for its
// entries; the warps share the vocabulary evenly.  Nothing is copied first: rows
// off the 16-byte grid are read in words of 4 or 2 bytes.  (Reading the aligned 16
// bytes around a piece and shifting between neighbouring lanes was slower: 236 us
// against 108 us for one row of 65536 x 4100, since every piece then waits for its
// load before the next.)
//
// Bound by memory.  Against the tensor-core product (its tiles nearly empty, W
// copied first if unaligned or fp32), 65536 x 4096: one bf16 row 94 us (5.7 TB/s)
// to 100 us; aligned bf16 rows from two on are the product's (two rows 113 us);
// eight rows at 4100 columns 192 to 329 us; eight fp32 rows 210 us (5.1 TB/s) to
// 1000 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "loss_rows.cuh"

namespace tgemm {
namespace {

constexpr int kEntries = 4;  // rows of W per warp and step
// Eight rows of H fill shared memory: one block of 16 warps per SM; with fewer
// rows, blocks of 8 warps, as many as registers allow.
constexpr int few_threads(int tn) { return tn == 8 ? 512 : 256; }
constexpr int few_per_sm(int tn) { return tn == 8 ? 1 : tn == 4 ? 2 : 4; }

template <typename E>
constexpr int lane_elems() { return 16 / static_cast<int>(sizeof(E)); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The 16 bytes of a row from element c on, as raw words; elements at or past
// `cols` read as zero.  G: alignment of the rows in bytes.
template <typename E, int G>
__device__ __forceinline__ uint4 load_piece(const E* row, int c, int cols) {
  constexpr int N = lane_elems<E>();
  if (G == 16 && c + N <= cols) return __ldg(reinterpret_cast<const uint4*>(row + c));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if constexpr (G >= 4) {
    constexpr int PER = 4 / static_cast<int>(sizeof(E));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + (i + 1) * PER <= cols)
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + c) + i);
      else if (PER == 2 && c + i * PER < cols)
        w[i] = __ldg(reinterpret_cast<const uint16_t*>(row + c) + 2 * i);
    }
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(row + c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) w[i / 2] |= static_cast<uint32_t>(__ldg(s + i)) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename E>
__device__ __forceinline__ void unpack(const uint4& p, float (&v)[lane_elems<E>()]) {
  const E* e = reinterpret_cast<const E*>(&p);
#pragma unroll
  for (int i = 0; i < lane_elems<E>(); ++i) v[i] = to_f32(e[i]);
}

// TN: rows of H, T rounded up to a power of two (the padding is zero).  GRAD:
// the gradient of the logits goes to dz[v][t] instead of statistics (0 for
// padding and for rows that do not count).
template <typename E, int TN, int G, bool GRAD>
__global__ void __launch_bounds__(few_threads(TN), few_per_sm(TN)) few_logits_kernel(const FewArgs a) {
  constexpr int N = lane_elems<E>();
  constexpr int THREADS = few_threads(TN), WARPS = THREADS / 32;
  constexpr int VALUES = kEntries * TN;  // sums a warp holds: 4 to 32
  extern __shared__ __align__(16) float s_h[];  // [t][half of the 16 bytes][group][4]
  __shared__ float s_part[3][WARPS][TN];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (a.D + N - 1) / N;
  for (int i = threadIdx.x; i < TN * groups; i += THREADS) {
    const int t = i / groups, g = i - t * groups;
    float v[N];
    if (t < a.T) {
      const E* row = static_cast<const E*>(a.H) + t * a.ldh;
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = g * N + j < a.D ? to_f32(row[g * N + j]) : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < N / 4; ++p)
      reinterpret_cast<float4*>(s_h)[(t * (N / 4) + p) * groups + g] =
          make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
  }
  __syncthreads();

  // after the reduction lane l holds the sum of value l / (32 / VALUES)
  const int value = lane / (32 / VALUES);
  const int t = value % TN, r = value / TN;
  const bool owner = lane % (32 / VALUES) == 0 && t < a.T;
  // this lane's row: its target, or its list walked as the entries ascend
  int next = INT_MAX, pos = 0;
  const int64_t list = static_cast<int64_t>(t) * a.K;
  if (owner) {
    if (a.targets) {
      const int64_t y = a.targets[t];
      next = y >= 0 && y < a.V ? static_cast<int>(y) : INT_MAX;
    } else {
      next = a.ids[list];
    }
  }
  float m = -INFINITY, s = 0.0f, dot = 0.0f, zs = 0.0f;
  float cp = 0.0f, cq = 0.0f, lse = 0.0f;
  bool counts = false;
  if (GRAD && owner) {
    counts = row_flag(a.rule, t) == kRowCounts;
    lse = a.lse[t];
    cq = a.grad[t] * a.scale;
    cp = a.z_loss == 0.0f ? cq : cq * (1.0f + 2.0f * a.z_loss * lse);
  }

  // an even share of the vocabulary, one after another; the groups of a last,
  // incomplete step repeat its last entry, which costs no memory traffic
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * WARPS + warp, workers = static_cast<int64_t>(gridDim.x) * WARPS;
  const int v_end = static_cast<int>(a.V * (worker + 1) / workers);
  for (int v0 = static_cast<int>(a.V * worker / workers); v0 < v_end; v0 += kEntries) {
    const E* rows[kEntries];
#pragma unroll
    for (int e = 0; e < kEntries; ++e)
      rows[e] = static_cast<const E*>(a.W) + static_cast<int64_t>(min(v0 + e, v_end - 1)) * a.ldw;
    float2 acc[VALUES];
#pragma unroll
    for (int i = 0; i < VALUES; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll(TN == 8 ? 1 : 2)
    for (int g = lane; g < groups; g += 32) {
      uint4 p[kEntries];
#pragma unroll
      for (int e = 0; e < kEntries; ++e) p[e] = load_piece<E, G>(rows[e], g * N, a.D);
      float w[kEntries][N];
#pragma unroll
      for (int e = 0; e < kEntries; ++e) unpack<E>(p[e], w[e]);
#pragma unroll
      for (int q = 0; q < TN; ++q)
#pragma unroll
        for (int hf = 0; hf < N / 4; ++hf) {
          const float4 h = reinterpret_cast<const float4*>(s_h)[(q * (N / 4) + hf) * groups + g];
#pragma unroll
          for (int e = 0; e < kEntries; ++e) {
            float2& c = acc[e * TN + q];
            c = __ffma2_rn(make_float2(w[e][4 * hf], w[e][4 * hf + 1]), make_float2(h.x, h.y), c);
            c = __ffma2_rn(make_float2(w[e][4 * hf + 2], w[e][4 * hf + 3]), make_float2(h.z, h.w), c);
          }
        }
    }
    // each step halves the values a lane holds and the lanes that share one
    float z[VALUES];
#pragma unroll
    for (int i = 0; i < VALUES; ++i) z[i] = acc[i].x + acc[i].y;
    int o = 16;
#pragma unroll
    for (int n = VALUES; n > 1; n >>= 1, o >>= 1)
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float mine = (lane & o) ? z[i + n / 2] : z[i];
        const float theirs = (lane & o) ? z[i] : z[i + n / 2];
        z[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
      }
    float sum = z[0];
#pragma unroll
    for (; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int v = v0 + r;
    if constexpr (GRAD) {
      if (lane % (32 / VALUES) == 0 && v < v_end) {
        float d = 0.0f;
        if (owner && counts) {
          d = fmaf(cp, expf(fmaf(sum, a.scale, -lse)), -cq * a.flat);
          while (next <= v) {
            if (next == v) d -= cq * (a.targets ? a.mass : a.q[list + pos]);
            ++pos;
            next = !a.targets && pos < a.K ? a.ids[list + pos] : INT_MAX;
          }
        }
        a.dz[static_cast<int64_t>(v) * TN + t] = d;
      }
    } else if (owner && v < v_end) {
      join(m, s, sum * a.k2, 1.0f);
      zs += sum;
      while (next < v) {  // entries other warps and lanes take
        ++pos;
        next = !a.targets && pos < a.K ? a.ids[list + pos] : INT_MAX;
      }
      while (next == v) {
        dot = fmaf(a.targets ? a.mass : a.q[list + pos], sum, dot);
        ++pos;
        next = !a.targets && pos < a.K ? a.ids[list + pos] : INT_MAX;
      }
    }
  }
  if constexpr (GRAD) return;
  if (a.flat != 0.0f) dot = fmaf(a.flat, zs, dot);  // 0 times the sum of an infinite logit is no number
  // the warp's entries of one row, then the block's warps, in fixed order
  if (!owner) {
    m = -INFINITY;
    s = dot = 0.0f;
  }
#pragma unroll
  for (int o = 32 / kEntries; o < 32; o <<= 1) {  // lanes that differ in r
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float d2 = __shfl_xor_sync(0xffffffffu, dot, o);
    join(m, s, m2, s2);
    dot += d2;
  }
  if (lane % (32 / VALUES) == 0 && r == 0) {
    s_part[0][warp][t] = m;
    s_part[1][warp][t] = s;
    s_part[2][warp][t] = dot;
  }
  __syncthreads();
  if (threadIdx.x < a.T) {
    const int q = threadIdx.x;
    m = s_part[0][0][q];
    s = s_part[1][0][q];
    dot = s_part[2][0][q];
    for (int w = 1; w < WARPS; ++w) {
      join(m, s, s_part[0][w][q], s_part[1][w][q]);
      dot += s_part[2][w][q];
    }
    a.ms[static_cast<int64_t>(blockIdx.x) * a.ld_stats + q] = make_float2(m, s);
    a.dot[static_cast<int64_t>(blockIdx.x) * a.ld_stats + q] = dot;
  }
}

// Launch dependent on the kernel before it.
template <typename Args>
cudaError_t launch_few_kernel(void (*kernel)(Args), const Args& a, dim3 grid, int threads, int smem,
                              std::atomic<uint64_t>& done_mask, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (smem && !(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename E, int TN, int G, bool GRAD>
cudaError_t launch_logits(const FewArgs& a, int blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  const int groups = (a.D + lane_elems<E>() - 1) / lane_elems<E>();
  return launch_few_kernel(few_logits_kernel<E, TN, G, GRAD>, a, dim3(blocks), few_threads(TN),
                           TN * groups * lane_elems<E>() * 4, done_mask, stream);
}

inline int rows_held(int64_t T) { return T <= 1 ? 1 : T <= 2 ? 2 : T <= 4 ? 4 : 8; }

}  // namespace
}  // namespace tgemm
