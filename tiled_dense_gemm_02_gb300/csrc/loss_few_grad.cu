// Backward of the vocabulary-head losses for a few rows: dz by the logits' kernel
// (loss_few.cuh), then dW = dz^T H and dH = dz W in one pass that reads W and
// writes dW; dz and all sums are fp32.  Bound by memory: W twice, dW once.
//
// A thread owns one 16-byte piece of the columns.  It holds those columns of H
// and of the sums of dH in registers for all rows of H and walks its share of the
// vocabulary: a piece of W in, T multiply-adds an element into the sums, T
// multiply-adds into the piece of dW that goes out.  Where a row has few pieces,
// groups of warps take different entries; their sums join in order at the end.
//
// Against the tensor-core products, a backward call on 65536 x 4096: bf16 one row
// 316 to 353 us, two 335 to 353, from three on the products' (350 to 390 here); off
// the 16-byte grid, where dW leaves in words of 8 bytes or less, the products' (at
// 4100 columns one row 807 to 647 us); fp32 one row 536 us (6.0 TB/s), two 619, four
// 588 (with the 16-byte loads of dz and the 128 registers that two rows do not
// have), eight 671 (144 registers, one block an SM, took 920) to 1730 us.
#include "loss_few.cuh"

namespace tgemm {
namespace {

constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32;
constexpr int kGradUnroll = 4;  // entries whose loads are in flight together

__device__ __forceinline__ void round_to(float v, float& o) { o = v; }
__device__ __forceinline__ void round_to(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void round_to(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// This lane's 16 bytes of a row of dW whose warp holds columns [c0, c0 + 32 N):
// in one piece where rows are aligned, else through shared memory, neighbouring
// lanes writing neighbouring words.
template <typename E>
__device__ __forceinline__ void store_piece(E* row, int c0, int cols, const uint4& p, int granule, uint4* stage,
                                            int lane) {
  constexpr int N = lane_elems<E>();
  if (granule == 16) {
    const int c = c0 + lane * N;
    if (c + N <= cols) {
      *reinterpret_cast<uint4*>(row + c) = p;
    } else {
      const E* e = reinterpret_cast<const E*>(&p);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) row[c + i] = e[i];
    }
    return;
  }
  __syncwarp();
  stage[lane] = p;
  __syncwarp();
  if (sizeof(E) == 2 && granule >= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = i * 32 + lane, c = c0 + 2 * w;
      if (c + 2 <= cols)
        *reinterpret_cast<uint32_t*>(row + c) = reinterpret_cast<const uint32_t*>(stage)[w];
      else if (c < cols)
        row[c] = reinterpret_cast<const E*>(stage)[2 * w];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * 32 + lane;
      if (c < cols) row[c] = reinterpret_cast<const E*>(stage)[i * 32 + lane];
    }
  }
}

// The gradients of one entry's logits, or zeros.
template <int TN>
__device__ __forceinline__ void load_dz(float (&d)[TN], const float* src, bool in) {
  if constexpr (TN >= 4) {
#pragma unroll
    for (int t = 0; t < TN; t += 4) {
      const float4 x = in ? __ldcg(reinterpret_cast<const float4*>(src + t)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      d[t] = x.x;
      d[t + 1] = x.y;
      d[t + 2] = x.z;
      d[t + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int t = 0; t < TN; ++t) d[t] = in ? __ldcg(src + t) : 0.0f;
  }
}

template <typename E, int TN, bool ALIGNED>
__global__ void __launch_bounds__(kGradThreads, TN >= 4 ? 2 : 1) few_grad_kernel(const FewGradArgs a) {
  constexpr int N = lane_elems<E>();
  constexpr int G = ALIGNED ? 16 : static_cast<int>(sizeof(E));
  __shared__ float s_sum[kGradThreads * N];
  __shared__ uint4 s_stage[kGradWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = blockIdx.y * kGradThreads;  // of the columns' pieces
  const int here = min(kGradThreads, (a.D + N - 1) / N - first);
  const int wide = (here + 31) / 32, groups = kGradWarps / wide;  // warps an entry, entries at a time
  const int group = warp / wide, slot = warp % wide;
  const int c0 = (first + slot * 32) * N, c = c0 + lane * N;
  const bool on = group < groups && slot * 32 + lane < here;

  float h[TN][N], sum[TN][N];
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const bool counts = on && t < a.T && row_flag(a.rule, t) == kRowCounts;
    const E* row = static_cast<const E*>(a.H) + t * a.ldh;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      h[t][i] = counts && c + i < a.D ? to_f32(row[c + i]) : 0.0f;
      sum[t][i] = 0.0f;
    }
  }
  const int lo = static_cast<int>(static_cast<int64_t>(a.V) * blockIdx.x / a.shares);
  const int hi = static_cast<int>(static_cast<int64_t>(a.V) * (blockIdx.x + 1) / a.shares);
  if (group < groups) {
    for (int v0 = lo + group; v0 < hi; v0 += groups * kGradUnroll) {
      uint4 p[kGradUnroll];
      float d[kGradUnroll][TN];
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u) {
        const int v = v0 + u * groups;
        const bool in = v < hi;
        p[u] = in && on && a.acc ? load_piece<E, G>(static_cast<const E*>(a.W) + static_cast<int64_t>(v) * a.ldw, c, a.D)
                                 : make_uint4(0u, 0u, 0u, 0u);
        load_dz<TN>(d[u], a.dz + static_cast<int64_t>(v) * TN, in);
      }
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u) {
        const int v = v0 + u * groups;
        if (v >= hi) break;
        if (a.acc) {
          float w[N];
          unpack<E>(p[u], w);
#pragma unroll
          for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int i = 0; i < N; ++i) sum[t][i] = fmaf(d[u][t], w[i], sum[t][i]);
        }
        if (a.dW) {
          uint4 o;
          E* e = reinterpret_cast<E*>(&o);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float x = 0.0f;
#pragma unroll
            for (int t = 0; t < TN; ++t) x = fmaf(d[u][t], h[t][i], x);
            round_to(x, e[i]);
          }
          store_piece(static_cast<E*>(a.dW) + static_cast<int64_t>(v) * a.lddw, c0, a.D, o, a.store_granule,
                      s_stage[warp], lane);
        }
      }
    }
  }
  if (!a.acc) return;
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    if (t >= a.T) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s_sum[threadIdx.x * N + i] = sum[t][i];
    __syncthreads();
    if (on && group == 0) {
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = sum[t][i];
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += s_sum[(threadIdx.x + g * wide * 32) * N + i];
      float* out = a.acc + (static_cast<int64_t>(blockIdx.x) * a.T + t) * a.ld_acc + c;
#pragma unroll
      for (int i = 0; i < N; i += 4)  // the pitch is a multiple of four
        if (c + i < a.ld_acc)
          *reinterpret_cast<float4*>(out + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
  }
}

template <typename E, int TN, bool ALIGNED>
cudaError_t launch_both(const FewArgs& f, const FewGradArgs& g, int blocks, cudaStream_t stream) {
  constexpr int G = ALIGNED ? 16 : static_cast<int>(sizeof(E));
  cudaError_t e = launch_logits<E, TN, G, true>(f, blocks, stream);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> done_mask{0};
  const int pieces = (g.D + lane_elems<E>() - 1) / lane_elems<E>();
  return launch_few_kernel(few_grad_kernel<E, TN, ALIGNED>, g,
                           dim3(g.shares, (pieces + kGradThreads - 1) / kGradThreads), kGradThreads, 0, done_mask,
                           stream);
}

template <typename E, bool ALIGNED>
cudaError_t launch_rows(const FewArgs& f, const FewGradArgs& g, int blocks, cudaStream_t stream) {
  if constexpr (sizeof(E) == 4 || ALIGNED) {
    if (f.T <= 1) return launch_both<E, 1, ALIGNED>(f, g, blocks, stream);
    if (f.T <= 2) return launch_both<E, 2, ALIGNED>(f, g, blocks, stream);
  }
  if constexpr (sizeof(E) == 4) {
    if (f.T <= 4) return launch_both<E, 4, ALIGNED>(f, g, blocks, stream);
    return launch_both<E, 8, ALIGNED>(f, g, blocks, stream);
  }
  return cudaErrorInvalidValue;  // 16-bit rows past these take the tensor cores
}

template <typename E>
cudaError_t launch_type(const FewArgs& f, const FewGradArgs& g, bool aligned, int blocks, cudaStream_t stream) {
  return aligned ? launch_rows<E, true>(f, g, blocks, stream) : launch_rows<E, false>(f, g, blocks, stream);
}

}  // namespace

int few_held(int64_t T) { return rows_held(T); }

int few_shares(int64_t V, int64_t D, bool f32) {
  // four blocks an SM over the columns' chunks, each with entries for all its warps
  const int64_t chunk = kGradThreads * (f32 ? 4 : 8), chunks = (D + chunk - 1) / chunk;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4 * kFewSms / chunks, V / 32)));
}

cudaError_t launch_few_grad(const FewArgs& f, const FewGradArgs& g, int type, bool aligned, int blocks,
                            cudaStream_t stream) {
  if (type == 0) return launch_type<__nv_bfloat16>(f, g, aligned, blocks, stream);
  if (type == 1) return launch_type<__half>(f, g, aligned, blocks, stream);
  return launch_type<float>(f, g, aligned, blocks, stream);
}

}  // namespace tgemm
