// Row kernels of the vocabulary-head losses: the teacher's lists, the gather of
// the rows that count, the joining of the tiles' statistics, the last step of
// dH, and the bf16 planes of fp32 operands.  All of them are bound by memory or
// by latency and move a small part of what the products do.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "loss_rows.cuh"

namespace tgemm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Every kernel of a call is launched as a programmatic dependent of the one
// before it: its blocks may be set up while that one ends, and touch memory
// only after it has completed.  Each kernel waits before it does anything, so
// completion carries over the whole chain.
__device__ __forceinline__ void chain() {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), int64_t blocks, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------ teacher lists
// One warp per row: softmax over the used places, then the places in ascending
// order of their ids (each place's rank by counting, ties by position), so that
// a tile of the product finds its entries by a binary search.
constexpr int kListWarps = 4;
constexpr int kListMax = 256;  // TGEMM_DISTILL_MAX_K
__global__ void __launch_bounds__(kListWarps * 32)
    distill_lists_kernel(const int64_t* __restrict__ ids, int64_t ld_ids, const float* __restrict__ logits,
                         int64_t ld_logits, int T, int V, int K, float scale, HeadRows rows) {
  __shared__ int s_id[kListWarps][kListMax];
  chain();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kListWarps + warp;
  if (t >= T) return;
  constexpr int PER = kListMax / 32;
  float y[PER];
  int id[PER];
  float top = -INFINITY;
  bool some = false, bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int k = lane + 32 * j;
    id[j] = INT_MAX;
    y[j] = -INFINITY;
    if (k >= K) continue;
    const int64_t v = ids[t * ld_ids + k];
    if (v >= 0) {
      bad |= v >= V;
      id[j] = v >= V ? INT_MAX : static_cast<int>(v);
      y[j] = logits[t * ld_logits + k];
      some |= !(y[j] == -INFINITY);
      top = fmaxf(top, y[j]);
    }
    s_id[warp][k] = id[j];
  }
  bad = __any_sync(0xffffffffu, bad);
  some = __any_sync(0xffffffffu, some);
  top = warp_max(top);
  // scaled after the maximum is taken off: a multiple of the type's lowest or
  // largest value would leave fp32's range
  float e[PER], total = 0.0f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool none = y[j] == -INFINITY;
    y[j] = (y[j] - top) * scale;
    e[j] = none ? 0.0f : expf(y[j]);
    total += e[j];
  }
  total = warp_sum(total);
  const float log_total = logf(total);
  float own = 0.0f;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int k = lane + 32 * j;
    if (k >= K) continue;
    const float q = some ? e[j] / total : 0.0f;
    own += q == 0.0f ? 0.0f : q * (y[j] - log_total);
    int rank = 0;
    for (int i = 0; i < K; ++i) {
      const int other = s_id[warp][i];
      rank += (other < id[j] || (other == id[j] && i < k)) ? 1 : 0;
    }
    const int64_t at = static_cast<int64_t>(t) * K + rank;
    rows.ids[at] = id[j];
    rows.q[at] = q;
  }
  own = warp_sum(own);
  if (lane == 0) {
    rows.own[t] = own;
    rows.flags[t] = bad ? kRowBad : some ? kRowCounts : kRowIgnored;
  }
}

// ---------------------------------------------------------------- the gather
// loss and lse of a row that does not count
__device__ __forceinline__ float row_value(unsigned char flag) {
  return flag == kRowBad ? __int_as_float(0x7FC00000) : 0.0f;
}

__device__ __forceinline__ float grad_p(const GatherArgs& a, int t) {
  const float g = a.grad[t];
  return a.z_loss == 0.0f ? g : g * (1.0f + 2.0f * a.z_loss * a.lse[t]);
}

// Copies `count` rows of `bytes` (a multiple of G) each, src[r] -> dst + r *
// pitch, with the whole block.
template <int G>
__device__ __forceinline__ void copy_rows(uint8_t* dst, int64_t pitch, const uint8_t* H, int64_t src_pitch,
                                          const int* src, int count, int bytes) {
  using Word = typename std::conditional<
      G == 16, uint4, typename std::conditional<G == 8, uint2, typename std::conditional<G == 4, uint32_t, uint16_t>::type>::type>::type;
  const int words = bytes / G;
  if (count * words <= 2 * static_cast<int>(blockDim.x) || words >= static_cast<int>(blockDim.x)) {
    // long rows, one after another, or hardly any work
    for (int r = 0; r < count; ++r) {
      const Word* s = reinterpret_cast<const Word*>(H + static_cast<int64_t>(src[r]) * src_pitch);
      Word* d = reinterpret_cast<Word*>(dst + r * pitch);
#pragma unroll 4
      for (int i = threadIdx.x; i < words; i += blockDim.x) d[i] = s[i];
    }
  } else {  // short rows, one per warp
    for (int r = threadIdx.x >> 5; r < count; r += blockDim.x >> 5) {
      const Word* s = reinterpret_cast<const Word*>(H + static_cast<int64_t>(src[r]) * src_pitch);
      Word* d = reinterpret_cast<Word*>(dst + r * pitch);
#pragma unroll 4
      for (int i = threadIdx.x & 31; i < words; i += 32) d[i] = s[i];
    }
  }
}

// A finite value past bf16's largest would round to infinity.
__device__ __forceinline__ float within_bf16(float x) {
  constexpr float most = 3.38953139e38f;  // (2 - 2^-7) 2^127
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -most), most) : x;
}

// An fp32 row as three bf16 planes.  A value that is not finite goes to the
// first plane alone.  `lanes` threads, four elements each; the planes' pitch is a
// multiple of 8, so whole groups are written.
__device__ __forceinline__ void split_row(uint16_t* dst, int64_t plane, const float* src, int cols, bool vec,
                                          int lane, int lanes) {
#pragma unroll 2
  for (int c = lane * 4; c < cols; c += 4 * lanes) {
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (vec && c + 4 <= cols) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + c));
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < cols) x[i] = __ldg(src + c + i);
    }
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(within_bf16(x[2 * i]), within_bf16(x[2 * i + 1]));
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
        const float lo = __low2float(b), hi = __high2float(b);
        x[2 * i] = isfinite(lo) ? x[2 * i] - lo : 0.0f;
        x[2 * i + 1] = isfinite(hi) ? x[2 * i + 1] - hi : 0.0f;
      }
      *reinterpret_cast<uint2*>(dst + p * plane + c) = make_uint2(w[0], w[1]);
    }
  }
}

// Every block counts the rows that count over all T (their flags are a few KB
// in L2) to know where its own go, so the gather is one launch with a fixed
// order.  In the backward pass it also finds the largest |grad|, which the
// 16-bit gradients are divided by: a mean's 1/n is then exactly 1, and small
// gradients do not fall below the format's range.
constexpr int kGatherThreads = 256;
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherArgs a, int rows_per) {
  __shared__ int s_before[kGatherThreads / 32], s_total[kGatherThreads / 32], s_warp[kGatherThreads / 32];
  __shared__ float s_g[kGatherThreads / 32], s_c[kGatherThreads / 32], s_least[kGatherThreads / 32];
  __shared__ int s_src[kGatherThreads];
  chain();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * rows_per, t1 = min(a.T, t0 + rows_per);
  int before = 0, total = 0;
  float gmax = 0.0f, cmax = 0.0f, least = INFINITY;  // least: the smallest row's larger coefficient
  // nothing in the loop waits for a row's flag, so the loads of several rows overlap
#pragma unroll 8
  for (int t = tid; t < a.T; t += kGatherThreads) {
    const bool counts = row_flag(a.rule, t) == kRowCounts;
    total += counts ? 1 : 0;
    before += counts && t < t0 ? 1 : 0;
    if (a.grad) {
      const float g = fabsf(a.grad[t]), c = a.z_loss == 0.0f ? g : fabsf(grad_p(a, t));
      gmax = counts && isfinite(g) ? fmaxf(gmax, g) : gmax;
      cmax = counts && isfinite(c) ? fmaxf(cmax, c) : cmax;
      const float both = fmaxf(g, c);
      least = counts && both > 0.0f ? fminf(least, both) : least;
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  gmax = warp_max(gmax);
  cmax = warp_max(cmax);
  least = -warp_max(-least);
  const int t = t0 + tid;
  const unsigned char flag = t < t1 ? row_flag(a.rule, t) : kRowIgnored;
  const unsigned ballot = __ballot_sync(0xffffffffu, flag == kRowCounts);
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
    s_g[warp] = gmax;
    s_c[warp] = cmax;
    s_least[warp] = least;
    s_warp[warp] = __popc(ballot);
  }
  __syncthreads();
  before = total = 0;
  gmax = cmax = 0.0f;
  int mine = 0, local = 0;
#pragma unroll
  for (int w = 0; w < kGatherThreads / 32; ++w) {
    before += s_before[w];
    total += s_total[w];
    gmax = fmaxf(gmax, s_g[w]);
    cmax = fmaxf(cmax, s_c[w]);
    least = fminf(least, s_least[w]);
    if (w < warp) local += s_warp[w];
    mine += s_warp[w];
  }
  // unit * pow >= every |coefficient|; pow (a power of two) only where z_loss
  // makes the softmax's coefficient larger than the target's
  const float unit = gmax > 0.0f ? gmax : 1.0f;
  float pow2 = 1.0f;
  if (cmax > unit) {
    int e;
    const float f = frexpf(cmax / unit, &e);
    pow2 = exp2f(static_cast<float>(min(f == 0.5f ? e - 1 : e, 60)));
  }
  const bool spread = a.rows.spread && least < kSpread * (unit * pow2);
  if (blockIdx.x == 0 && tid == 0) {
    *a.rows.count = total;
    if (a.rows.spread) *a.rows.spread = spread ? 1 : 0;
    if (a.grad) *a.rows.factor = unit * (a.scale * pow2 / a.range);
  }
  if (t < t1) {
    const int place = before + local + __popc(ballot & ((1u << lane) - 1u));
    const bool counts = flag == kRowCounts;
    a.rows.place[t] = counts ? place : -1;
    if (counts) {
      a.rows.source[place] = t;
      if (a.rule.targets) a.rows.target[place] = a.rule.targets[t];
      s_src[place - before] = t;
      if (a.grad) {
        const float up = a.range / pow2;
        const float cp = grad_p(a, t) / unit * up, cq = a.grad[t] / unit * up;
        float own = 1.0f;
        const float size = fmaxf(fabsf(cp), fabsf(cq)) / a.range;  // of the row, at most 1
        if (spread && size > 0.0f && isfinite(size)) {
          int e;
          frexpf(size, &e);
          own = exp2f(static_cast<float>(min(max(-e, 0), 100)));
        }
        a.rows.coef[place] = make_float4(cp, cq, a.lse[t] * kLog2e, own);
      }
    } else if (a.loss_out) {
      a.loss_out[t] = a.lse_out[t] = row_value(flag);
    }
  }
  __syncthreads();
  uint16_t* const out = static_cast<uint16_t*>(a.rows.h);
  if (a.es == 4) {
    // a row per warp, or the block's warps share rows too few for them
    const int per = mine < kGatherThreads / 32 ? kGatherThreads / 32 / max(1, mine) : 1;  // warps per row
    for (int r = warp / per; r < mine; r += kGatherThreads / 32 / per)
      split_row(out + static_cast<int64_t>(before + r) * a.rows.ldh, a.rows.plane,
                static_cast<const float*>(a.H) + static_cast<int64_t>(s_src[r]) * a.ldh, a.D, a.granule == 16,
                (warp % per) * 32 + lane, 32 * per);
  } else {
    uint8_t* dst = reinterpret_cast<uint8_t*>(out + static_cast<int64_t>(before) * a.rows.ldh);
    const uint8_t* H = static_cast<const uint8_t*>(a.H);
    const int64_t pitch = a.rows.ldh * 2, src_pitch = a.ldh * 2;
    const int bytes = a.D * 2;
    int g = a.granule;
    while (bytes % g) g >>= 1;
    switch (g) {
      case 16: copy_rows<16>(dst, pitch, H, src_pitch, s_src, mine, bytes); break;
      case 8: copy_rows<8>(dst, pitch, H, src_pitch, s_src, mine, bytes); break;
      case 4: copy_rows<4>(dst, pitch, H, src_pitch, s_src, mine, bytes); break;
      default: copy_rows<2>(dst, pitch, H, src_pitch, s_src, mine, bytes); break;
    }
  }
  // zeros from the last gathered row to the end of its block of rows, which
  // the products read (the pitch is a multiple of 16 bytes)
  const int64_t blocks = max(1, (total + kRowBlock - 1) / kRowBlock);
  const int end = static_cast<int>(min(static_cast<int64_t>(a.T), blocks * kRowBlock));
  const int planes = a.es == 4 ? kPlanes : 1;
  for (int r = total + blockIdx.x * (kGatherThreads / 32) + warp; r < end; r += gridDim.x * (kGatherThreads / 32))
    for (int p = 0; p < planes; ++p) {
      uint4* dst = reinterpret_cast<uint4*>(out + p * a.rows.plane + static_cast<int64_t>(r) * a.rows.ldh);
      for (int64_t i = lane; i < a.rows.ldh / 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// --------------------------------------------------- joining tile statistics
// A block of 256 threads joins the parts of ROWS rows: 8 (64 contiguous bytes
// of a part are read at a time), or 1 where there are too few rows to fill the
// SMs and a row's parts are spread over the whole block.
constexpr int kCombineThreads = 256;
template <int ROWS>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const float2* ms, const float* dot, int tiles, int T, float scale,
                   float z_loss, HeadRows rows, RowRule rule, float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int SLOTS = kCombineThreads / ROWS;
  __shared__ float s_m[SLOTS][ROWS], s_s[SLOTS][ROWS], s_d[SLOTS][ROWS];
  chain();
  const int n = rows.count ? min(*rows.count, T) : T;
  const int r0 = blockIdx.x * ROWS;
  if (r0 >= n) return;
  const int lr = threadIdx.x % ROWS, slot = threadIdx.x / ROWS;
  const int r = r0 + lr;
  float m = -INFINITY, s = 0.0f, d = 0.0f;
  if (r < n) {
#pragma unroll 4
    for (int i = slot; i < tiles; i += SLOTS) {
      const float2 p = __ldcg(ms + static_cast<int64_t>(i) * T + r);
      d += __ldcg(dot + static_cast<int64_t>(i) * T + r);
      join(m, s, p.x, p.y);
    }
  }
  s_m[slot][lr] = m;
  s_s[slot][lr] = s;
  s_d[slot][lr] = d;
  __syncthreads();
  for (int w = SLOTS / 2; w > 0; w >>= 1) {
    if (slot < w) {
      float m1 = s_m[slot][lr], s1 = s_s[slot][lr];
      join(m1, s1, s_m[slot + w][lr], s_s[slot + w][lr]);
      s_m[slot][lr] = m1;
      s_s[slot][lr] = s1;
      s_d[slot][lr] += s_d[slot + w][lr];
    }
    __syncthreads();
  }
  if (slot == 0 && r < n) {
    const int t = rows.source ? rows.source[r] : r;
    const float l = s_m[0][lr] * kLn2 + logf(s_s[0][lr]);
    float v = (rows.own ? rows.own[t] : 0.0f) + (l - scale * s_d[0][lr]);
    if (z_loss != 0.0f) v = fmaf(z_loss * l, l, v);
    const unsigned char flag = rows.count ? kRowCounts : row_flag(rule, t);
    loss[t] = flag == kRowCounts ? v : row_value(flag);
    lse[t] = flag == kRowCounts ? l : row_value(flag);
  }
}

// ------------------------------------------------------------ last step of dH
template <typename Out>
__device__ __forceinline__ Out to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half to_out<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Four columns of one row per thread; the sums' pitch is a multiple of four.
// LANES threads share the splits of the same columns (8 for many splits, which
// one thread would read one after another); their sums join in a fixed order.
constexpr int kFinishThreads = 128;
template <typename Out, int LANES>
__global__ void __launch_bounds__(kFinishThreads) finish_dh_kernel(const float* acc, int64_t ld_acc,
                                                                   int64_t split_stride, int splits, int T, int D,
                                                                   HeadRows rows, RowRule rule, Out* __restrict__ dH,
                                                                   int64_t lddh, int wide) {
  chain();
  const int groups = (D + 3) / 4;
  const int lane = threadIdx.x % LANES;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kFinishThreads / LANES) + threadIdx.x / LANES;
  const int64_t row = i / groups;
  const int c = static_cast<int>(i - row * groups) * 4;
  const bool inside = row < T;
  const int t = inside ? static_cast<int>(row) : 0;
  // without gathered rows a row's sums are in its own place
  const int place = !inside ? -1 : rows.place ? rows.place[t] : row_flag(rule, t) == kRowCounts ? t : -1;
  const float f = !rows.factor ? 1.0f : rows.spread && place >= 0 ? *rows.factor / rows.coef[place].w : *rows.factor;
  Out* out = dH + static_cast<int64_t>(t) * lddh + c;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (place >= 0) {
    const float* src = acc + static_cast<int64_t>(place) * ld_acc + c;
#pragma unroll 8
    for (int s = lane; s < splits; s += LANES) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(src + s * split_stride));
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  if (!inside || lane != 0) return;
  // no sum of a row that does not count: its place holds zeros whatever f is
  if (place >= 0) {
    v.x *= f;
    v.y *= f;
    v.z *= f;
    v.w *= f;
  }
  const Out o[4] = {to_out<Out>(v.x), to_out<Out>(v.y), to_out<Out>(v.z), to_out<Out>(v.w)};
  if (wide && c + 4 <= D) {
    if constexpr (sizeof(Out) == 4)
      *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(o);
    else
      *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < D) out[j] = o[j];
  }
}

// One block per 4 rows of an fp32 matrix, read once and written as planes.
__global__ void __launch_bounds__(128) split_kernel(const float* __restrict__ W, int64_t ldw, uint16_t* __restrict__ out,
                                                    int64_t ld_out, int64_t plane, int rows, int cols, int vec) {
  chain();
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  split_row(out + r * ld_out, plane, W + r * ldw, cols, vec != 0, threadIdx.x & 31, 32);
}

}  // namespace

cudaError_t launch_distill_lists(const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits, int T,
                                 int V, int K, float scale, const HeadRows& rows, cudaStream_t stream) {
  return launch_chained(distill_lists_kernel, (T + kListWarps - 1) / kListWarps, kListWarps * 32, stream, ids, ld_ids,
                        logits, ld_logits, T, V, K, scale, rows);
}

cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream) {
  // a few blocks per SM, at most one row per thread of a block
  const int target = 4 * sms;
  int rows_per = (a.T + target - 1) / target;
  if (rows_per > kGatherThreads) rows_per = kGatherThreads;
  return launch_chained(gather_kernel, (a.T + rows_per - 1) / rows_per, kGatherThreads, stream, a, rows_per);
}

cudaError_t launch_combine(const float2* ms, const float* dot, int tiles, int T, float scale, float z_loss,
                           const HeadRows& rows, const RowRule& rule, float* loss, float* lse, cudaStream_t stream) {
  if (T <= 1024)
    return launch_chained(combine_kernel<1>, T, kCombineThreads, stream, ms, dot, tiles, T, scale, z_loss, rows, rule,
                          loss, lse);
  return launch_chained(combine_kernel<8>, (T + 7) / 8, kCombineThreads, stream, ms, dot, tiles, T, scale, z_loss, rows,
                        rule, loss, lse);
}

cudaError_t launch_finish_dh(const float* acc, int64_t ld_acc, int64_t split_stride, int splits, int T, int D,
                             const HeadRows& rows, const RowRule& rule, int type, void* dH, int64_t lddh,
                             cudaStream_t stream) {
  const int es = type == 2 ? 4 : 2;
  const int wide = reinterpret_cast<uint64_t>(dH) % (4 * es) == 0 && lddh % 4 == 0 ? 1 : 0;
  const int lanes = splits >= 8 ? 8 : 1;
  const int64_t per = kFinishThreads / lanes;
  const int64_t blocks = (static_cast<int64_t>(T) * ((D + 3) / 4) + per - 1) / per;
#define TGEMM_FINISH(OUT)                                                                                          \
  launch_chained(lanes == 8 ? finish_dh_kernel<OUT, 8> : finish_dh_kernel<OUT, 1>, blocks, kFinishThreads, stream, \
                 acc, ld_acc, split_stride, splits, T, D, rows, rule, static_cast<OUT*>(dH), lddh, wide)
  if (type == 0) return TGEMM_FINISH(__nv_bfloat16);
  if (type == 1) return TGEMM_FINISH(__half);
  return TGEMM_FINISH(float);
#undef TGEMM_FINISH
}

cudaError_t launch_split(const float* W, int64_t ldw, void* out, int64_t ld_out, int64_t plane, int rows, int cols,
                         bool vec, cudaStream_t stream) {
  return launch_chained(split_kernel, (rows + 3) / 4, 128, stream, W, ldw, static_cast<uint16_t*>(out), ld_out, plane,
                        rows, cols, vec ? 1 : 0);
}

}  // namespace tgemm
