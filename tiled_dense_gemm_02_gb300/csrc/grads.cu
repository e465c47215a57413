// Norm over many gradients and their clipping (include/tgemm_grads.h).
//
// Bound by bytes: the norm reads every gradient once, clipping reads it again and
// writes it.  The second pass needs the whole norm, so what does not fit L2 is
// read twice; it walks the list backwards, and so finds in L2 what the first pass
// read last.
//
// The tensors are cut into chunks of 32 KB (kChunk) of their 16-byte words, dealt
// to the blocks in turn; a launch carries its list of up to kList tensors in its
// parameters, so the call keeps no table in device memory and can be captured.
// Each thread has eight 16-byte loads in flight: whole chunks load without a condition.
//
// Squares: a thread adds the at most 32 squares of half of its share of a chunk in fp32
// (an error of a few 2^-24, random over threads) and the shares in fp64, one
// addition per 64 bytes, since fp64 additions per element would take three times
// the bytes' time.  A share whose fp32 sum leaves [2^-90, 2^100) is summed again in fp64, from registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "../../include/tgemm_grads.h"
#include "loss_internal.h"
#include "ptx.cuh"

namespace tgemm {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 8;                          // 16-byte words of a thread's share of a chunk
constexpr int kChunk = kThreads * kVectors;          // words of a chunk
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = kBlocksPerSm * 152;       // of one launch
constexpr int64_t kMaxElements = int64_t(1) << 40;     // chunks stay ints
constexpr int kShort = 40, kList = 1000;             // tensors of a launch; short lists have less to copy

template <int MOST>
struct List {
  int n;
  int chunks;                  // of all tensors
  const void* in[MOST];
  void* out[MOST];
  int64_t count[MOST];         // elements << 2 | type (0 bf16, 1 f16, 2 f32)
  int first[MOST + 1];         // first chunk of each tensor
};
static_assert(sizeof(List<kList>) <= 32000, "kernel parameters");

__device__ __forceinline__ float2 halves(uint32_t w, int type) {
  if (type == 0) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A tensor as 16-byte words of memory: element `skip` of word 0 is its first.
struct View {
  const uint8_t* base;  // 16-byte aligned
  int skip, type, shift;  // shift: log2 of the elements of a word
  int64_t count, words;
  template <int MOST>
  __device__ __forceinline__ View(const List<MOST>& l, int t) {
    const uint64_t p = reinterpret_cast<uint64_t>(l.in[t]);
    type = static_cast<int>(l.count[t] & 3);
    count = l.count[t] >> 2;
    shift = type == 2 ? 2 : 3;
    base = reinterpret_cast<const uint8_t*>(p & ~uint64_t(15));
    skip = static_cast<int>(p & 15) >> (4 - shift);
    words = (skip + count + (1 << shift) - 1) >> shift;
  }
  // a chunk's words of this thread, from w0 on
  __device__ __forceinline__ void load_chunk(int64_t w0, uint4 (&x)[kVectors]) const {
    const int64_t c0 = w0 - threadIdx.x;
    if (((c0 << shift) >= skip) && ((c0 + kChunk) << shift) - skip <= count) {  // all words whole
#pragma unroll
      for (int j = 0; j < kVectors; ++j) x[j] = __ldcg(reinterpret_cast<const uint4*>(base) + w0 + j * kThreads);
    } else {
#pragma unroll
      for (int j = 0; j < kVectors; ++j) x[j] = load(w0 + j * kThreads);
    }
  }
  // word w; elements outside the tensor are 0 and not read
  __device__ __forceinline__ uint4 load(int64_t w) const {
    if (w >= words) return make_uint4(0u, 0u, 0u, 0u);
    const int64_t e0 = (w << shift) - skip;  // tensor element of the word's first
    if (e0 >= 0 && e0 + (1 << shift) <= count) return __ldcg(reinterpret_cast<const uint4*>(base) + w);
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (type == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i >= 0 && e0 + i < count) v[i] = __ldcg(reinterpret_cast<const uint32_t*>(base) + w * 4 + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i >= 0 && e0 + i < count)
          v[i / 2] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const uint16_t*>(base) + w * 8 + i)) << (16 * (i & 1));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

__device__ __forceinline__ float square_sum(const uint4& v, int type, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == 2) {
      const float x = __uint_as_float(w[i]);
      s = fmaf(x, x, s);
    } else {
      const float2 x = halves(w[i], type);
      s = fmaf(x.x, x.x, s);
      s = fmaf(x.y, x.y, s);
    }
  }
  return s;
}

__device__ __noinline__ double square_sum_wide(uint4 a, uint4 b, uint4 c, uint4 d, int type) {
  const uint32_t w[16] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (type == 2) {
      const double x = __uint_as_float(w[i]);
      s = fma(x, x, s);
    } else {
      const float2 x = halves(w[i], type);
      s = fma(static_cast<double>(x.x), static_cast<double>(x.x), s);
      s = fma(static_cast<double>(x.y), static_cast<double>(x.y), s);
    }
  }
  return s;
}

// Sum over the block, in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double s, double* shared) {
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = s;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) total += shared[i];
  return total;
}

template <int MOST>
__device__ __forceinline__ int tensor_of(const List<MOST>& l, int chunk) {
  int lo = 0, hi = l.n;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int MOST>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) square_kernel(const __grid_constant__ List<MOST> l, double* partial) {
  __shared__ double shared[kThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  double sum = 0.0;
  for (int c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const int t = tensor_of(l, c);
    const View v(l, t);
    const int64_t w0 = static_cast<int64_t>(c - l.first[t]) * kChunk + threadIdx.x;
    uint4 x[kVectors];
    v.load_chunk(w0, x);
#pragma unroll
    for (int part = 0; part < kVectors; part += 4) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s = square_sum(x[part + j], v.type, s);
      if (s >= 0x1p-90f && s < 0x1p100f) {
        sum += s;
      } else {
        uint32_t any = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) any |= x[part + j].x | x[part + j].y | x[part + j].z | x[part + j].w;
        if (any) sum += square_sum_wide(x[part], x[part + 1], x[part + 2], x[part + 3], v.type);
      }
    }
  }
  sum = block_sum(sum, shared);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from all launches' partial sums, the same in every block.
__device__ __forceinline__ double norm_of(const double* partial, int n, double* shared) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += __ldcg(partial + i);
  return sqrt(block_sum(s, shared));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* partial, int n, float* norm) {
  __shared__ double shared[kThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const double total = norm_of(partial, n, shared);
  if (threadIdx.x == 0) *norm = static_cast<float>(total);
}

__device__ __forceinline__ uint4 scaled(const uint4& v, int type, float f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == 2) {
      w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
    } else {
      const float2 x = halves(w[i], type);
      if (type == 0) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * f, x.y * f);
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
      } else {
        const __half2 y = __floats2half2_rn(x.x * f, x.y * f);
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// `first`: this launch writes the norm.
template <int MOST>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) scale_kernel(const __grid_constant__ List<MOST> l, const double* partial,
                                                            int n, float max_norm, float* norm, int first) {
  __shared__ double shared[kThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const double total = norm_of(partial, n, shared);
  if (first && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  // by the norm that the caller sees: past fp32's largest number it is infinite
  const bool clips = total > static_cast<double>(max_norm) && static_cast<float>(total) < INFINITY;
  const float f = clips ? static_cast<float>(static_cast<double>(max_norm) / total) : 1.0f;
  const int last = l.chunks - 1;
  for (int c = last - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int t = tensor_of(l, c);
    if (!clips && l.out[t] == l.in[t]) continue;
    const View v(l, t);
    const int64_t w0 = static_cast<int64_t>(c - l.first[t]) * kChunk + threadIdx.x;
    uint4 x[kVectors];
    v.load_chunk(w0, x);
    uint8_t* out = static_cast<uint8_t*>(l.out[t]);
    const int es = 16 >> v.shift, per = 1 << v.shift;
    // outputs at another offset modulo 16 are stored element by element: 600 M bf16 values 1650 us, and 578 together
    const bool together = ((reinterpret_cast<uint64_t>(out) ^ reinterpret_cast<uint64_t>(l.in[t])) & 15) == 0;
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      const int64_t w = w0 + j * kThreads;
      if (w >= v.words) continue;
      const uint4 y = clips ? scaled(x[j], v.type, f) : x[j];
      const int64_t e0 = (w << v.shift) - v.skip;
      if (together && e0 >= 0 && e0 + per <= v.count) {
        __stcs(reinterpret_cast<uint4*>(out + e0 * es), y);  // first to leave L2: the gradients still to be read stay
      } else if (v.type == 2) {
        const uint32_t p[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e0 + i >= 0 && e0 + i < v.count) reinterpret_cast<uint32_t*>(out)[e0 + i] = p[i];
      } else {
        const uint32_t p[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e0 + i >= 0 && e0 + i < v.count)
            reinterpret_cast<uint16_t*>(out)[e0 + i] = static_cast<uint16_t>(p[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

// ------------------------------------------------------------------- host

struct GradCall {
  int64_t n = 0;
  const void* const* grads = nullptr;
  const int64_t* counts = nullptr;
  const int* dtypes = nullptr;
  void* const* outputs = nullptr;
  bool clip = false;
  float max_norm = 0.0f;
  float* norm = nullptr;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  cudaStream_t stream = nullptr;
};

int64_t workspace_bytes(int64_t n) {
  const int64_t launches = std::max<int64_t>(1, (n + kList - 1) / kList);
  return launches * kMaxBlocks * static_cast<int64_t>(sizeof(double));
}

int type_of(int dtype) { return dtype == TGEMM_BF16 ? 0 : dtype == TGEMM_F16 ? 1 : dtype == TGEMM_F32 ? 2 : -1; }

struct Range {
  uint64_t lo, hi;
  int64_t tensor;  // -1: the call's own
  bool written;
};

int check_call(const GradCall& c) {
  if (c.n < 0 || !c.norm || (c.n > 0 && (!c.grads || !c.counts || !c.dtypes))) return TGEMM_ERR_INVALID_VALUE;
  if (c.clip && !(c.max_norm >= 0.0f)) return TGEMM_ERR_INVALID_VALUE;
  if (c.n > TGEMM_GRAD_MAX_TENSORS) return TGEMM_ERR_TOO_LARGE;
  int64_t total = 0;
  for (int64_t i = 0; i < c.n; ++i) {
    if (c.counts[i] < 0) return TGEMM_ERR_INVALID_VALUE;
    if (type_of(c.dtypes[i]) < 0) return TGEMM_ERR_UNSUPPORTED_DTYPE;
    if (c.counts[i] >= kMaxElements || (total += c.counts[i]) >= kMaxElements) return TGEMM_ERR_TOO_LARGE;
    if (c.counts[i] == 0) continue;
    if (!c.grads[i] || (c.outputs && !c.outputs[i])) return TGEMM_ERR_INVALID_VALUE;
  }
  if (!c.workspace || reinterpret_cast<uint64_t>(c.workspace) % 256 ||
      c.workspace_bytes < static_cast<size_t>(workspace_bytes(c.n)))
    return TGEMM_ERR_INVALID_VALUE;
  if (reinterpret_cast<uint64_t>(c.norm) % 4) return TGEMM_ERR_MISALIGNED;
  std::vector<Range> ranges;
  ranges.reserve(2 * c.n + 2);
  const auto add = [&ranges](const void* p, uint64_t bytes, int64_t tensor, bool written) {
    const uint64_t lo = reinterpret_cast<uint64_t>(p);
    ranges.push_back({lo, lo + bytes, tensor, written});
  };
  add(c.norm, 4, -1, true);
  add(c.workspace, c.workspace_bytes, -1, true);
  for (int64_t i = 0; i < c.n; ++i) {
    if (c.counts[i] == 0) continue;
    const uint64_t es = c.dtypes[i] == TGEMM_F32 ? 4 : 2, bytes = c.counts[i] * es;
    const void* out = c.outputs ? c.outputs[i] : c.grads[i];
    if (reinterpret_cast<uint64_t>(c.grads[i]) % es || reinterpret_cast<uint64_t>(out) % es) return TGEMM_ERR_MISALIGNED;
    if (!c.clip || out != c.grads[i]) add(c.grads[i], bytes, i, false);
    if (c.clip) add(out, bytes, i, true);
  }
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  // nothing overlaps anything where one of the two is written; readers may overlap one another
  uint64_t any_end = 0, written_end = 0;
  for (const Range& r : ranges) {
    if (r.lo < written_end || (r.written && r.lo < any_end)) return TGEMM_ERR_ALIAS;
    any_end = std::max(any_end, r.hi);
    if (r.written) written_end = std::max(written_end, r.hi);
  }
  return TGEMM_OK;
}

template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), int blocks, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tensors [begin, end) that have elements.
template <int MOST>
void fill(List<MOST>& l, const GradCall& c, int64_t begin, int64_t end) {
  l.n = 0;
  int64_t chunks = 0;
  for (int64_t i = begin; i < end; ++i) {
    if (c.counts[i] == 0) continue;
    const int type = type_of(c.dtypes[i]), shift = type == 2 ? 2 : 3;
    const int64_t skip = static_cast<int64_t>(reinterpret_cast<uint64_t>(c.grads[i]) & 15) >> (4 - shift);
    const int64_t words = (skip + c.counts[i] + (1 << shift) - 1) >> shift;
    l.in[l.n] = c.grads[i];
    l.out[l.n] = c.outputs ? c.outputs[i] : const_cast<void*>(c.grads[i]);
    l.count[l.n] = c.counts[i] << 2 | type;
    l.first[l.n] = static_cast<int>(chunks);
    chunks += (words + kChunk - 1) / kChunk;
    ++l.n;
  }
  l.first[l.n] = static_cast<int>(chunks);
  l.chunks = static_cast<int>(chunks);
}

template <int MOST>
int run_lists(const GradCall& c, int sms) {
  double* partial = static_cast<double*>(c.workspace);
  const int most = std::min(kMaxBlocks, kBlocksPerSm * std::max(1, sms));
  const auto list = std::unique_ptr<List<MOST>>(new (std::nothrow) List<MOST>);
  if (!list) return host_cuda_fail(cudaErrorMemoryAllocation, "gradient list");
  int parts = 0;
  for (int64_t at = 0; at < c.n; at += MOST) {
    fill(*list, c, at, std::min<int64_t>(c.n, at + MOST));
    if (list->chunks == 0) continue;
    const int blocks = std::min(list->chunks, most);
    const cudaError_t e = launch_next(square_kernel<MOST>, blocks, c.stream, *list, partial + parts);
    if (e != cudaSuccess) return host_cuda_fail(e, "square launch");
    parts += blocks;
  }
  if (!c.clip || parts == 0) {
    const cudaError_t e = launch_next(norm_kernel, 1, c.stream, partial, parts, c.norm);
    return e == cudaSuccess ? TGEMM_OK : host_cuda_fail(e, "norm launch");
  }
  // the last list first: L2 holds the most of it
  bool first = true;
  for (int64_t at = (c.n - 1) / MOST * MOST; at >= 0; at -= MOST) {
    if (c.n > MOST || first) fill(*list, c, at, std::min<int64_t>(c.n, at + MOST));
    if (list->chunks == 0) continue;
    const int blocks = std::min(list->chunks, most);
    const cudaError_t e = launch_next(scale_kernel<MOST>, blocks, c.stream, *list, partial, parts, c.max_norm, c.norm,
                                      first ? 1 : 0);
    if (e != cudaSuccess) return host_cuda_fail(e, "scale launch");
    first = false;
  }
  return TGEMM_OK;
}

int run_grads(const GradCall& c) {
  int st = TGEMM_OK;
  try {
    st = check_call(c);
  } catch (const std::bad_alloc&) {
    return host_cuda_fail(cudaErrorMemoryAllocation, "gradient ranges");
  }
  if (st != TGEMM_OK) return st;
  int sms = 0, pairs = 0;
  unsigned int* status = nullptr;
  st = host_device(&sms, &pairs, &status);
  if (st != TGEMM_OK) return st;
  return c.n <= kShort ? run_lists<kShort>(c, sms) : run_lists<kList>(c, sms);
}

}  // namespace
}  // namespace tgemm

extern "C" {

int tgemm_grad_workspace_size(int64_t n, size_t* bytes) {
  if (n < 0 || !bytes) return TGEMM_ERR_INVALID_VALUE;
  if (n > TGEMM_GRAD_MAX_TENSORS) return TGEMM_ERR_TOO_LARGE;
  *bytes = static_cast<size_t>(tgemm::workspace_bytes(n));
  return TGEMM_OK;
}

int tgemm_grad_norm(int64_t n, const void* const* grads, const int64_t* counts, const int* dtypes, float* norm,
                    void* workspace, size_t workspace_bytes, void* stream) {
  tgemm::GradCall c;
  c.n = n;
  c.grads = grads;
  c.counts = counts;
  c.dtypes = dtypes;
  c.norm = norm;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_grads(c);
}

int tgemm_grad_clip(int64_t n, const void* const* grads, const int64_t* counts, const int* dtypes,
                    void* const* outputs, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                    void* stream) {
  tgemm::GradCall c;
  c.n = n;
  c.grads = grads;
  c.counts = counts;
  c.dtypes = dtypes;
  c.outputs = outputs;
  c.clip = true;
  c.max_norm = max_norm;
  c.norm = norm;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_grads(c);
}

}  // extern "C"
