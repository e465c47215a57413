// Routing of tokens to experts and its backward pass (include/tgemm_experts.h).
//
// One warp a row.  Lane l holds experts l, l + 32, ..., so a row is read in
// coalesced pieces, once, and stays in registers.  Experts are picked by as many
// rounds of "largest key, lowest index": keys as integers in the order of their
// numbers, so that a round is a local maximum and two warp reductions
// (redux.sync).  Rows are bytes-bound from some thousand rows on; below, the call is
// one launch.
//
// Which keys.  Softmax and sigmoid grow with the logit, so without a bias (and
// without sums of keys) the logits themselves are compared.  With one, score +
// bias in fp32 may order two experts otherwise than the real numbers do, and picks
// are whole numbers that a reader of the weights takes for exact: a row in which
// two neighbouring picks, or two groups at the border, are closer than the keys'
// errors (kMargin) is picked again with fp64 keys, unless the two are equal in logit
// and bias and tie for certain.  About one row in a hundred at 256 experts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "../../include/tgemm_experts.h"
#include "loss_internal.h"
#include "ptx.cuh"

namespace tgemm {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;
// Errors of fp32 keys: a score s is off by at most 2^-20.6 s (the exponential's two
// last bits, the rounding of x - max, which is below 2^-24 |x - max| and weighs s
// |x - max| < 1/e at most, the sum's and the division's), and key and sum of two
// keys round once more; a difference of two sums has four such keys.
constexpr float kMargin = 0x1p-18f;

struct RouteArgs {
  int T, E, k;
  const void* logits;
  int64_t ld;
  const float* bias;
  int sigmoid, renormalize, groups, top_groups, top2;
  float scale;
  int64_t* ids;
  float* weights;
  // backward
  const int64_t* ids_in;
  const float* grad;
  void* d_logits;
  int64_t ld_out;
};

template <typename T>
__device__ __forceinline__ float to_float(T v) {
  return static_cast<float>(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  return T(v);
}

// Numbers as unsigned integers in the same order; NaN is the largest.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 is 0
  return x != x ? 0xffffffffu : b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return x != x ? ~0ull : b ^ (b >> 63 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float number(uint32_t o) {
  return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o);
}

// The warp's largest key and the lowest index that holds it.
__device__ __forceinline__ void best_of(uint32_t& key, int& at) {
  const uint32_t top = __reduce_max_sync(kAll, key);
  at = static_cast<int>(__reduce_min_sync(kAll, key == top ? static_cast<unsigned>(at) : UINT_MAX));
  key = top;
}
__device__ __forceinline__ void best_of(uint64_t& key, int& at) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t other = __shfl_xor_sync(kAll, key, d);
    const int where = __shfl_xor_sync(kAll, at, d);
    if (other > key || (other == key && where < at)) {
      key = other;
      at = where;
    }
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <typename K>
__device__ __forceinline__ K warp_sum(K v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

template <typename K>
__device__ __forceinline__ K sigmoid_of(K x) {
  return K(1) / (K(1) + exp(-x));
}

template <typename K>
struct Order;
template <>
struct Order<float> {
  using type = uint32_t;
};
template <>
struct Order<double> {
  using type = uint64_t;
};

// Keeps the top_groups groups of the largest value: `keep` is their bit mask.  False:
// the border is closer than `margin`.
template <typename K>
__device__ __forceinline__ bool pick_groups(const K* keys, const RouteArgs& a, int lane, float margin, uint32_t& keep) {
  using O = typename Order<K>::type;
  const int size = a.E / a.groups;
  O value = 0;
  if (lane < a.groups) {
    K first = -INFINITY, second = -INFINITY;
    bool nan = false;
    const K* mine = keys + lane * size;
    int i = lane % size;  // lanes start apart, so that they meet different banks
    for (int n = 0; n < size; ++n) {
      const K v = mine[i];
      nan |= v != v;
      if (v > first) {
        second = first;
        first = v;
      } else if (v > second) {
        second = v;
      }
      if (++i == size) i = 0;
    }
    const K sum = a.top2 && second > -INFINITY ? first + second : first;
    // a group that is masked whole has no part: 0, below every number's order
    value = nan ? ordered(K(NAN)) : first > -INFINITY ? ordered(sum) : O(0);
  }
  keep = 0u;
  O last = 0;
  bool sure = true;
  for (int r = 0; r <= a.top_groups; ++r) {
    O top = value;
    int at = lane;
    best_of(top, at);
    if (top == 0) break;
    if (r == a.top_groups) {
      if constexpr (sizeof(K) == 4) sure = !(number(last) - number(top) <= margin);
      break;
    }
    last = top;
    keep |= 1u << at;
    if (lane == at) value = 0;
  }
  return sure;
}

// The row's picks: lane r gets the r-th's index, or -1.  False (fp32): not certain.
template <typename K, int N, typename Key>
__device__ __forceinline__ bool pick(Key key_of, const RouteArgs& a, int lane, K* shared, bool certain, float margin,
                                     int& mine, const float (&x)[N]) {
  using O = typename Order<K>::type;
  O order[N];
  bool sure = true;
  uint32_t keep = kAll;
  {
    K key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = key_of(i);
    if (a.groups > 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * 32 + lane < a.E) shared[i * 32 + lane] = key[i];
      __syncwarp();
      sure = pick_groups(shared, a, lane, margin, keep);
      if (certain) sure = true;
      __syncwarp();
    }
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * 32 + lane;
      const bool in = e < a.E && (a.groups == 1 || (keep >> (e / size) & 1u));
      // masked: 0, below every number's order (and -inf's)
      order[i] = in && !(key[i] == -INFINITY) ? ordered(key[i]) : O(0);
    }
  }
  mine = -1;
  O before = 0;
  int before_at = 0;
  const int rounds = certain ? a.k : a.k + 1;  // the first that is not picked decides too
  for (int r = 0; r < rounds; ++r) {
    O top = order[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (order[i] > top) {
        top = order[i];
        at = i * 32 + lane;
      }
    best_of(top, at);
    if (top == 0) break;
    if constexpr (sizeof(K) == 4) {
      if (!certain && r > 0 && number(before) - number(top) <= margin) {
        // equal in logit and bias: a tie whatever the arithmetic
        float xa = 0.0f, xb = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (before_at / 32 == i) xa = x[i];
          if (at / 32 == i) xb = x[i];
        }
        xa = __shfl_sync(kAll, xa, before_at & 31);
        xb = __shfl_sync(kAll, xb, at & 31);
        if (xa != xb || (a.bias && a.bias[before_at] != a.bias[at])) sure = false;
      }
    }
    before = top;
    before_at = at;
    if (lane == r && r < a.k) mine = at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at == i * 32 + lane) order[i] = 0;
  }
  return sure;
}

template <typename In, int N>
__device__ __forceinline__ void load_row(float (&x)[N], const RouteArgs& a, int row, int lane) {
  const In* src = static_cast<const In*>(a.logits) + row * a.ld;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = i * 32 + lane < a.E ? to_float(src[i * 32 + lane]) : -INFINITY;
}

// Maximum and sum of exponentials of a row's logits (0 where all are masked).
template <typename K, int N>
__device__ __forceinline__ void softmax_of(const float (&x)[N], float& top, K& total) {
  top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  total = K(0);
  if (top == -INFINITY) {
    // all masked, or NaN beside masked ones
#pragma unroll
    for (int i = 0; i < N; ++i) total += x[i] != x[i] ? K(NAN) : K(0);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) total += exp(K(x[i]) - K(top));
  }
  total = warp_sum(total);
}

// The score of a picked expert relative to the others': where `shift` is the
// largest picked logit if that is below 0, e^-shift sigmoid(x) without underflow.
__device__ __forceinline__ float shifted_sigmoid(float x, float shift) {
  return x <= 0.0f ? expf(x - shift) / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
}

template <typename In, int N>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ double shared_keys[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kWarps + warp;
  if (row >= a.T) return;
  double* shared = shared_keys + (a.groups > 1 ? warp * a.E : 0);
  float x[N];
  load_row<In>(x, a, row, lane);
  float top = 0.0f, total = 0.0f;
  const bool scores = a.bias || (a.groups > 1 && a.top2);  // keys are scores, not logits
  if (!a.sigmoid && (scores || !a.renormalize)) softmax_of(x, top, total);
  int mine;
  if (!scores) {
    pick<float, N>([&](int i) { return x[i]; }, a, lane, reinterpret_cast<float*>(shared), true, 0.0f, mine, x);
  } else {
    float b[N], most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      b[i] = a.bias && i * 32 + lane < a.E ? a.bias[i * 32 + lane] : 0.0f;
      most = fmaxf(most, fabsf(b[i]) < INFINITY ? fabsf(b[i]) : 0.0f);
    }
    most = warp_max(most);
    const float inv = 1.0f / total;
    const float margin = kMargin * (most + (a.sigmoid ? 1.0f : fminf(inv, 1.0f)));  // softmax's largest is 1 / total
    const bool sure = pick<float, N>(
        [&](int i) {
          if (x[i] == -INFINITY) return x[i];
          return (a.sigmoid ? sigmoid_of(x[i]) : expf(x[i] - top) * inv) + b[i];
        },
        a, lane, reinterpret_cast<float*>(shared), false, margin, mine, x);
    if (!sure) {
      float top64;
      double total64 = 1.0;
      if (!a.sigmoid) softmax_of(x, top64, total64);
      pick<double, N>(
          [&](int i) {
            if (x[i] == -INFINITY) return -static_cast<double>(INFINITY);
            const double v = x[i];
            return (a.sigmoid ? sigmoid_of(v) : exp(v - static_cast<double>(top)) / total64) + static_cast<double>(b[i]);
          },
          a, lane, shared, true, 0.0f, mine, x);
    }
  }
  // lane r: the r-th pick's weight
  const bool used = mine >= 0;
  const float v = used ? to_float(static_cast<const In*>(a.logits)[row * a.ld + mine]) : -INFINITY;
  float w = 0.0f;
  if (a.renormalize) {
    const float most = warp_max(v);  // NaN is passed over: it comes back in the sum
    if (used) w = a.sigmoid ? shifted_sigmoid(v, fminf(most, 0.0f)) : expf(v - most);
    const float sum = warp_sum(w);
    if (used) w = w / sum;
  } else if (used) {
    w = a.sigmoid ? sigmoid_of(v) : expf(v - top) / total;
  }
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(row) * a.k + lane;
    a.ids[at] = mine;
    a.weights[at] = used ? a.scale * w : 0.0f;
  }
}

// dx of sum_j grad_j weight_j.  With s the scores, p the picked ones' shares:
//   softmax, renormalized   dx_i = scale p_i (g_i - sum_j g_j p_j), picked ones only
//   softmax                 dx_e = scale s_e ([picked] g_e - sum_j g_j s_j)
//   sigmoid, renormalized   dx_i = scale p_i (1 - s_i) (g_i - sum_j g_j p_j)
//   sigmoid                 dx_i = scale s_i (1 - s_i) g_i
template <typename In, int N>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const __grid_constant__ RouteArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= a.T) return;
  const In* src = static_cast<const In*>(a.logits) + row * a.ld;
  int mine = -1;
  float g = 0.0f;
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(row) * a.k + lane;
    const int64_t id = a.ids_in[at];
    if (id >= 0 && id < a.E) {
      mine = static_cast<int>(id);
      g = a.grad[at];
    }
  }
  const bool used = mine >= 0;
  const float v = used ? to_float(src[mine]) : -INFINITY;
  float d[N];
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = 0.0f;
  float own = 0.0f;  // this lane's pick's part
  if (a.renormalize) {
    const float most = warp_max(v);
    float p = 0.0f;
    if (used) p = a.sigmoid ? shifted_sigmoid(v, fminf(most, 0.0f)) : expf(v - most);
    const float sum = warp_sum(p);
    if (used) p = p / sum;
    const float mean = warp_sum(used ? g * p : 0.0f);
    own = p * (g - mean);
    if (a.sigmoid) own *= 1.0f / (1.0f + expf(v));
  } else if (a.sigmoid) {
    own = g * sigmoid_of(v) * (1.0f / (1.0f + expf(v)));
  } else {
    float x[N], top, total;
    load_row<In>(x, a, row, lane);
    softmax_of(x, top, total);
    if (used) own = g * (expf(v - top) / total);
    const float mean = warp_sum(used ? own : 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = x[i] == -INFINITY ? 0.0f : -mean * (expf(x[i] - top) / total);
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kAll, mine, j);
    const float part = __shfl_sync(kAll, own, j);
    if (e >= 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e == i * 32 + lane) d[i] += part;
    }
  }
  In* out = static_cast<In*>(a.d_logits) + row * a.ld_out;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * 32 + lane < a.E) out[i * 32 + lane] = from_float<In>(a.scale * d[i]);
}

template <typename In, int N>
cudaError_t launch_rows(const RouteArgs& a, bool backward, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + kWarps - 1) / kWarps, 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = !backward && a.groups > 1 ? kWarps * a.E * sizeof(double) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, backward ? route_backward_kernel<In, N> : route_kernel<In, N>, a);
}

template <typename In>
cudaError_t launch_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  const int per = (a.E + 31) / 32;
  if (per <= 1) return launch_rows<In, 1>(a, backward, stream);
  if (per <= 2) return launch_rows<In, 2>(a, backward, stream);
  if (per <= 4) return launch_rows<In, 4>(a, backward, stream);
  if (per <= 8) return launch_rows<In, 8>(a, backward, stream);
  if (per <= 16) return launch_rows<In, 16>(a, backward, stream);
  return launch_rows<In, 32>(a, backward, stream);
}

struct RouteSpan {
  const void* p;
  uint64_t bytes;
  int align;
  bool out;
};

int run_route(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ld, int dtype, const float* bias,
              const tgemm_route_options* o, const int64_t* ids_in, const float* grad, int64_t* ids, float* weights,
              void* d_logits, int64_t ld_out, bool backward, cudaStream_t stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || ld < E || (backward && ld_out < E)) return TGEMM_ERR_INVALID_VALUE;
  RouteArgs a = {};
  a.groups = a.top_groups = 1;
  a.scale = 1.0f;
  if (o) {
    if ((o->scoring != TGEMM_ROUTE_SOFTMAX && o->scoring != TGEMM_ROUTE_SIGMOID) || (o->renormalize & ~1) ||
        !std::isfinite(o->scale) || o->scale < 0.0f || o->groups < 0 || o->top_groups < 0 ||
        (o->group_score != TGEMM_ROUTE_GROUP_MAX && o->group_score != TGEMM_ROUTE_GROUP_TOP2) || o->reserved[0] ||
        o->reserved[1])
      return TGEMM_ERR_INVALID_VALUE;
    if (o->groups > TGEMM_ROUTE_MAX_GROUPS) return TGEMM_ERR_TOO_LARGE;
    a.sigmoid = o->scoring == TGEMM_ROUTE_SIGMOID;
    a.renormalize = o->renormalize;
    if (o->scale != 0.0f) a.scale = o->scale;
    if (o->groups) a.groups = o->groups;
    if (o->top_groups) a.top_groups = o->top_groups;
    a.top2 = o->group_score == TGEMM_ROUTE_GROUP_TOP2;
  }
  if (a.top_groups > a.groups || E % a.groups || k > E / a.groups * a.top_groups) return TGEMM_ERR_INVALID_VALUE;
  if (dtype != TGEMM_F32 && dtype != TGEMM_F16 && dtype != TGEMM_BF16) return TGEMM_ERR_UNSUPPORTED_DTYPE;
  if (E > TGEMM_ROUTE_MAX_EXPERTS || k > TGEMM_ROUTE_MAX_K || T >= (int64_t(1) << 31) - 256 ||
      ld >= int64_t(1) << 31 || ld_out >= int64_t(1) << 31)
    return TGEMM_ERR_TOO_LARGE;
  if (T == 0) return TGEMM_OK;
  if (!logits || (backward ? (!ids_in || !grad || !d_logits) : (!ids || !weights))) return TGEMM_ERR_INVALID_VALUE;
  const int es = dtype == TGEMM_F32 ? 4 : 2;
  const uint64_t places = static_cast<uint64_t>(T) * k;
  const uint64_t row_bytes = static_cast<uint64_t>(E) * es;
  RouteSpan spans[4];
  spans[0] = RouteSpan{logits, static_cast<uint64_t>(T - 1) * ld * es + row_bytes, es, false};
  if (backward) {
    spans[1] = RouteSpan{d_logits, static_cast<uint64_t>(T - 1) * ld_out * es + row_bytes, es, true};
    spans[2] = RouteSpan{ids_in, 8 * places, 8, false};
    spans[3] = RouteSpan{grad, 4 * places, 4, false};
  } else {
    spans[1] = RouteSpan{bias, 4ull * E, 4, false};
    spans[2] = RouteSpan{ids, 8 * places, 8, true};
    spans[3] = RouteSpan{weights, 4 * places, 4, true};
  }
  for (const RouteSpan& s : spans)
    if (reinterpret_cast<uint64_t>(s.p) % s.align) return TGEMM_ERR_MISALIGNED;
  for (const RouteSpan& s : spans)
    for (const RouteSpan& t : spans) {
      if (&s == &t || !s.out || !s.p || !t.p) continue;
      const uint64_t x = reinterpret_cast<uint64_t>(s.p), y = reinterpret_cast<uint64_t>(t.p);
      if (host_ranges_overlap(x, x + s.bytes, y, y + t.bytes)) return TGEMM_ERR_ALIAS;
    }
  int sms = 0, pairs = 0;
  unsigned int* status = nullptr;
  const int st = host_device(&sms, &pairs, &status);
  if (st != TGEMM_OK) return st;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.ids_in = ids_in;
  a.grad = grad;
  a.d_logits = d_logits;
  a.ld_out = ld_out;
  const cudaError_t e = dtype == TGEMM_F32   ? launch_route<float>(a, backward, stream)
                        : dtype == TGEMM_F16 ? launch_route<__half>(a, backward, stream)
                                             : launch_route<__nv_bfloat16>(a, backward, stream);
  return e == cudaSuccess ? TGEMM_OK : host_cuda_fail(e, "route launch");
}

}  // namespace
}  // namespace tgemm

extern "C" {

int tgemm_route_forward(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ld, int dtype, const float* bias,
                        const tgemm_route_options* opts, int64_t* ids, float* weights, void* stream) {
  return tgemm::run_route(T, E, k, logits, ld, dtype, bias, opts, nullptr, nullptr, ids, weights, nullptr, E, false,
                          static_cast<cudaStream_t>(stream));
}

int tgemm_route_backward(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ld, int dtype,
                         const int64_t* ids, const float* grad, const tgemm_route_options* opts, void* d_logits,
                         int64_t ld_out, void* stream) {
  return tgemm::run_route(T, E, k, logits, ld, dtype, nullptr, opts, ids, grad, nullptr, nullptr, d_logits, ld_out,
                          true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
