// Routing of tokens to experts and its backward pass (include/tgemm_experts.h).
//
// One warp a row.  Lane l holds experts l, l + 32, ..., so a row is read in
// coalesced pieces, once, and stays in registers.  Experts are picked by as many
// rounds of "largest key, lowest index": keys as integers in the order of their
// numbers, so that a round is a local maximum and two warp reductions
// (redux.sync).  Bound by instructions (issue active 63 % of the time) and by the loads of a
// row, which only other warps cover: 16384 rows of 256 fp32 logits (2.7 us of bytes)
// take 8 us for one pick and 1 us for each more, 19 us for eight with sigmoid scores and a
// bias, 30 us with eight groups of which four are kept.
//
// Which keys.  Softmax and sigmoid grow with the logit, so without a bias (and
// without sums of keys) the logits themselves are compared.  With one, score +
// bias in fp32 may order two experts otherwise than the real numbers do, and picks
// are whole numbers that a reader of the weights takes for exact.  So where two
// neighbours among the picks and the first that is not one are closer than the keys'
// errors (margin_of), and differ in logit or bias, the picks and what follows them within
// such steps are ranked by fp64 keys, one a lane.  Softmax scores (their total is a sum over
// the row), groups that close at the border, and more than 32 candidates take the row's
// fp64 keys whole.  About one row in a hundred at 256 experts is ranked again.
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
// How far two fp32 keys, or sums of two, may be off one another's difference, relative to
// the largest score plus the largest bias.  A score's exponential is off by 2^-22 of it
// and by the rounding of its argument, 1.44 |x| 2^-24 (|x| s (1 - s) and |x| s / s_max stay
// below 0.4); sum, quotient, bias and the sum of two keys round once each; a difference of
// two sums has four keys: below 2^-19 together.  Softmax: its total, a chain of n + 5
// additions, is off by one factor for all.  The lowest bits of a key, of n keys a lane, hold
// which of them it is: n units of 2^-23 on either side.
constexpr float margin_of(bool sigmoid, int n) {
  return 0x1p-19f + 2 * n * 0x1p-23f + (sigmoid ? 0.0f : (n + 5) * 0x1p-23f);
}

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
// For keys (margin_of): e^x, and 1 / (1 + e^-x).
__device__ __forceinline__ float key_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}
__device__ __forceinline__ float key_sigmoid(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + key_exp(-x)));
  return y;
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

// A group's value as an ordered number, 0 where it is masked whole: from its two largest keys.
template <typename K>
__device__ __forceinline__ typename Order<K>::type group_value(K first, K second, bool nan, const RouteArgs& a) {
  using O = typename Order<K>::type;
  const K sum = a.top2 && second > -INFINITY ? first + second : first;
  return nan ? ordered(K(NAN)) : first > -INFINITY ? ordered(sum) : O(0);
}

// Groups of any size, their keys in shared memory: lane g gets group g's value.
template <typename K>
__device__ __forceinline__ typename Order<K>::type shared_group(const K* keys, const RouteArgs& a, int lane) {
  if (lane >= a.groups) return 0;
  const int size = a.E / a.groups;
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
  return group_value(first, second, nan, a);
}

// Groups of 32, ordered keys: register g of every lane.  (16384 rows of eight such groups: 29.5 us, and
// 32.5 by way of shared memory.)
template <int N>
__device__ __forceinline__ uint32_t register_group(const uint32_t (&order)[N], const RouteArgs& a, int lane) {
  uint32_t first = 0u, second = 0u;
#pragma unroll
  for (int g = 0; g < N; ++g) {
    if (g >= a.groups) break;
    const uint32_t top = __reduce_max_sync(kAll, order[g]);
    const uint32_t holders = __ballot_sync(kAll, order[g] == top);
    const uint32_t next = __reduce_max_sync(kAll, lane == __ffs(holders) - 1 ? 0u : order[g]);
    if (lane == g) {
      first = top;
      second = next;
    }
  }
  const float f = first ? number(first) : -INFINITY;
  return group_value(f, second ? number(second) : -INFINITY, f != f, a);
}

// Keeps the top_groups groups of the largest value (lane g holds group g's): `keep` is
// their bit mask.  False: the border is closer than `margin`.
template <typename O>
__device__ __forceinline__ bool pick_groups(O value, const RouteArgs& a, int lane, float margin, uint32_t& keep) {
  int rank = 0;  // groups before this one
  for (int g = 0; g < a.groups; ++g) {
    const O other = __shfl_sync(kAll, value, g);
    rank += other > value || (other == value && g < lane) ? 1 : 0;
  }
  const bool there = lane < a.groups && value != 0;
  keep = __ballot_sync(kAll, there && rank < a.top_groups);
  if constexpr (sizeof(O) == 4) {
    const uint32_t last = __ballot_sync(kAll, there && rank == a.top_groups - 1);
    const uint32_t out = __ballot_sync(kAll, there && rank == a.top_groups);
    if (!last || !out) return true;
    return !(number(__shfl_sync(kAll, value, __ffs(last) - 1)) - number(__shfl_sync(kAll, value, __ffs(out) - 1)) <= margin);
  }
  return true;
}

// The row's largest key and the lowest index that holds it, which is taken out.
template <int N>
__device__ __forceinline__ void next_pick(uint32_t (&order)[N], bool marked, int lane, uint32_t& top, int& at) {
  uint32_t most = order[0];
#pragma unroll
  for (int i = 1; i < N; ++i) most = max(most, order[i]);
  top = __reduce_max_sync(kAll, most);
  if (marked) {  // the lowest bits tell which of a lane's keys it is
    const int holder = __ffs(__ballot_sync(kAll, most == top)) - 1;
    at = static_cast<int>(N - 1 - (top & (N - 1))) * 32 + holder;
    const bool mine = lane == holder;
#pragma unroll
    for (int i = 0; i < N; ++i) order[i] = mine && order[i] == top ? 0u : order[i];
  } else {
    unsigned mine = UINT_MAX;
#pragma unroll
    for (int i = N - 1; i >= 0; --i) mine = order[i] == top ? i * 32 + lane : mine;
    at = static_cast<int>(__reduce_min_sync(kAll, mine));
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at == i * 32 + lane) order[i] = 0u;
  }
}
template <int N>
__device__ __forceinline__ void next_pick(uint64_t (&order)[N], bool, int lane, uint64_t& top, int& at) {
  top = order[0];
  at = lane;
#pragma unroll
  for (int i = 1; i < N; ++i)
    if (order[i] > top) {
      top = order[i];
      at = i * 32 + lane;
    }
  best_of(top, at);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at == i * 32 + lane) order[i] = 0;
}

// The value of x at expert e, which any lane may hold.
template <int N>
__device__ __forceinline__ float value_at(const float (&x)[N], int e) {
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float got = __shfl_sync(kAll, x[i], e & 31);
    if (e >> 5 == i) v = got;
  }
  return v;
}

// The row's keys as ordered numbers, 0 where masked or in a group that is not kept.  False:
// two groups at the border are closer than margin.  MARKED: the lowest bits of a key tell
// which of the lane's it is.
template <bool MARKED, typename K, int N, typename Key>
__device__ __forceinline__ bool order_keys(typename Order<K>::type (&order)[N], Key key_of, const RouteArgs& a, int lane,
                                           K* shared, float margin) {
  using O = typename Order<K>::type;
  K key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    key[i] = key_of(i);
    order[i] = key[i] == -INFINITY ? O(0) : MARKED ? (ordered(key[i]) & ~O(N - 1)) | O(N - 1 - i) : ordered(key[i]);
  }
  if (a.groups == 1) return true;
  const int size = a.E / a.groups;
  uint32_t keep;
  O value = 0;
  bool in_registers = false;
  if constexpr (sizeof(K) == 4) {
    in_registers = size == 32;
    if (in_registers) value = register_group(order, a, lane);
  }
  if (!in_registers) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 + lane < a.E) shared[i * 32 + lane] = key[i];
    __syncwarp();
    value = shared_group(shared, a, lane);
    __syncwarp();
  }
  const bool sure = pick_groups(value, a, lane, margin, keep);
#pragma unroll
  for (int i = 0; i < N; ++i)  // past the last group: 0 already
    if (!(keep >> (size == 32 ? i : (i * 32 + lane) / size & 31) & 1u)) order[i] = 0;
  return sure;
}

// The largest k keys: lane r gets the r-th's index, or -1.
template <typename O, int N>
__device__ __forceinline__ int pick(O (&order)[N], int k, int lane) {
  int mine = -1;
  for (int r = 0; r < k; ++r) {
    O top;
    int at;
    next_pick(order, false, lane, top, at);
    if (top == 0) break;
    if (lane == r) mine = at;
  }
  return mine;
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

// The picks of a row with fp64 keys.
template <typename In, int N>
__device__ __noinline__ int pick_exact(const RouteArgs& a, int row, int lane, double* shared) {
  float x[N], top = 0.0f;
  load_row<In>(x, a, row, lane);
  double total = 1.0;
  if (!a.sigmoid) softmax_of(x, top, total);
  uint64_t order[N];
  order_keys<false>(
      order,
      [&](int i) {
        const double v = x[i];
        if (x[i] == -INFINITY) return v;
        const double b = a.bias ? static_cast<double>(a.bias[i * 32 + lane]) : 0.0;
        return (a.sigmoid ? sigmoid_of(v) : exp(v - static_cast<double>(top)) / total) + b;
      },
      a, lane, shared, 0.0f);
  return pick(order, a.k, lane);
}

// The picks by fp32 keys of scores, ranked again where they are closer than the margin.
template <typename In, int N>
__device__ __forceinline__ int pick_scores(uint32_t (&order)[N], const RouteArgs& a, int row, int lane, float margin,
                                           bool sure, double* shared) {
  uint32_t key = 0u, next = 0u;  // lane r: the r-th largest; the one after all of them
  int mine = -1, next_at = 0, n = 0;
  for (; n < a.k; ++n) {
    next_pick(order, true, lane, next, next_at);
    if (next == 0) break;
    if (lane == n) {
      key = next;
      mine = next_at;
    }
  }
  if (n == a.k) next_pick(order, true, lane, next, next_at);  // the first that is not picked decides too
  // lane r: the key and the index behind the r-th
  const auto behind = [&](int& at) {
    const uint32_t k = __shfl_down_sync(kAll, key, 1);
    at = __shfl_down_sync(kAll, mine, 1);
    if (lane == n - 1) at = next_at;
    return lane == n - 1 ? next : k;
  };
  int after_at;
  const uint32_t after = behind(after_at);
  const bool close = lane < n && after != 0 && number(key) - number(after) <= margin;
  if (sure && !__any_sync(kAll, close)) return mine;
  const In* logits = static_cast<const In*>(a.logits) + row * a.ld;
  // equal in logit and bias: a tie whatever the arithmetic
  const bool differ = close && (to_float(logits[mine]) != to_float(logits[after_at]) ||
                                (a.bias && a.bias[mine] != a.bias[after_at]));
  if (sure && !__any_sync(kAll, differ)) return mine;
  if (sure && a.sigmoid) {
    // as many more as follow one another within the margin
    uint32_t last = __shfl_sync(kAll, key, n - 1);
    while (next != 0 && n < 32 && number(last) - number(next) <= margin) {
      if (lane == n) {
        key = next;
        mine = next_at;
      }
      last = next;
      ++n;
      next_pick(order, true, lane, next, next_at);
    }
    if (next == 0 || !(number(last) - number(next) <= margin)) {
      double exact = -INFINITY;
      if (lane < n) {
        const double v = to_float(logits[mine]);
        exact = sigmoid_of(v) + (a.bias ? static_cast<double>(a.bias[mine]) : 0.0);
      }
      const uint64_t own = lane < n ? ordered(exact) : 0ull;
      int rank = 0;
      for (int r = 0; r < n; ++r) {
        const uint64_t other = __shfl_sync(kAll, own, r);
        const int at = __shfl_sync(kAll, mine, r);
        rank += other > own || (other == own && at < mine) ? 1 : 0;
      }
      int picked = -1;  // lane r takes the candidate of rank r
      for (int r = 0; r < n; ++r) {
        const int at = __shfl_sync(kAll, mine, r), place = __shfl_sync(kAll, rank, r);
        if (place == lane && lane < a.k) picked = at;
      }
      return picked;
    }
  }
  return pick_exact<In, N>(a, row, lane, shared);
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
  uint32_t order[N];
  if (!scores) {
    order_keys<false>(order, [&](int i) { return x[i]; }, a, lane, reinterpret_cast<float*>(shared), 0.0f);
    mine = pick(order, a.k, lane);
  } else {
    float b[N], most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      b[i] = a.bias && i * 32 + lane < a.E ? __ldg(a.bias + i * 32 + lane) : 0.0f;
      most = fmaxf(most, fabsf(b[i]) < INFINITY ? fabsf(b[i]) : 0.0f);
    }
    if (a.bias) most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(most)));
    const float inv = 1.0f / total;
    // softmax's largest score is 1 / total
    const float margin = a.sigmoid ? margin_of(true, N) * (most + 1.0f) : margin_of(false, N) * (most + fminf(inv, 1.0f));
    const bool sure = order_keys<true>(
        order,
        [&](int i) {
          if (x[i] == -INFINITY) return x[i];
          return (a.sigmoid ? key_sigmoid(x[i]) : key_exp(x[i] - top) * inv) + b[i];
        },
        a, lane, reinterpret_cast<float*>(shared), margin);
    mine = pick_scores<In, N>(order, a, row, lane, margin, sure, shared);
  }
  // lane r: the r-th pick's weight
  const bool used = mine >= 0;
  const float at_mine = value_at(x, max(mine, 0));
  const float v = used ? at_mine : -INFINITY;
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
  float x[N];
  load_row<In>(x, a, row, lane);  // the picked logits too come from here: no load waits for another
  int mine = -1;
  float g = 0.0f;
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(row) * a.k + lane;
    const int64_t id = a.ids_in[at];
    const float grad = a.grad[at];
    if (id >= 0 && id < a.E) {
      mine = static_cast<int>(id);
      g = grad;
    }
  }
  const bool used = mine >= 0;
  const float at_mine = value_at(x, max(mine, 0));
  const float v = used ? at_mine : -INFINITY;
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
    float top, total;
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
