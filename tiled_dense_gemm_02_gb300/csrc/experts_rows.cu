// What runs between the experts' products: places sorted by expert, rows gathered
// in that order and joined back into tokens, fp16 gradients rounded (experts_internal.h).
//
// The sort counts: every warp takes neighbouring places, counts them by expert,
// and after the counts are summed up places them in their order, so the
// sorted order is that of the places, whatever the timing.  Up to kPlaceBlock
// places take one block and one launch (a decoding step's latency); more take three:
// counts per block, one block that sums them up and lists the tiles, placement.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "experts_gate.cuh"
#include "experts_internal.h"
#include "ptx.cuh"

namespace tgemm {
namespace {

constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kOwnExperts = kMaxExperts / kSortThreads;  // experts of a thread, neighbours
constexpr uint32_t kAll = 0xffffffffu;

// The expert of a place, -1 where unused, -2 where there is no such expert.
__device__ __forceinline__ int expert_of(const OrderArgs& a, int64_t place) {
  if (place >= a.places) return -1;
  const int64_t id = __ldcg(a.ids + place);
  return id < 0 ? -1 : id < a.E ? static_cast<int>(id) : -2;
}

// counts[warp][e] of the block's places (zeroed here), `each` neighbours a warp.
__device__ __forceinline__ void count_places(const OrderArgs& a, int64_t base, int each, int* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * a.E; i += kSortThreads) counts[i] = 0;
  __syncthreads();
#pragma unroll 2
  for (int r = 0; r < each; r += 32) {
    const int e = expert_of(a, base + warp * each + r + lane);
    if (e >= 0) atomicAdd(&counts[warp * a.E + e], 1);
  }
  __syncthreads();
}

__device__ __forceinline__ void sort_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSortThreads) : "memory"); }

// Sum over the first kSortThreads threads of the block before this one, and of all of
// them; they alone call it.
__device__ __forceinline__ int block_scan(int v, int* total, int* shared) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int below = __shfl_up_sync(kAll, sum, d);
    if (lane >= d) sum += below;
  }
  if (lane == 31) shared[warp] = sum;
  sort_barrier();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    before += w < warp ? shared[w] : 0;
    all += shared[w];
  }
  sort_barrier();
  *total = all;
  return before + sum - v;
}

// From the number of rows n[i] of experts kOwnExperts * threadIdx.x + i: first rows,
// filling and tiles.  One block.  Returns the thread's first row.
__device__ __forceinline__ int list_tiles(const OrderArgs& a, const int (&n)[kOwnExperts], int* shared) {
  int rows = 0, tiles = 0, padded[kOwnExperts], parts[kOwnExperts];
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    padded[i] = (n[i] + kRowPad - 1) / kRowPad * kRowPad;
    parts[i] = (padded[i] + kTokenTile - 1) / kTokenTile;
    rows += padded[i];
    tiles += parts[i];
  }
  int all_rows, all_tiles;
  const int start = block_scan(rows, &all_rows, shared);
  int row = start, tile = block_scan(tiles, &all_tiles, shared);
  if (threadIdx.x == 0) {
    a.rows.head[0] = all_tiles;
    a.rows.head[1] = all_rows;
    a.rows.first[a.E] = all_rows;
  }
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    const int e = kOwnExperts * threadIdx.x + i;
    if (e >= a.E) break;
    a.rows.first[e] = row;
    a.rows.count[e] = n[i];
    if (n[i]) {
      // the smallest even parts; never fewer of them than `parts`, whose number the scan
      // counted: with r = padded / 32 >= 8 (parts - 1) + 1, parts of ceil(r / parts) leave
      // some for the last while (parts - 1)^2 < r, and from 9 parts on are of 8
      const int even = (padded[i] / parts[i] + kRowPad - 1) / kRowPad * kRowPad;
      const int each = even * parts[i] < padded[i] ? even + kRowPad : even;
      for (int at = 0; at < padded[i]; at += each) {
        const int size = min(each, padded[i] - at);
        a.rows.tiles[tile++] = make_int4(e, row + at, size, max(0, min(size, n[i] - at)));
      }
    }
    row += padded[i];
  }
  return start;
}

// Places the block's rows; next[warp][e] is where the warp's next row of expert e goes.
__device__ __forceinline__ void place_rows(const OrderArgs& a, int64_t base, int each, int* next) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ahead = expert_of(a, base + warp * each + lane);
#pragma unroll 1
  for (int r = 0; r < each; r += 32) {
    const int64_t place = base + warp * each + r + lane;
    const int e = ahead;
    if (r + 32 < each) ahead = expert_of(a, place + 32);
    const uint32_t same = __match_any_sync(kAll, e);
    if (e >= 0) {
      const int row = next[warp * a.E + e] + __popc(same & ((1u << lane) - 1u));
      a.rows.token[row] = static_cast<int>(place / a.k);
      a.rows.place[row] = static_cast<int>(place);
      a.rows.row[place] = row;
    } else if (place < a.places) {
      a.rows.row[place] = e;
    }
    __syncwarp();
    if (e >= 0 && (same >> lane) == 1u) next[warp * a.E + e] += __popc(same);  // the last of them
    __syncwarp();
  }
}

// The filling behind an expert's n rows.
__device__ __forceinline__ void fill_rows(const OrderArgs& a, int row, int n, int token) {
  const int end = row + (n + kRowPad - 1) / kRowPad * kRowPad;
  for (int r = row + n; r < end; ++r) {
    a.rows.token[r] = token;
    a.rows.place[r] = -1;
  }
}

__global__ void __launch_bounds__(kSortThreads) order_kernel(const __grid_constant__ OrderArgs a, int each) {
  extern __shared__ int counts[];  // kSortWarps x E
  __shared__ int scan[kSortWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  count_places(a, 0, each, counts);
  int n[kOwnExperts];
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    const int e = kOwnExperts * threadIdx.x + i;
    n[i] = 0;
    if (e < a.E)
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) n[i] += counts[w * a.E + e];
  }
  int row = list_tiles(a, n, scan);
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    const int e = kOwnExperts * threadIdx.x + i;
    if (e < a.E) {
      int at = row;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = counts[w * a.E + e];
        counts[w * a.E + e] = at;
        at += c;
      }
      row += (n[i] + kRowPad - 1) / kRowPad * kRowPad;
    }
  }
  __syncthreads();
  place_rows(a, 0, each, counts);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    const int first = a.rows.first[e], rows = a.rows.count[e];
    if (rows) fill_rows(a, first, rows, a.rows.token[first]);
  }
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ OrderArgs a, int each) {
  extern __shared__ int counts[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  count_places(a, static_cast<int64_t>(blockIdx.x) * each * kSortWarps, each, counts);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += counts[w * a.E + e];
    a.rows.partial[static_cast<int64_t>(blockIdx.x) * a.E + e] = n;
  }
}

// partial[block][e]: the block's rows of e -> the rows of e in the blocks before it.  The
// blocks are summed in `segments` parts side by side, then once more with what lies before
// each part.
constexpr int kTilesThreads = 1024;
__global__ void __launch_bounds__(kTilesThreads) tiles_kernel(const __grid_constant__ OrderArgs a, int blocks, int segments) {
  __shared__ int totals[kTilesThreads];  // [segment][e]
  __shared__ int scan[kSortWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int segment = threadIdx.x / a.E, e = threadIdx.x - segment * a.E;
  const int each = (blocks + segments - 1) / segments;
  const int begin = min(blocks, segment * each), end = segment < segments ? min(blocks, begin + each) : begin;
  int* p = a.rows.partial + e;
  int sum = 0;
#pragma unroll 16
  for (int b = begin; b < end; ++b) sum += __ldcg(p + static_cast<int64_t>(b) * a.E);
  totals[threadIdx.x] = sum;
  __syncthreads();
  if (segment < segments) {
    int before = 0;
    for (int i = 0; i < segment; ++i) before += totals[i * a.E + e];
    int b = begin;
    for (; b + 8 <= end; b += 8) {
      int v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldcg(p + static_cast<int64_t>(b + i) * a.E);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[static_cast<int64_t>(b + i) * a.E] = before;
        before += v[i];
      }
    }
    for (; b < end; ++b) {
      const int v = __ldcg(p + static_cast<int64_t>(b) * a.E);
      p[static_cast<int64_t>(b) * a.E] = before;
      before += v;
    }
  }
  if (threadIdx.x >= kSortThreads) return;
  int n[kOwnExperts];
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    const int own = kOwnExperts * threadIdx.x + i;
    n[i] = 0;
    if (own < a.E)
      for (int k = 0; k < segments; ++k) n[i] += totals[k * a.E + own];
  }
  int row = list_tiles(a, n, scan);
#pragma unroll
  for (int i = 0; i < kOwnExperts; ++i) {
    fill_rows(a, row, n[i], 0);  // calls of so many places gather no rows by their tokens
    row += (n[i] + kRowPad - 1) / kRowPad * kRowPad;
  }
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const __grid_constant__ OrderArgs a, int each) {
  extern __shared__ int counts[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * each * kSortWarps;
  count_places(a, base, each, counts);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int row = __ldcg(a.rows.first + e) + __ldcg(a.rows.partial + static_cast<int64_t>(blockIdx.x) * a.E + e);
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = counts[w * a.E + e];
      counts[w * a.E + e] = row;
      row += c;
    }
  }
  __syncthreads();
  place_rows(a, base, each, counts);
}

// ----------------------------------------------------- weights off the 16-byte grid
// Copies of the weights in an aligned pitch, which the products' bulk-tensor copies need, of
// the experts that have rows.  A warp a row, 16 bytes a lane: an aligned word, shifted together
// with the next lane's; what a row's last word takes from behind the row is never used.  Bound by
// bytes: 50 experts of 477 x 2079 (600 MB read and written) 110 us, 10 of 1001 x 500 (60 MB) 19;
// two rows a warp 124, four 140 (64 registers).
constexpr int kCopyThreads = 256;

// The bytes from `off` (a multiple of 2, below 16) on of two neighbouring words.
__device__ __forceinline__ uint4 across(const uint4& a, const uint4& b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t shift = 8u * (off & 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], shift);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The elements of an aligned word that lie in [begin, end), bytes from p.
__device__ __forceinline__ uint4 word_inside(const uint8_t* p, int begin, int end) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i >= begin && 2 * i < end) w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p) + i)) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kCopyThreads, 8) copy_weights_kernel(const int* count, int E,
                                                                    const __grid_constant__ WeightCopy in,
                                                                    const __grid_constant__ WeightCopy out) {
  __shared__ int used[kMaxExperts];
  __shared__ int in_warp[kCopyThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int listed = 0;
  for (int e0 = 0; e0 < E; e0 += kCopyThreads) {
    const int e = e0 + threadIdx.x;
    const bool some = e < E && __ldcg(count + e) > 0;
    const uint32_t mask = __ballot_sync(kAll, some);
    if (lane == 0) in_warp[warp] = __popc(mask);
    __syncthreads();
    int at = listed + __popc(mask & ((1u << lane) - 1u));
    for (int w = 0; w < kCopyThreads / 32; ++w) {
      if (w < warp) at += in_warp[w];
      listed += in_warp[w];
    }
    if (some) used[at] = e;
    __syncthreads();
  }
  const uint32_t each = in.rows + out.rows;  // rows of an expert
  const int64_t total = int64_t(listed) * each, warps = int64_t(gridDim.x) * (kCopyThreads / 32);
  for (int64_t r = int64_t(blockIdx.x) * (kCopyThreads / 32) + warp; r < total; r += warps) {
    const uint32_t slot = static_cast<uint32_t>(r) / each;
    uint32_t row = static_cast<uint32_t>(r) - slot * each;
    const bool second = row >= static_cast<uint32_t>(in.rows);
    const WeightCopy& m = second ? out : in;
    if (second) row -= in.rows;
    const int64_t at = int64_t(used[slot]) * m.rows + row, last = int64_t(E) * m.rows - 1;
    const uint8_t* src = static_cast<const uint8_t*>(m.from) + at * m.ld_from * 2;
    uint8_t* dst = static_cast<uint8_t*>(m.to) + at * m.ld_to * 2;
    const int off = static_cast<int>(reinterpret_cast<uint64_t>(src) & 15u), bytes = 2 * m.cols;
    src -= off;  // the matrix lies in [low, high) from here
    const int low = static_cast<int>(max(int64_t(0), off - at * m.ld_from * 2));
    const int high = static_cast<int>(min(off + ((last - at) * m.ld_from + m.cols) * 2, int64_t(INT_MAX)));
    for (int d0 = 0; d0 < bytes; d0 += 31 * 16) {  // the last lane has the second word of the one before
      const int d = d0 + lane * 16;
      uint4 v = make_uint4(0u, 0u, 0u, 0u), next;
      if (d < bytes + off) {
        if (d >= low && d + 16 <= high)
          v = __ldg(reinterpret_cast<const uint4*>(src + d));
        else
          v = word_inside(src + d, low - d, high - d);
      }
      next.x = __shfl_down_sync(kAll, v.x, 1);
      next.y = __shfl_down_sync(kAll, v.y, 1);
      next.z = __shfl_down_sync(kAll, v.z, 1);
      next.w = __shfl_down_sync(kAll, v.w, 1);
      if (lane < 31 && d < bytes) *reinterpret_cast<uint4*>(dst + d) = across(v, next, off);
    }
  }
}

// ----------------------------------------------------------------- gather
// A warp a row, up to eight 16-byte loads a lane in flight, the next row's token loaded
// ahead.  Bound by bytes: a token's row is read k times, the later times from L2, and
// every sorted row is written once (8192 tokens of 2048, 8 places each: a block a row 61 us).
constexpr int kGatherThreads = 256;

template <int G>  // granule of x's rows in bytes
__device__ __forceinline__ uint4 load_word(const uint16_t* src, int d, int D) {
  if (d >= D) return make_uint4(0u, 0u, 0u, 0u);
  if (G == 16 && d + 8 <= D) return __ldg(reinterpret_cast<const uint4*>(src + d));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (G >= 4 && d + 8 <= D) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src + d) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d + i < D) w[i / 2] |= static_cast<uint32_t>(__ldg(src + d + i)) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int G>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const int* head, const int* token, const int* place,
                                                                const uint16_t* x, int64_t ldx, int D, uint16_t* out,
                                                                int64_t ld_out, unsigned int* zeros, int words) {
  constexpr int kFlight = G == 16 ? 8 : 2;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (zeros && blockIdx.x == 0)
    for (int i = threadIdx.x; i < words; i += kGatherThreads) zeros[i] = 0u;
  const int rows = __ldcg(head + 1), lane = threadIdx.x & 31;
  const int warp = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kGatherThreads / 32);
  const auto token_of = [&](int r) { return r >= rows || __ldcg(place + r) < 0 ? -1 : __ldcg(token + r); };
  int next = token_of(warp);
  for (int r = warp; r < rows; r += warps) {
    const int t = next;
    next = token_of(r + warps);
    const uint16_t* src = x + (t < 0 ? 0 : t * ldx);
    uint16_t* dst = out + r * ld_out;
    const int end = t < 0 ? 0 : D;  // the filling: zeros
    for (int d0 = lane * 8; d0 < D; d0 += kFlight * 256) {
      uint4 v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) v[i] = load_word<G>(src, d0 + i * 256, end);
#pragma unroll
      for (int i = 0; i < kFlight; ++i)  // D is filled up to the pitch, a multiple of 8
        if (d0 + i * 256 < D) *reinterpret_cast<uint4*>(dst + d0 + i * 256) = v[i];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pair_of(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// ------------------------------------------------------- fp16 gradients rounded
// dg, du and w h in halves, after their largest ones are known: a scale from the gradient alone
// (or none) leaves infinities where W_out or u are large and nothing where weights are small, since
// dg = w v u silu'(g) with v a sum over D.  The largest of an expert at 2^14 keeps all bits of
// what is above 2^-28 of it.  A block has 32 rows (of one expert) and kRoundFeatures features, a warp
// four rows and a lane two neighbouring features.  Bound by bytes: v, g and u are read, 12
// bytes a value, and 6 written (32768 rows of 1408: 831 MB in 136 us, 0.9 of copy).
constexpr int kRoundThreads = 256, kRoundFeatures = 512;

__global__ void __launch_bounds__(kRoundThreads) round_kernel(const __grid_constant__ RoundArgs a) {
  __shared__ int owner;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int row0 = blockIdx.x * kRowPad;
  if (row0 >= __ldcg(a.rows.head + 1)) return;
  for (int e = threadIdx.x; e < a.E; e += kRoundThreads)
    if (__ldcg(a.rows.first + e) <= row0 && row0 < __ldcg(a.rows.first + e + 1)) owner = e;
  __syncthreads();
  const float scale = expert_scale(__ldcg(a.largest + 2 * owner)), scale_h = expert_scale(__ldcg(a.largest + 2 * owner + 1));
  const int lane = threadIdx.x & 31;
  const int64_t row = row0 + (threadIdx.x >> 5) * 4;
  float w[4];
  bool used[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int place = __ldcg(a.rows.place + row + r);
    used[r] = place >= 0;
    w[r] = used[r] ? __ldg(a.weights + place) : 0.0f;
  }
  const float4* g4 = reinterpret_cast<const float4*>(a.gu) + row / 4 * 2 * a.ldg;
  const float4* v4 = reinterpret_cast<const float4*>(a.v) + row / 4 * a.ldg;
  uint16_t* dg_row = static_cast<uint16_t*>(a.dgu) + row * a.ld_dgu;
  uint16_t* h_row = static_cast<uint16_t*>(a.h) + row * a.ldh;
  const bool odd = (a.F & 1) != 0;
  const int end = min(a.F, (static_cast<int>(blockIdx.y) + 1) * kRoundFeatures);
#pragma unroll 2
  for (int f = blockIdx.y * kRoundFeatures + 2 * lane; f < end; f += 64) {
    float dg[2][4], du[2][4], wh[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // the pitch, a multiple of 4, holds f + 1
      const float4 g = __ldcs(g4 + f + i), u = __ldcs(g4 + a.ldg + f + i), v = __ldcs(v4 + f + i);
      const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const GatedGradient d = gated_gradient(gs[r], us[r], w[r] * vs[r]);
        dg[i][r] = used[r] ? scale * d.dg : 0.0f;
        du[i][r] = used[r] ? scale * d.du : 0.0f;
        wh[i][r] = used[r] ? scale_h * (w[r] * d.h) : 0.0f;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t p[3] = {pair_of<false>(dg[0][r], dg[1][r]), pair_of<false>(du[0][r], du[1][r]), pair_of<false>(wh[0][r], wh[1][r])};
      uint16_t* to[3] = {dg_row + r * a.ld_dgu + f, dg_row + r * a.ld_dgu + a.F + f, h_row + r * a.ldh + f};
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (!odd) {
          *reinterpret_cast<uint32_t*>(to[i]) = p[i];
        } else {
          to[i][0] = static_cast<uint16_t>(p[i]);
          if (f + 1 < a.F) to[i][1] = static_cast<uint16_t>(p[i] >> 16);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- join
// One thread: eight columns of a token.  Bound by y's bytes, read once.
constexpr int kJoinThreads = 128, kJoinColumns = 8;

struct JoinKernelArgs {
  const int* row;
  const float* weights;
  int k, D;
  const void* y;
  const uint8_t* y_exponent;
  int64_t ldy;
  void* out;
  int64_t ld_out;
  int vec;  // out's rows are 16-byte aligned and D a multiple of 8
  const float* dots;
  int parts;
  float* d_weights;
};

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ JoinKernelArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t t = blockIdx.x;
  const int* rows = a.row + t * a.k;
  if (a.d_weights && blockIdx.y == 0) {  // a warp a place
    const int lane = threadIdx.x & 31;
    for (int j = threadIdx.x >> 5; j < a.k; j += kJoinThreads / 32) {
      const int row = __ldcg(rows + j);
      float sum = 0.0f;
      if (row >= 0)
        for (int i = lane; i < a.parts; i += 32) sum += __ldcg(a.dots + static_cast<int64_t>(row) * a.parts + i);
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
      if (lane == 0) a.d_weights[t * a.k + j] = row == -2 ? NAN : sum;
    }
  }
  const int d = (blockIdx.y * kJoinThreads + threadIdx.x) * kJoinColumns;
  if (!a.out || d >= a.D) return;
  float sum[kJoinColumns];
#pragma unroll
  for (int i = 0; i < kJoinColumns; ++i) sum[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int row = __ldcg(rows + j);
    if (row >= 0) {
      float w = a.weights ? __ldg(a.weights + t * a.k + j) : 1.0f;
      float y[kJoinColumns];
      if constexpr (BF16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.y) + row * a.ldy + d));
        const uint32_t p[4] = {v.x, v.y, v.z, v.w};
        const uint32_t e = __ldcg(a.y_exponent + (row / 16 * (a.ldy / 32) + d / 32) * 16 + row % 16);
        if (e != 0u) {
          w *= __uint_as_float((e - 14u) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
            y[2 * i] = f.x;
            y[2 * i + 1] = f.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(p[i] << 16);
            y[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
          }
        }
      } else {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.y) + row * a.ldy + d);
        const float4 lo = __ldcs(src), hi = __ldcs(src + 1);
        y[0] = lo.x;
        y[1] = lo.y;
        y[2] = lo.z;
        y[3] = lo.w;
        y[4] = hi.x;
        y[5] = hi.y;
        y[6] = hi.z;
        y[7] = hi.w;
      }
#pragma unroll
      for (int i = 0; i < kJoinColumns; ++i) sum[i] = fmaf(w, y[i], sum[i]);
    } else if (row == -2) {
#pragma unroll
      for (int i = 0; i < kJoinColumns; ++i) sum[i] = NAN;
    }
  }
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair_of<BF16>(sum[2 * i], sum[2 * i + 1]);
  uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.ld_out + d;
  if (a.vec) {
    *reinterpret_cast<uint4*>(out) = make_uint4(p[0], p[1], p[2], p[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kJoinColumns; ++i)
      if (d + i < a.D) out[i] = static_cast<uint16_t>(p[i / 2] >> (16 * (i & 1)));
  }
}

template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                        const Args&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// Blocks of the sort: of 512 places, which many blocks make short, while one block can
// sum up their counts in some microseconds, else of 2048.
int order_blocks(int64_t places) {
  if (places <= kPlaceBlock) return 1;
  const int64_t each = places <= 128 * 1024 ? 512 : kPlaceBlock;
  return static_cast<int>((places + each - 1) / each);
}

cudaError_t launch_order(const OrderArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(int) * kSortWarps * a.E;  // at most 32 KB
  const int blocks = order_blocks(a.places);
  if (blocks == 1) {
    const int each = static_cast<int>((a.places + 32 * kSortWarps - 1) / (32 * kSortWarps) * 32);
    return launch_next(order_kernel, dim3(1), kSortThreads, smem, stream, a, each);
  }
  const int each = (a.places <= 128 * 1024 ? 512 : kPlaceBlock) / kSortWarps;
  cudaError_t e = launch_next(count_kernel, dim3(blocks), kSortThreads, smem, stream, a, each);
  if (e == cudaSuccess) e = launch_next(tiles_kernel, dim3(1), kTilesThreads, 0, stream, a, blocks, std::min(16, kTilesThreads / a.E));
  if (e == cudaSuccess) e = launch_next(place_kernel, dim3(blocks), kSortThreads, smem, stream, a, each);
  return e;
}

cudaError_t launch_copy_weights(const int* count, int E, int64_t used, const WeightCopy& in, const WeightCopy& out, int sms,
                                cudaStream_t stream) {
  constexpr int kRows = kCopyThreads / 32;
  const int64_t rows = used * (int64_t(in.rows) + out.rows);
  const int blocks = static_cast<int>(std::min<int64_t>((rows + kRows - 1) / kRows, 32 * std::max(1, sms)));
  return launch_next(copy_weights_kernel, dim3(blocks), kCopyThreads, 0, stream, count, E, in, out);
}

cudaError_t launch_gather_rows(const ExpertRows& rows, int64_t most_rows, const void* x, int64_t ldx, int granule, int D,
                               void* out, int64_t ld_out, unsigned int* zeros, int words, int sms, cudaStream_t stream) {
  constexpr int kWarps = kGatherThreads / 32;
  const auto kernel = granule == 16 ? gather_kernel<16> : granule >= 4 ? gather_kernel<4> : gather_kernel<2>;
  const int blocks = static_cast<int>(std::min<int64_t>((most_rows + kWarps - 1) / kWarps, 4 * std::max(1, sms)));
  return launch_next(kernel, dim3(blocks), kGatherThreads, 0, stream,
                     static_cast<const int*>(rows.head), static_cast<const int*>(rows.token),
                     static_cast<const int*>(rows.place), static_cast<const uint16_t*>(x), ldx, D,
                     static_cast<uint16_t*>(out), ld_out, zeros, words);
}

cudaError_t launch_round_gradients(const RoundArgs& a, int64_t most_rows, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((most_rows + kRowPad - 1) / kRowPad), (a.F + kRoundFeatures - 1) / kRoundFeatures, 1);
  return launch_next(round_kernel, grid, kRoundThreads, 0, stream, a);
}

cudaError_t launch_join(const JoinArgs& j, cudaStream_t stream) {
  JoinKernelArgs a = {};
  a.row = j.rows->row;
  a.weights = j.weights;
  a.k = j.k;
  a.D = j.D;
  a.y = j.y;
  a.y_exponent = j.y_exponent;
  a.ldy = j.ldy;
  a.out = j.out;
  a.ld_out = j.ld_out;
  a.vec = j.out && j.D % 8 == 0 && j.ld_out % 8 == 0 && reinterpret_cast<uint64_t>(j.out) % 16 == 0;
  a.dots = j.dots;
  a.parts = j.parts;
  a.d_weights = j.d_weights;
  constexpr int kWide = kJoinThreads * kJoinColumns;
  const int across = j.out ? (j.D + kWide - 1) / kWide : 1;
  const dim3 grid(static_cast<unsigned>(j.T), across, 1);
  return j.type == 0 ? launch_next(join_kernel<true>, grid, kJoinThreads, 0, stream, a)
                     : launch_next(join_kernel<false>, grid, kJoinThreads, 0, stream, a);
}

}  // namespace tgemm
