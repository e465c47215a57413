// Tensor-core products of the vocabulary-head losses, on CTA pairs: one 256 x
// 256 tile per pair, tcgen05.mma.cta_group::2 (M = 256), fp32 accumulators in
// tensor memory, two of them, so a tile's epilogue runs under the next tile's
// MMAs.  Four products share the pipeline and differ in operand layout and
// epilogue:
//
//   STATS  y = k2 H W^T       row max, sum of 2^(y - max), sum q z of the tile
//   DZ     the same product   dz = c_p 2^(y - lse2) - c_q q, 16-bit, stored
//   DH     dz . W             fp32 sums, stored or added (bulk-tensor reduce)
//   DW     dz^T . H           times a factor, rounded once, stored
//
// with k2 = scale log2(e), so that one fused multiply-add and one 2^x serve
// each logit.  H and W are read K-major (their rows are the k axis) by STATS
// and DZ; W as the N-major B of DH; dz as the M-major A and H as the N-major B
// of DW: no operand is ever transposed in memory.
//
// The adder of tcgen05.mma truncates: every step (16 products added to the fp32
// sum) moves the sum towards 0 by up to its last bit, so a long k axis would lose
// D / 16 of them.  Sums leave tensor memory every `chunk` stages and are added
// in registers with rounding to nearest, by the thread that owns the element,
// under the next chunk's MMAs.  The last sum goes back to tensor memory, where
// the epilogues read it.  (One factor for the mean loss, in its place, moved
// sums that are exact, and covered a quarter of the loss of one sign's.)
//
// PLANES = 3: fp32 operands come as three bf16 planes (loss_rows.cu), and a
// stage of the k axis is then six stages, one per pair of planes, the small
// terms first: the last sixth alone adds to a sum of full size, so the adder's
// truncation is that of a 16-bit product.
// PLANES = 2: 16-bit operands, dz as two planes (its rounding and what that
// leaves), so that few rows' gradients do not depend on how the one or two
// entries that matter happen to round.
//
// Roles (both CTAs unless noted):
//   warp 0      bulk-tensor producer of this CTA's 128 rows of A and 128
//               columns of B; completion on the leader CTA's full barrier
//   warp 1      tensor-memory allocation; MMA issue by one thread of the leader
//   warps 2..   epilogue of this CTA's 128 rows, one row per thread: eight warps
//               with half of the columns each, or four for STATS with one chunk
//               of middle length (loss_api.cu)
//
// The number of gathered rows is known on the device only (rows that do not
// count are not gathered), so every role derives the tile list from it.  Every
// wait is bounded (tc_common.cuh).
#pragma once

#include <atomic>
#include <climits>

#include "loss_internal.h"
#include "tc_common.cuh"

namespace tgemm {
namespace {

constexpr int kSub = kTileM * kTileK * 2;        // 16 KB: one CTA's share of A or B in one stage
constexpr int kStage = 2 * kSub;
// PARTS: epilogue warps per quarter of the rows; each of the gradients' has 4 KB to stage stores.
constexpr int head_threads(int parts) { return 32 * (2 + 4 * parts); }
constexpr int head_epi_bytes(int mode, int parts) { return mode == HEAD_STATS ? 0 : 4 * parts * 4096; }
constexpr int head_stages(int mode, int parts) {
  return (kSmemLimit - 1024 - head_epi_bytes(mode, parts) - kBarrierBytes) / kStage;
}
constexpr int head_smem(int mode, int parts) {
  return 1024 + head_stages(mode, parts) * kStage + head_epi_bytes(mode, parts) + kBarrierBytes;
}
constexpr bool a_m_major(int mode) { return mode == HEAD_DW; }
constexpr bool b_n_major(int mode) { return mode == HEAD_DH || mode == HEAD_DW; }

// Pairs of planes in the order they are summed: fp32 (2,0) (0,2) (1,1) (1,0)
// (0,1) (0,0); two planes of dz (1,0) (0,0).
template <int MODE, int PLANES>
struct Terms {
  static constexpr bool logits = MODE == HEAD_STATS || MODE == HEAD_DZ;  // operands H and W
  static constexpr int count = PLANES == 3 ? 6 : PLANES == 2 && !logits ? 2 : 1;
  static __device__ __forceinline__ int a(int term) {
    return count == 6 ? (0x001102 >> (4 * term)) & 0xF : count - 1 - term;
  }
  static __device__ __forceinline__ int b(int term) { return count == 6 ? (0x010120 >> (4 * term)) & 0xF : 0; }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds a shared-memory box to the fp32 tensor at (x, y, z).
__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                  uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

constexpr int kGroupM = 8;  // block-rows walked together; a power of two, so that a full group's quotient is a shift

// The tile list of a launch, derived from the gathered row count.
struct Tiles {
  int m, n, units, k_blocks;
  float per_inv, group_inv;  // 1 / (m n), 1 / (kGroupM n)
};

template <int MODE>
__device__ __forceinline__ Tiles head_tiles(const HeadArgs& a, int rows) {
  Tiles t;
  t.m = ((MODE == HEAD_DW ? a.cols : rows) + kHeadTile - 1) / kHeadTile;
  t.n = ((MODE == HEAD_DH || MODE == HEAD_DW ? a.D : a.cols) + kHeadTile - 1) / kHeadTile;
  t.k_blocks = MODE == HEAD_DW ? (rows + kTileK - 1) / kTileK : a.k_blocks;
  t.units = t.m * t.n * (MODE == HEAD_DH ? a.splits : 1);
  t.per_inv = 1.0f / static_cast<float>(t.m * t.n);
  t.group_inv = 1.0f / static_cast<float>(kGroupM * t.n);
  return t;
}

// i / d and i % d with a given reciprocal of d.  The product in fp32 is off by
// less than one quotient while i stays below 2^23; beyond (T V of 2^39), the
// plain division.  The division of every tile by every role was a third of a
// short tile's time.
__device__ __forceinline__ void divide(int i, int d, float inv, int& q, int& r) {
  if (i < (1 << 23)) {
    q = __float2int_rz(__int2float_rn(i) * inv);
    r = i - q * d;
    if (r < 0) {
      --q;
      r += d;
    } else if (r >= d) {
      ++q;
      r -= d;
    }
  } else {
    q = i / d;
    r = i - q * d;
  }
}

struct HeadUnit {
  int mb, nb, split, lo, hi;
};

// Unit -> tile and k-stage range: groups of kGroupM block-rows are walked
// column by column (as the plain product does), split after split.
template <int MODE>
__device__ __forceinline__ HeadUnit head_unit(const HeadArgs& a, const Tiles& t, int u) {
  HeadUnit w;
  int i = u;
  w.split = 0;
  if (MODE == HEAD_DH) divide(u, t.m * t.n, t.per_inv, w.split, i);
  int g, r;
  divide(i, kGroupM * t.n, t.group_inv, g, r);
  const int first = g * kGroupM;
  const int gsz = t.m - first;
  if (gsz >= kGroupM) {
    w.mb = first + (r & (kGroupM - 1));
    w.nb = r / kGroupM;
  } else {
    w.nb = r / gsz;
    w.mb = first + r - w.nb * gsz;
  }
  w.lo = MODE == HEAD_DH ? min(w.split * a.k_per_split, t.k_blocks) : 0;
  w.hi = MODE == HEAD_DH ? min(w.lo + a.k_per_split, t.k_blocks) : t.k_blocks;
  return w;
}

// A row's targets, walked in ascending order as its columns go by.
struct Walk {
  const int* ids;
  const float* q;
  int pos, K, next;
  float one;  // mass of a single target (K = 0)
  // `y`: the row's target (cross entropy), loaded ahead
  __device__ __forceinline__ void start(const HeadArgs& a, int row, int n, int first, int64_t y) {
    K = pos = 0;
    next = INT_MAX;
    ids = nullptr;
    q = nullptr;
    one = a.mass;
    if (row >= n) return;
    if (a.target) {
      if (y >= first && y < a.V) next = static_cast<int>(y);
      return;
    }
    const int t = a.source ? a.source[row] : row;
    K = a.K;
    ids = a.ids + static_cast<int64_t>(t) * K;
    q = a.q + static_cast<int64_t>(t) * K;
    int len = K;
    while (len > 0) {  // first place whose id is not below `first`
      const int half = len >> 1;
      if (ids[pos + half] < first) {
        pos += half + 1;
        len -= half + 1;
      } else {
        len = half;
      }
    }
    next = pos < K ? ids[pos] : INT_MAX;
  }
  __device__ __forceinline__ float mass() const { return K ? q[pos] : one; }
  __device__ __forceinline__ void step() {
    ++pos;
    next = pos < K ? ids[pos] : INT_MAX;
  }
};

// Running statistics of a row: maximum of the logits so far, sum of 2^(k2 (z -
// maximum)), sum q z, and sum z (where eps needs it).
struct RowStats {
  float m = -INFINITY, s = 0.0f, dot = 0.0f, zs = 0.0f;

  // 32 more columns from entry `base` on, `limit` of them inside the piece
  __device__ __forceinline__ void add(const uint32_t (&raw)[32], int base, int limit, Walk& walk, const HeadArgs& a) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
    if (limit < 32) {  // columns past the piece are no entries
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = i < limit ? v[i] : -INFINITY;
    }
    float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
    const float m_new = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    const float ref = m_new == -INFINITY ? 0.0f : m_new;  // nothing but -inf so far: every term is 0
    const float2 k2 = make_float2(a.k2, a.k2), off = make_float2(-ref * a.k2, -ref * a.k2);
    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), k2, off);
      part[i & 1] = __fadd2_rn(part[i & 1], make_float2(exp2_fast(x.x), exp2_fast(x.y)));
    }
    const float2 both = __fadd2_rn(part[0], part[1]);
    s = fmaf(s, exp2_fast((m - ref) * a.k2), both.x + both.y);
    m = m_new;
    if (a.flat != 0.0f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) zs += i < limit ? v[i] : 0.0f;
    }
    while (__any_sync(0xffffffffu, walk.next < base + 32)) {
      if (walk.next < base + 32) {
        const int t = walk.next - base;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) z = i == t ? v[i] : z;
        dot = fmaf(walk.mass(), z, dot);
        walk.step();
      }
    }
  }
};

// The sums of this thread's row and 128 columns: a first chunk's, one more
// chunk's added, and the whole ones back in tensor memory.
__device__ __forceinline__ void load_sums(uint32_t tcol, uint32_t (&sum)[8][16]) {
#pragma unroll
  for (int b = 0; b < 8; ++b) ptx::tmem_ld_32x32b_x16(tcol + b * 16, sum[b]);
  ptx::tmem_wait_ld();
}
__device__ __forceinline__ void add_sums(uint32_t tcol, uint32_t (&sum)[8][16]) {
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    uint32_t raw[16];
    ptx::tmem_ld_32x32b_x16(tcol + b * 16, raw);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      sum[b][i] = __float_as_uint(__uint_as_float(sum[b][i]) + __uint_as_float(raw[i]));
  }
}
__device__ __forceinline__ void store_sums(uint32_t tcol, const uint32_t (&sum)[8][16]) {
#pragma unroll
  for (int b = 0; b < 8; ++b) ptx::tmem_st_32x32b_x16(tcol + b * 16, sum[b]);
  ptx::tmem_wait_st();
}

// Statistics of this thread's row over its part of the tile's columns.  Of two
// parts the second leaves them in the accumulator's columns, which it has read,
// and the first joins and writes both: `handed` is completed by the one and
// awaited by the other.  False: the wait ran out.
template <int PARTS>
__device__ __forceinline__ bool epilogue_stats(uint32_t tbase, int row, int n, int nb, int part, Walk& walk,
                                               const HeadArgs& a, uint32_t handed, uint32_t parity, const Ctl& ctl) {
  constexpr int CHUNKS = kHeadTile / 32 / PARTS;
  const int first = a.col0 + nb * kHeadTile;  // vocabulary entry of the tile's first column
  const int width = a.cols - nb * kHeadTile;
  RowStats st;
#pragma unroll 1
  for (int c = part * CHUNKS; c < (part + 1) * CHUNKS; ++c) {
    if (c * 32 >= width) break;
    uint32_t raw[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, raw);
    ptx::tmem_wait_ld();
    st.add(raw, first + c * 32, width - c * 32, walk, a);
  }
  float m = st.m * a.k2, s = st.s, dot = fmaf(a.flat, st.zs, st.dot);
  if constexpr (PARTS == 2) {
    uint32_t x[4] = {__float_as_uint(m), __float_as_uint(s), __float_as_uint(dot), 0u};
    if (part == 1) {
      ptx::tmem_st_32x32b_x4(tbase + kHeadTile / 2, x);
      ptx::tmem_wait_st();
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (ptx::lane_id() == 0) ptx::mbar_arrive(handed);
      return true;
    }
    if (!warp_wait(handed, parity, ctl, SITE_EPI_ACC_FULL)) return false;
    ptx::tc_fence_after_sync();
    ptx::tmem_ld_32x32b_x4(tbase + kHeadTile / 2, x);
    ptx::tmem_wait_ld();
    const float m2 = __uint_as_float(x[0]), top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
    s = s * exp2_fast(m - ref) + __uint_as_float(x[1]) * exp2_fast(m2 - ref);
    m = top;
    dot += __uint_as_float(x[2]);
  }
  if (row < n) {
    const int64_t at = static_cast<int64_t>(a.tile0 + nb) * a.T + row;
    a.ms[at] = make_float2(m, s);
    a.dot[at] = dot;
  }
  return true;
}

// 32 logits of a row -> their gradient.
__device__ __forceinline__ void gradient_chunk(uint32_t (&raw)[32], int base, int limit, const float4& k,
                                               const HeadArgs& a, Walk& walk) {
  const float flat = k.y * a.flat;
  const float2 k2 = make_float2(a.k2, a.k2), off = make_float2(-k.z, -k.z);
  const float2 cp = make_float2(k.x, k.x), cf = make_float2(-flat, -flat);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1])), k2, off);
    const float2 d = __ffma2_rn(cp, make_float2(exp2_fast(x.x), exp2_fast(x.y)), cf);
    raw[2 * i] = __float_as_uint(d.x);
    raw[2 * i + 1] = __float_as_uint(d.y);
  }
  while (__any_sync(0xffffffffu, walk.next < base + 32)) {
    if (walk.next < base + 32) {
      const int t = walk.next - base;
      const float d = k.y * walk.mass();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        raw[i] = i == t ? __float_as_uint(__uint_as_float(raw[i]) - d) : raw[i];
      walk.step();
    }
  }
  if (limit < 32) {  // columns past the piece contribute nothing to the products that follow
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i] = i < limit ? raw[i] : 0u;
  }
}

// This warp's staging buffer, once the last copy out of it has been read.
__device__ __forceinline__ void stage_row(uint8_t* buf, int lane, const uint32_t (&w)[32]) {
  if (lane == 0) ptx::bulk_wait_group_read<0>();
  __syncwarp();
#pragma unroll
  for (int ch = 0; ch < 8; ++ch)
    *reinterpret_cast<uint4*>(buf + sw128_offset(lane, ch * 16)) =
        make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
}

// One 64-column chunk of 16-bit words of 32 rows, to the tensor at (col, row0, plane).
__device__ __forceinline__ void store_words(const uint32_t (&w)[32], const CUtensorMap* mapC, int col, int row0,
                                            int plane, uint8_t* buf, int lane) {
  stage_row(buf, lane, w);
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    ptx::tma_store_3d(mapC, col, row0, plane, ptx::smem_u32(buf));
    ptx::bulk_commit_group();
  }
}

// The same to rows that are not 16-byte aligned: the warp writes one row after
// another, neighbouring lanes neighbouring elements.
__device__ __forceinline__ void store_words_plain(const uint32_t (&w)[32], uint16_t* dst, int64_t ld, int rows,
                                                  int cols, int granule, uint8_t* buf, int lane) {
  stage_row(buf, lane, w);
  __syncwarp();
  if (granule >= 4) {
    const bool whole = 2 * lane + 2 <= cols, single = !whole && 2 * lane < cols;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 8) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint32_t*>(buf + sw128_offset(r0 + i, lane * 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint16_t* row = dst + (r0 + i) * ld;
        if (r0 + i < rows && whole) reinterpret_cast<uint32_t*>(row)[lane] = v[i];
        if (r0 + i < rows && single) row[2 * lane] = static_cast<uint16_t>(v[i] & 0xFFFFu);
      }
    }
  } else {
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 8) {
      uint16_t v[8][2];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[i][h] = *reinterpret_cast<const uint16_t*>(buf + sw128_offset(r0 + i, (lane + 32 * h) * 2));
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r0 + i < rows && lane + 32 * h < cols) dst[(r0 + i) * ld + lane + 32 * h] = v[i][h];
    }
  }
  __syncwarp();
}

// dz of 32 rows, 64 columns at a time; `own`: a second time, times the row's own
// scale k.w, to the planes after the first ones.
template <int PLANES, int PARTS>
__device__ __forceinline__ void epilogue_dz(uint32_t tbase, int row0, int n, int nb, int part, const float4& k,
                                            Walk& walk, const HeadArgs& a, bool own, const CUtensorMap* mapC,
                                            uint8_t* buf, int lane) {
  if (row0 >= a.T) return;
  const int c0 = part * (kHeadTile / 64 / PARTS), c1 = c0 + kHeadTile / 64 / PARTS;
  const int row = row0 + lane;
  const int first = a.col0 + nb * kHeadTile;
  const int width = a.cols - nb * kHeadTile;
  const int fmt = a.bf16 ? OUT_BF16 : OUT_F16;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    if (c * 64 >= width) break;
    uint32_t w[32];
    if constexpr (PLANES == 1) {
      uint32_t scaled[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32];
        ptx::tmem_ld_32x32b_x32(tbase + c * 64 + h * 32, d);
        ptx::tmem_wait_ld();
        gradient_chunk(d, first + c * 64 + h * 32, width - c * 64 - h * 32, k, a, walk);
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // rows past the count: zeros, which the products read
          const float x = __uint_as_float(d[2 * i]), y = __uint_as_float(d[2 * i + 1]);
          w[16 * h + i] = row < n ? pack_pair(x, y, fmt) : 0u;
          scaled[16 * h + i] = row < n ? pack_pair(x * k.w, y * k.w, fmt) : 0u;
        }
      }
      store_words(w, mapC, nb * kHeadTile + c * 64, row0, 0, buf, lane);
      if (own) store_words(scaled, mapC, nb * kHeadTile + c * 64, row0, 1, buf, lane);
      continue;
    }
    uint32_t lo[32], hi[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 64, lo);
    ptx::tmem_wait_ld();
    ptx::tmem_ld_32x32b_x32(tbase + c * 64 + 32, hi);
    gradient_chunk(lo, first + c * 64, width - c * 64, k, a, walk);
    ptx::tmem_wait_ld();
    gradient_chunk(hi, first + c * 64 + 32, width - c * 64 - 32, k, a, walk);
    if (row >= n) {
#pragma unroll
      for (int i = 0; i < 32; ++i) lo[i] = hi[i] = 0u;
    }
    if constexpr (PLANES == 2) {
#pragma unroll 1
      for (int p = 0; p < (own ? 4 : 2); ++p) {
        const float scale = p >= 2 ? k.w : 1.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t* v = i < 16 ? &lo[2 * i] : &hi[2 * i - 32];
          const float x = scale * __uint_as_float(v[0]), y = scale * __uint_as_float(v[1]);
          w[i] = pack_pair(x, y, fmt);
          if (p & 1) {  // what the first plane leaves (0 where it is not finite)
            float px = __uint_as_float(w[i] << 16), py = __uint_as_float(w[i] & 0xFFFF0000u);
            if (fmt == OUT_F16) {
              px = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] & 0xFFFFu)));
              py = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] >> 16)));
            }
            w[i] = pack_pair(isfinite(px) ? x - px : 0.0f, isfinite(py) ? y - py : 0.0f, fmt);
          }
        }
        store_words(w, mapC, nb * kHeadTile + c * 64, row0, p, buf, lane);
      }
    } else {
#pragma unroll
      for (int p = 0; p < PLANES; ++p) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          uint32_t* v = i < 16 ? &lo[2 * i] : &hi[2 * i - 32];
          const float x = __uint_as_float(v[0]), y = __uint_as_float(v[1]);
          w[i] = pack_pair(x, y, OUT_BF16);
          if (p + 1 < PLANES) {  // what the plane leaves (0 where it is not finite)
            const float px = __uint_as_float(w[i] << 16), py = __uint_as_float(w[i] & 0xFFFF0000u);
            v[0] = isfinite(px) ? __float_as_uint(x - px) : 0u;
            v[1] = isfinite(py) ? __float_as_uint(y - py) : 0u;
          }
        }
        store_words(w, mapC, nb * kHeadTile + c * 64, row0, p, buf, lane);
      }
    }
  }
}

// fp32 DW whose rows are off the 16-byte grid: this thread's row, times f.
template <int PARTS>
__device__ __forceinline__ void epilogue_f32(uint32_t tbase, float* row, bool valid_row, int nb, int part, int cols,
                                             float f) {
  const int c0 = part * (kHeadTile / 32 / PARTS), c1 = c0 + kHeadTile / 32 / PARTS;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int col = nb * kHeadTile + c * 32;
    if (col >= cols) break;
    uint32_t w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, w);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (valid_row && col + i < cols) __stcg(row + col + i, f * __uint_as_float(w[i]));
  }
}

// fp32 sums of 32 rows, times f, to the tensor at (column, row0, z) by bulk
// copies: stored, or added.
template <int PARTS>
__device__ __forceinline__ void epilogue_sums(uint32_t tbase, int row0, int nb, int z, int part, int cols, float f,
                                              bool add, const CUtensorMap* mapC, uint8_t* buf, int lane) {
  const int c0 = part * (kHeadTile / 32 / PARTS), c1 = c0 + kHeadTile / 32 / PARTS;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int col = nb * kHeadTile + c * 32;
    if (col >= cols) break;
    uint32_t w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, w);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(f * __uint_as_float(w[i]));
    stage_row(buf, lane, w);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add)
        tma_reduce_add_3d(mapC, col, row0, z, ptx::smem_u32(buf));
      else
        ptx::tma_store_3d(mapC, col, row0, z, ptx::smem_u32(buf));
      ptx::bulk_commit_group();
    }
  }
}

template <int PARTS>
__device__ __forceinline__ void epilogue_dw(uint32_t tbase, int row0, int nb, int part, float f, const HeadArgs& a,
                                            const CUtensorMap* mapC, uint8_t* buf, int lane) {
  const int fmt = a.bf16 ? OUT_BF16 : OUT_F16;
  const int c0 = part * (kHeadTile / 64 / PARTS), c1 = c0 + kHeadTile / 64 / PARTS;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int col = nb * kHeadTile + c * 64;
    if (col >= a.D) break;
    uint32_t lo[32], hi[32], w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 64, lo);
    ptx::tmem_ld_32x32b_x32(tbase + c * 64 + 32, hi);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w[i] = pack_pair(f * __uint_as_float(lo[2 * i]), f * __uint_as_float(lo[2 * i + 1]), fmt);
      w[16 + i] = pack_pair(f * __uint_as_float(hi[2 * i]), f * __uint_as_float(hi[2 * i + 1]), fmt);
    }
    if (a.store_granule == 0)
      store_words(w, mapC, col, a.out_row0 + row0, 0, buf, lane);
    else
      store_words_plain(w, static_cast<uint16_t*>(a.out) + static_cast<int64_t>(a.out_row0 + row0) * a.ld_out + col,
                        a.ld_out, a.cols - row0, a.D - col, a.store_granule, buf, lane);
  }
}

// One product, by CTA pair `worker` of `workers`.  CHUNKS: its k axis may be
// longer than a chunk.
template <int MODE, int PLANES, int PARTS, bool CHUNKS>
__device__ __forceinline__ void head_product(const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                                             const HeadArgs& args, const int worker, const int workers) {
  constexpr int STAGES = head_stages(MODE, PARTS);
  using Plane = Terms<MODE, PLANES>;
  constexpr int TERMS = Plane::count;
  constexpr int ACC = 256;
  constexpr uint32_t TMEM_COLS = 512;
  static_assert(head_smem(MODE, PARTS) <= kSmemLimit, "shared memory per CTA");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sC = smem + STAGES * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(sC + head_epi_bytes(MODE, PARTS));
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* handed = acc_empty + 2;  // STATS: [unit & 1][quarter]
  uint64_t* drain = handed + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  static_assert((2 * STAGES + 13) * 8 + 8 <= kBarrierBytes, "barrier area");
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(ptx::cluster_ctarank() & 1u);  // which 128 rows of the pair's tile
  const bool leader = cta == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&acc_full[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&acc_empty[b]), 2 * 4 * PARTS);
    }
    for (int i = 0; i < 8; ++i) ptx::mbar_init(ptx::smem_u32(&handed[i]), 1);
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&mapA);
    ptx::tma_prefetch_desc(&mapB);
    if (MODE != HEAD_STATS) ptx::tma_prefetch_desc(&mapC);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before_sync();
  ptx::cluster_sync();
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // set-up overlaps the end of the kernel before; its results are read from here on
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  const Ctl ctl{abort_flag, args.timeout_ns, args.status};
  const int n = args.count ? min(*args.count, args.T) : args.T;
  const Tiles tiles = head_tiles<MODE>(args, max(1, n));
  // stages summed in tensor memory at a time: a unit's, in even parts of at most args.chunk
  static_assert(!CHUNKS || PARTS == 2, "128 columns a thread");
  const int stages_all = MODE == HEAD_DH ? min(args.k_per_split, tiles.k_blocks) : tiles.k_blocks;
  const int chunks = (stages_all + args.chunk - 1) / args.chunk;
  const int chunk = CHUNKS ? max(1, (stages_all + chunks - 1) / max(1, chunks)) : INT_MAX / 2;

  if (warp == 0) {
    // ------------------------------------------------ bulk-tensor producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, last_parity = 0;
      bool ok = true;
      const int first_plane = MODE == HEAD_DH && PLANES < 3 && args.spread && __ldcg(args.spread) ? PLANES : 0;
      for (int i = worker; ok && i < tiles.units; i += workers) {
        const HeadUnit u = head_unit<MODE>(args, tiles, i);
        const int m0 = u.mb * kHeadTile + cta * kTileM;
        const int n0 = u.nb * kHeadTile + cta * (kHeadTile / 2);
        for (int lo = u.lo; ok && lo < u.hi; lo += chunk) {
          const int span = min(chunk, u.hi - lo);
          for (int it = 0; it < TERMS * span; ++it) {
            if (!wait_bounded(ptx::smem_u32(&empty[stage]), phase ^ 1u, ctl, SITE_PRODUCER_EMPTY)) {
              ok = false;
              break;
            }
            // fp32: one pair of planes over all stages after another; two planes
            // of dz: stage by stage, so that the second finds W in L2
            const int term = TERMS == 6 ? it / span : it % TERMS;
            const int k0 = (lo + (TERMS == 6 ? it - term * span : it / TERMS)) * kTileK;  // past the k axis: zeros
            const int pa = first_plane + Plane::a(term), pb = Plane::b(term);
            const uint32_t fb_local = ptx::smem_u32(&full[stage]);
            const uint32_t fb = ptx::mapa_shared(fb_local, 0);
            if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2u * kStage);
            const uint32_t sa = ptx::smem_u32(smem + stage * kStage), sb = sa + kSub;
            if constexpr (a_m_major(MODE)) {
              ptx::tma_load_3d_pair(sa, &mapA, m0, k0, pa, fb);
              ptx::tma_load_3d_pair(sa + 8192, &mapA, m0 + 64, k0, pa, fb);
            } else {
              ptx::tma_load_3d_pair(sa, &mapA, k0, m0, pa, fb);
            }
            if constexpr (b_n_major(MODE)) {
              const int kr = k0 + (MODE == HEAD_DH ? args.b_row0 : 0);
              ptx::tma_load_3d_pair(sb, &mapB, n0, kr, pb, fb);
              ptx::tma_load_3d_pair(sb + 8192, &mapB, n0 + 64, kr, pb, fb);
            } else {
              ptx::tma_load_3d_pair(sb, &mapB, k0, args.b_row0 + n0, pb, fb);
            }
            filled |= 1u << stage;
            last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      // loads in flight land before shared memory is released (see tc_gemm_2sm.cu)
      for (int s = 0; s < STAGES; ++s)
        if ((filled >> s) & 1u) {
          const uint32_t par = (last_parity >> s) & 1u;
          wait_teardown(ptx::smem_u32(leader ? &full[s] : &empty[s]), par, ctl, SITE_TEARDOWN);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------ MMA issuer (leader CTA only)
    if (leader && lane == 0) {
      // kind::f16 instruction descriptor: D fp32, A and B format, A M-major
      // (bit 15), B N-major (bit 16), N >> 3, M >> 4
      const uint32_t ab = args.bf16 ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (ab << 7) | (ab << 10) | (a_m_major(MODE) ? 1u << 15 : 0u) |
                             (b_n_major(MODE) ? 1u << 16 : 0u) | (static_cast<uint32_t>(kHeadTile >> 3) << 17) |
                             (static_cast<uint32_t>((2 * kTileM) >> 4) << 24);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = worker; ok && i < tiles.units; i += workers) {
        const HeadUnit u = head_unit<MODE>(args, tiles, i);
        for (int lo = u.lo; ok && lo < u.hi; lo += chunk) {
          if (!wait_bounded(ptx::smem_u32(&acc_empty[acc]), acc_phase ^ 1u, ctl, SITE_MMA_ACC_EMPTY)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * ACC);
          const int stages = TERMS * min(chunk, u.hi - lo);
          for (int it = 0; it < stages; ++it) {
            if (!wait_bounded(ptx::smem_u32(&full[stage]), phase, ctl, SITE_MMA_FULL)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after_sync();
            const uint32_t a0 = ptx::smem_u32(smem + stage * kStage), b0 = a0 + kSub;
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k) {
              const uint64_t da =
                  a_m_major(MODE) ? sw128_desc(a0 + k * 2048, 8192, 1024) : sw128_desc(a0 + k * 32, 16, 1024);
              const uint64_t db =
                  b_n_major(MODE) ? sw128_desc(b0 + k * 2048, 8192, 1024) : sw128_desc(b0 + k * 32, 16, 1024);
              ptx::tc_mma_f16_pair(d_tmem, da, db, idesc, (it != 0 || k != 0) ? 1u : 0u);
            }
            ptx::tc_commit_pair_multicast(ptx::smem_u32(&empty[stage]), 0x3);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          ptx::tc_commit_pair_multicast(ptx::smem_u32(&acc_full[acc]), 0x3);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_teardown(ptx::smem_u32(drain), 0, ctl, SITE_DRAIN);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue
    const int quarter = warp & 3;              // tensor-memory lanes of this warp
    const int part = (warp - 2) / 4;           // its part of the tile's columns
    uint8_t* buf = sC + (warp - 2) * 4096;
    const float factor = MODE == HEAD_DW ? __ldcg(args.factor) : 1.0f;
    const bool own = MODE == HEAD_DZ && PLANES < 3 && args.spread && __ldcg(args.spread);
    int acc = 0, done = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    // the next accumulator, once its sums are complete
    const auto taken = [&]() {
      ok = warp_wait(ptx::smem_u32(&acc_full[acc]), acc_phase, ctl, SITE_EPI_ACC_FULL);
      ptx::tc_fence_after_sync();
      return tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * ACC);
    };
    // The accumulator's reads are complete (tcgen05.wait::ld).  The arrival
    // orders nothing else: a releasing one would wait for this tile's global
    // stores, 1500 cycles a tile.
    const auto given_back = [&]() {
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&acc_empty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    };
    HeadUnit u;
    int64_t target = -1;
    float4 coef = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto look_up = [&](const HeadUnit& w) {
      if constexpr (MODE == HEAD_STATS || MODE == HEAD_DZ) {
        const int row = w.mb * kHeadTile + cta * kTileM + quarter * 32 + lane;
        if (args.target) target = row < n ? __ldcg(args.target + row) : -1;
        if (MODE == HEAD_DZ) coef = row < n ? __ldcg(args.coef + row) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    };
    // One chunk: the next tile is found, and its rows' targets and coefficients
    // loaded, while this one's products run; a short k axis would not hide it.
    // Several: they are found behind the last chunk, whose epilogue has the next
    // tile's first chunk to run under, and no register is theirs beside the sums.
    HeadUnit next;
    const auto look_ahead = [&](int i) {
      if (i >= tiles.units) return;
      next = head_unit<MODE>(args, tiles, i);
      look_up(next);
    };
    if constexpr (!CHUNKS) look_ahead(worker);
    for (int i = worker; ok && i < tiles.units; i += workers) {
      u = CHUNKS ? head_unit<MODE>(args, tiles, i) : next;
      const int row0 = u.mb * kHeadTile + cta * kTileM + quarter * 32;
      const int rows_end = MODE == HEAD_DW ? args.cols : MODE == HEAD_DZ ? args.T : n;
      const int first = args.col0 + u.nb * kHeadTile + part * (kHeadTile / PARTS);
      float4 k = coef;
      Walk walk;
      uint32_t tbase;
      if (u.lo >= u.hi) {  // a split past the end of a short last piece
        if constexpr (!CHUNKS) look_ahead(i + workers);
        continue;
      }
      if constexpr (CHUNKS) {
        int lo = u.lo + chunk;  // end of the chunk to come
        tbase = taken();
        if (lo < u.hi && row0 < rows_end) {
          // every path to a use of the sums passes their first load: else they
          // would be live, and registers short, in all of the epilogue
          if (ok) {
            uint32_t sum[8][16];
            load_sums(tbase + part * (kHeadTile / 2), sum);
            given_back();
            for (lo += chunk;; lo += chunk) {
              tbase = taken();
              if (!ok) break;
              add_sums(tbase + part * (kHeadTile / 2), sum);
              if (lo >= u.hi) {
                store_sums(tbase + part * (kHeadTile / 2), sum);
                break;
              }
              given_back();
            }
          }
        } else {
          for (; ok && lo < u.hi; lo += chunk) {
            given_back();
            tbase = taken();
          }
        }
        look_up(u);
        k = coef;
        if constexpr (MODE == HEAD_STATS || MODE == HEAD_DZ) walk.start(args, row0 + lane, n, first, target);
      } else {
        if constexpr (MODE == HEAD_STATS || MODE == HEAD_DZ) walk.start(args, row0 + lane, n, first, target);
        look_ahead(i + workers);
        tbase = taken();
      }
      if (!ok) break;
      if (row0 < rows_end) {
        if constexpr (MODE == HEAD_STATS) {
          ok = epilogue_stats<PARTS>(tbase, row0 + lane, n, u.nb, part, walk, args,
                                     ptx::smem_u32(&handed[(done & 1) * 4 + quarter]), (done >> 1) & 1, ctl);
          ++done;
        } else if constexpr (MODE == HEAD_DZ) {
          epilogue_dz<PLANES, PARTS>(tbase, row0, n, u.nb, part, k, walk, args, own, &mapC, buf, lane);
        } else if constexpr (PLANES < 3 && MODE == HEAD_DW) {
          epilogue_dw<PARTS>(tbase, row0, u.nb, part, factor, args, &mapC, buf, lane);
        } else if (MODE == HEAD_DH || args.store_granule == 0) {
          epilogue_sums<PARTS>(tbase, MODE == HEAD_DW ? args.out_row0 + row0 : row0, u.nb, u.split, part, args.D, factor,
                               args.reduce, &mapC, buf, lane);
        } else {
          const int row = row0 + lane;
          float* out = static_cast<float*>(args.out) + static_cast<int64_t>(args.out_row0 + row) * args.ld_out;
          epilogue_f32<PARTS>(tbase, out, row < rows_end, u.nb, part, args.D, factor);
        }
      }
      given_back();
    }
    if (lane == 0) ptx::bulk_wait_group_read<0>();
    __syncwarp();
  }

  // ------------------------------------------------------------- teardown
  ptx::tc_fence_before_sync();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int MODE, int PLANES, int PARTS, bool CHUNKS>
__global__ void __launch_bounds__(head_threads(PARTS), 1)
    head_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ CUtensorMap mapC, const __grid_constant__ HeadArgs args) {
  head_product<MODE, PLANES, PARTS, CHUNKS>(mapA, mapB, mapC, args, blockIdx.x / 2, gridDim.x / 2);
}

// Launch of a kernel on `pairs` clusters of two CTAs, dependent on the kernel before it.
template <typename... Params, typename... Args>
cudaError_t launch_pairs(void (*kernel)(Params...), int smem, int threads, std::atomic<uint64_t>& done_mask, int pairs,
                         cudaStream_t stream, const Args&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MODE, int PLANES, int PARTS, bool CHUNKS>
cudaError_t launch(const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap& mC, const HeadArgs& args,
                   int pairs, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  return launch_pairs(head_kernel<MODE, PLANES, PARTS, CHUNKS>, head_smem(MODE, PARTS), head_threads(PARTS), done_mask, pairs,
                      stream, mA, mB, mC, args);
}

}  // namespace
}  // namespace tgemm
