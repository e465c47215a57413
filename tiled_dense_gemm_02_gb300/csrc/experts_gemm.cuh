// Tensor-core products of the experts, on CTA pairs: tcgen05.mma.cta_group::2, M =
// 256, fp32 accumulators in tensor memory, two of them, so a tile's epilogue
// runs under the next tile's MMAs.
//
// With e an expert, its rows' tokens t and 1 <= n <= 256 of its rows a tile:
//
//   UP    W_in[e] x_t           M = 128 features' gates and ups, N = n, K = D
//   DOWN  W_out[e] h            M = D, N = n, K = F
//   DH    W_out[e]^T d_out_t    M = F, N = n, K = D
//   DX    W_in[e]^T (dg, du)    M = D, N = n, K = 2 F
//   DIN   (dg, du)^T x          M = 2 F, N = D, K = the expert's rows
//   DOUT  d_out^T (w h)         M = D, N = F, K = the expert's rows
//
// The weight is the M operand and the tokens are N, which tcgen05 takes in steps of
// 32: an expert with a handful of rows computes 32 columns, not 256, and the same
// kernel serves one token (bound by the weights' bytes, each read once) and a
// training batch (bound by the MMAs).  Rows of x and d_out lie sorted in the
// workspace (gather_rows); no operand is transposed in memory.  Calls of few rows
// read x where it lies (GATHER) by gathering bulk-tensor copies of four rows each
// (tile::gather4), every lane of the producer warp issuing its own: one launch
// less, but from some hundred rows a tile on these copies are the bound (8192 tokens
// in 64 experts: UP 1260 us, and 560 with sorted rows).
//
// UP interleaves 16 gate rows with their 16 ups, so that a warp's 32 lanes
// of tensor memory hold both of 16 features: of 16 columns, lane l finishes
// the first eight and lane l + 16 the others, after an exchange of eight values.
//
// The adder of tcgen05.mma truncates: a step moves the sum towards 0 by up to 2^-23
// of it.  Sums leave tensor memory every `chunk` stages (four steps each) and are
// added in registers, with rounding to nearest, under the next chunk's MMAs; the
// last sum goes back to tensor memory, where the epilogues read it.
//
// Rounded to 16 bits between two products, by choice: h into DOWN, and dg, du and w h into DX, DIN
// and DOUT (fp16: with their expert's powers of two, round_kernel), since the tensor cores take
// both operands in the weights' type.  Results are then 1.42 times as far off, in the norm, as
// their own last rounding (1.65e-3 in bf16).  A second plane with what the first loses would make
// that 1.0 and double those products' steps: 8192 tokens, 8 of 64 experts of 2048 x 1024, DOWN
// 230 -> 388 us of 746; a step of 8192 x 4 of 32 experts of 2048 x 1408, the four 798 -> 1451 us of 1600
// (each timed with twice the k axis).  Built for forward calls of up to 2048 places, where the weights'
// bytes are the bound, it took 64 tokens, 8 of 128 experts of 2048 x 768 from 195 to 207 us and 1024
// tokens, 2 of 8 of 4096 x 4096 from 459 to 548, and such a call's out was no longer the bits that a
// call gives which keeps g and u.  g, u, d_weights and all sums are fp32.
//
// Roles: warp 0 copies, warp 1 MMAs (one thread of the leader), warps 2.. epilogue,
// eight, or sixteen (DH, and UP where g and u are kept: they move most bytes): a
// quarter of the lanes and a share of the columns each.  Every role
// derives the units from the tile list, which is known on the device only.  Every
// wait is bounded (tc_common.cuh).
#pragma once

#include "experts_gate.cuh"
#include "experts_internal.h"
#include "tc_pair.cuh"

namespace tgemm {
namespace {

constexpr bool weight_gradient(int mode) { return mode == EXPERT_DIN || mode == EXPERT_DOUT; }
// PARTS: epilogue warps per quarter of the lanes.
constexpr int expert_threads(int parts) { return 32 * (2 + 4 * parts); }
// 16-bit results on their way out: 4 KB a warp (weights' gradients), or for each part three
// buffers of 16 rows and the CTA's 64 features (UP), or two of 32 rows and its 128.
constexpr int staged_bytes(int mode) { return mode == EXPERT_UP ? 2048 : 8192; }
constexpr int staged_buffers(int mode) { return mode == EXPERT_UP ? 3 : 2; }
constexpr int expert_epi_bytes(int mode, int parts) {
  return weight_gradient(mode) ? 4 * parts * 4096 : mode == EXPERT_DH ? 0 : staged_buffers(mode) * parts * staged_bytes(mode);
}
constexpr int expert_stages(int mode, int parts) {
  return (kSmemLimit - 1024 - expert_epi_bytes(mode, parts) - kBarrierBytes) / kStage;
}
constexpr int expert_smem(int mode, int parts) {
  return 1024 + expert_stages(mode, parts) * kStage + expert_epi_bytes(mode, parts) + kBarrierBytes;
}
constexpr bool expert_a_m_major(int mode) { return mode >= EXPERT_DH; }
constexpr bool expert_b_n_major(int mode) { return weight_gradient(mode); }

// Four rows of a tensor, 64 columns from x on, into 512 bytes of this CTA's shared
// memory; completion on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* map, int32_t x, const int4& rows,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar_cluster)
      : "memory");
}

// A tile of a product: block mb of M, and N's columns (rows row0.. of the sorted
// matrices, n with the filling and `valid` without; gradients of the weights:
// column block nb, and rows row0.. are the k axis).
struct ExpertUnit {
  int expert, mb, nb, row0, n, valid;
};

template <int MODE>
struct ExpertUnits {
  int count;
  __device__ __forceinline__ explicit ExpertUnits(const ExpertArgs& a) {
    count = weight_gradient(MODE) ? a.E * a.m_blocks * a.n_blocks : __ldcg(a.rows.head) * a.m_blocks;
  }
  __device__ __forceinline__ ExpertUnit get(const ExpertArgs& a, int i) const {
    ExpertUnit u = {};
    if (i >= count) return u;
    if constexpr (weight_gradient(MODE)) {
      const int per = a.m_blocks * a.n_blocks;
      u.expert = i / per;
      i -= u.expert * per;
      u.nb = i / a.m_blocks;
      u.mb = i - u.nb * a.m_blocks;
      u.row0 = __ldcg(a.rows.first + u.expert);
      u.n = __ldcg(a.rows.first + u.expert + 1) - u.row0;
      u.valid = u.n;
    } else {
      const int t = i / a.m_blocks;
      u.mb = i - t * a.m_blocks;
      const int4 tile = __ldcg(a.rows.tiles + t);
      u.expert = tile.x;
      u.row0 = tile.y;
      u.n = tile.z;
      u.valid = tile.w;
    }
    return u;
  }
  __device__ __forceinline__ int stages(const ExpertArgs& a, const ExpertUnit& u) const {
    return weight_gradient(MODE) ? (u.n + kTileK - 1) / kTileK : a.k_blocks;
  }
};

// Sums of this thread's lane in its MOST blocks of 16 columns, every STEP-th one.
// (Blocks past the tile's columns are summed too: a condition on each would cost
// the registers that hold them, and no other warp has them.)
template <int STEP, int MOST>
__device__ __forceinline__ void first_sums(uint32_t tcol, uint32_t (&sum)[MOST][16]) {
#pragma unroll
  for (int b = 0; b < MOST; ++b) ptx::tmem_ld_32x32b_x16(tcol + b * STEP * 16, sum[b]);
  ptx::tmem_wait_ld();
}
template <int STEP, int MOST>
__device__ __forceinline__ void more_sums(uint32_t tcol, uint32_t (&sum)[MOST][16]) {
#pragma unroll
  for (int b = 0; b < MOST; ++b) {
    uint32_t raw[16];
    ptx::tmem_ld_32x32b_x16(tcol + b * STEP * 16, raw);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      sum[b][i] = __float_as_uint(__uint_as_float(sum[b][i]) + __uint_as_float(raw[i]));
  }
}
template <int STEP, int MOST>
__device__ __forceinline__ void whole_sums(uint32_t tcol, const uint32_t (&sum)[MOST][16]) {
#pragma unroll
  for (int b = 0; b < MOST; ++b) ptx::tmem_st_32x32b_x16(tcol + b * STEP * 16, sum[b]);
  ptx::tmem_wait_st();
}

// Where a lane stores 16-bit values of its feature, two rows at a time.  Neighbouring
// lanes hold neighbouring features; PAIRS: each stores both features of one of the
// two rows (the matrix's features pair up in words), else both rows of its own.
template <bool PAIRS>
struct RowStore {
  uint16_t* p;
  int64_t ld;
  bool odd, in;
  // feature: the lane's, of F
  __device__ __forceinline__ RowStore(void* base, int64_t row, int64_t pitch, int feature, int F, int lane)
      : p(static_cast<uint16_t*>(base) + row * pitch + feature), ld(pitch), odd((lane & 1) != 0), in(feature < F) {
    if (PAIRS && odd) p += ld - 1;
  }
  // word: {row, next row} of the lane's feature
  __device__ __forceinline__ void put(uint32_t word) {
    if constexpr (PAIRS) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 1);
      const uint32_t both = odd ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
      if (in) *reinterpret_cast<uint32_t*>(p) = both;
    } else if (in) {
      p[0] = static_cast<uint16_t>(word & 0xFFFFu);
      p[ld] = static_cast<uint16_t>(word >> 16);
    }
    p += 2 * ld;
  }
};

// The same by way of shared memory: the four warps of a part (the quarters of the lanes)
// put 16 rows of their CTA's features together, 128-byte-swizzled blocks of 64, and one
// of them stores these by bulk copies.  Stores of 64 bytes a row by the threads themselves
// share the SM's port with the operands' loads, piece by piece.
template <int BUFFERS, int BYTES>
struct StagedRows {
  uint8_t* buffers;
  int next, part, quarter;

  __device__ __forceinline__ void barrier() const { asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory"); }
  // The buffer at hand may be written.  Of three it may since the last barrier: the copy out
  // of it was followed by one whose issuer waited for it before that barrier.
  __device__ __forceinline__ void acquire(int lane) const {
    if constexpr (BUFFERS == 2) {
      if (quarter == 0 && lane == 0) ptx::bulk_wait_group_read<1>();
      barrier();
    }
  }
  // Where the lane's 64 features of the buffer's block (16 rows) lie.  feature: the lane's,
  // in the CTA.
  __device__ __forceinline__ uint8_t* block(int feature, int b = 0) const {
    return buffers + next * BYTES + b * 4096 + feature / 64 * 2048;
  }
  // word: {row, row + 1} of the lane's feature, row even
  static __device__ __forceinline__ void put(uint8_t* block, uint32_t word, int row, int feature, int lane) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 1);
    const bool odd = (lane & 1) != 0;
    const uint32_t both = odd ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
    *reinterpret_cast<uint32_t*>(block + sw128_offset(row + (odd ? 1 : 0), (feature & 62) * 2)) = both;
  }
  // The buffer's words are there: one warp stores `columns` of them from column x on, to rows
  // `row`.. and (blocks 2) `other`...
  __device__ __forceinline__ void store(const CUtensorMap* map, int x, int columns, int row, int blocks, int other, int lane) {
    ptx::fence_proxy_async_smem();
    barrier();
    if (quarter == 0 && lane == 0) {
      const uint32_t src = ptx::smem_u32(buffers + next * BYTES);
      for (int b = 0; b < blocks; ++b) {
        if (columns > 0) ptx::tma_store_3d(map, x, b ? other : row, 0, src + b * 4096);
        if (columns > 64) ptx::tma_store_3d(map, x + 64, b ? other : row, 0, src + b * 4096 + 2048);
      }
      ptx::bulk_commit_group();
      if (BUFFERS == 3) ptx::bulk_wait_group_read<1>();
    }
    if (++next == BUFFERS) next = 0;
  }
};
// Whether all four warps of a part go on (a wait that ran out in one of them ends them all:
// none waits for another at a barrier).
__device__ __forceinline__ bool part_agrees(bool ok, int part) {
  uint32_t all;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 q, %1, 0;\n"
      "bar.red.and.pred p, %2, 128, q;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(1 + part)
      : "memory");
  return all != 0;
}

// 16 columns of UP: gates in lanes 0..15, ups in lanes 16..31 -> h, and g and u.
// `row`: the columns' first row, of which `valid` are no filling (which gets 0).
// g and u lie as {g, u} x features x 4 rows for every four rows: 16 bytes a lane.
// staged: the lane's feature in the CTA is `own`.
template <typename Staged>
__device__ __forceinline__ void finish_up(const uint32_t (&v)[16], const ExpertArgs& a, int feature, int64_t row,
                                          int valid, int fmt, int lane, int own, const Staged& staged) {
  const bool low = lane < 16;
  const int c0 = low ? 0 : 8;
  uint8_t* h = staged.block(own);
  float g[8], u[8], x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, low ? v[8 + i] : v[i], 16);
    g[i] = __uint_as_float(low ? v[i] : got);
    u[i] = __uint_as_float(low ? got : v[8 + i]);
    x[i] = g[i] * fast_sigmoid(g[i]) * u[i];
  }
  if (valid < 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c0 + i < valid ? x[i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) Staged::put(h, pack_pair(x[i], x[i + 1], fmt), c0 + i, own, lane);
  if (a.gu && feature < a.F) {
    float4* gu = reinterpret_cast<float4*>(a.gu) + (row + c0) / 4 * 2 * a.ldg + feature;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      __stcs(gu, make_float4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]));
      __stcs(gu + a.ldg, make_float4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]));
      gu += 2 * a.ldg;
    }
  }
}

// 8 columns of DH: v = d_out W_out of this lane's feature, with g and u.  0 in the filling,
// whatever the weights hold, and past the last feature, where the weights are 0 and an infinite
// gradient makes NaN of their product, which has no part in the row's dot.
struct HiddenColumns {
  float g[8], u[8], d[8];
  __device__ __forceinline__ HiddenColumns(const uint32_t (&v)[8], const ExpertArgs& a, int feature, int64_t row, int valid) {
    const float4* gu = reinterpret_cast<const float4*>(a.gu) + row / 4 * 2 * a.ldg + feature;
    float4 g4[2], u4[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      g4[q] = u4[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (feature < a.F) {
        g4[q] = __ldcg(gu);
        u4[q] = __ldcg(gu + a.ldg);
      }
      gu += 2 * a.ldg;
      g[4 * q] = g4[q].x, g[4 * q + 1] = g4[q].y, g[4 * q + 2] = g4[q].z, g[4 * q + 3] = g4[q].w;
      u[4 * q] = u4[q].x, u[4 * q + 1] = u4[q].y, u[4 * q + 2] = u4[q].z, u[4 * q + 3] = u4[q].w;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) d[c] = __uint_as_float(v[c]);
    const int there = feature < a.F ? valid : 0;
    if (there < 8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c >= there) g[c] = u[c] = d[c] = 0.0f;
      }
    }
  }
};

// Sums of h v over the 32 lanes (d: h v of 8 columns): a lane keeps half of its columns at each
// exchange, and ends with a quarter of one column's.
__device__ __forceinline__ void finish_dots(float (&d)[8], const ExpertArgs& a, int64_t row, int valid, int lane, int part,
                                            int parts) {
#pragma unroll
  for (int width = 4; width >= 1; width >>= 1) {
    const bool high = (lane & (4 * width)) != 0;
#pragma unroll
    for (int c = 0; c < width; ++c) {
      const float got = __shfl_xor_sync(0xffffffffu, high ? d[c] : d[c + width], 4 * width);
      d[c] = (high ? d[c + width] : d[c]) + got;
    }
  }
  float sum = d[0] + __shfl_xor_sync(0xffffffffu, d[0], 2);
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  const int c = lane >> 2;
  if ((lane & 3) == 0 && c < valid) __stcg(a.dots + (row + c) * parts + part, sum);
}

// 8 columns of DH for bf16 operands: dg, du and w h in 16 bits.  `mine`: in lane first + c the
// weight of column c.
template <bool PAIRS>
__device__ __forceinline__ void finish_dh(const uint32_t (&v)[8], const ExpertArgs& a, int feature, int64_t row,
                                          int valid, int fmt, int lane, float mine, int first, int part, int parts) {
  HiddenColumns x(v, a, feature, row, valid);
  RowStore<PAIRS> dg_rows(a.dgu, row, a.ld_dgu, feature, a.F, lane), hw_rows(a.h, row, a.ldh, feature, a.F, lane);
  RowStore<PAIRS> du_rows = dg_rows;
  du_rows.p += a.F;
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    float dg[2], du[2], h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float w = __shfl_sync(0xffffffffu, mine, first + c + e);
      const GatedGradient d = gated_gradient(x.g[c + e], x.u[c + e], w * x.d[c + e]);
      dg[e] = d.dg;
      du[e] = d.du;
      x.d[c + e] *= d.h;
      h[e] = w * d.h;
    }
    dg_rows.put(pack_pair(dg[0], dg[1], fmt));
    du_rows.put(pack_pair(du[0], du[1], fmt));
    hw_rows.put(pack_pair(h[0], h[1], fmt));
  }
  finish_dots(x.d, a, row, valid, lane, part, parts);
}

// The larger of `most` and |x| where x is finite, as floats' bits.
__device__ __forceinline__ uint32_t larger_finite(uint32_t most, float x) {
  const uint32_t size = __float_as_uint(x) & 0x7FFFFFFFu;
  return size < 0x7F800000u ? max(most, size) : most;
}

// The same for fp16 operands: v in fp32, 16 bytes a lane, and the largest finite |dg|, |du| and
// |w h| so far.
__device__ __forceinline__ void finish_v(const uint32_t (&v)[8], const ExpertArgs& a, int feature, int64_t row, int valid,
                                         int lane, float mine, int first, int part, int parts, uint32_t (&most)[2]) {
  HiddenColumns x(v, a, feature, row, valid);
  if (feature < a.F) {
    float4* to = reinterpret_cast<float4*>(a.v) + row / 4 * a.ldg + feature;
    __stcs(to, make_float4(x.d[0], x.d[1], x.d[2], x.d[3]));
    __stcs(to + a.ldg, make_float4(x.d[4], x.d[5], x.d[6], x.d[7]));
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float w = __shfl_sync(0xffffffffu, mine, first + c);
    const GatedGradient d = gated_gradient(x.g[c], x.u[c], w * x.d[c]);
    most[0] = larger_finite(larger_finite(most[0], d.dg), d.du);
    most[1] = larger_finite(most[1], w * d.h);
    x.d[c] *= d.h;
  }
  finish_dots(x.d, a, row, valid, lane, part, parts);
}

// 16 columns of DOWN or DX for fp16 operands: fp32 times f, one row's 32 neighbouring elements
// a store.
__device__ __forceinline__ void finish_y(const uint32_t (&v)[16], const ExpertArgs& a, int d, int64_t row, int valid, float f) {
  if (d >= a.D) return;
  float* y = static_cast<float*>(a.y) + row * a.ldy + d;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    if (c < valid) __stcg(y, f * __uint_as_float(v[c]));
    y += a.ldy;
  }
}

// The same for bf16 operands: halves, with one power of two for a row's 32 neighbours that
// brings the largest finite one to [2^14, 2^15).  A half's 11 bits are off by 1.4e-4 on
// average, which beside h's rounding and the result's (1.65e-3 each) is 0.2 % of the error; y's
// bytes, written here and read by the join, are what DOWN's epilogue costs (8192 tokens, 64
// experts, fp32: join 94 us, 53 so).  Where one of the 32 is no 0 and below 2^-28 of the largest, and
// would lose bits as a half, they are stored as bf16, with its range, under the exponent 0.
// y: the block's words in shared memory; own: the lane's feature in the CTA.
__device__ __forceinline__ void row_sizes(const uint32_t (&v)[16], uint32_t (&most)[16]) {
  uint32_t all = 0u;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    most[c] = __reduce_max_sync(0xffffffffu, v[c] & 0x7FFFFFFFu);
    all = max(all, most[c]);
  }
  if (all >= 0x7F800000u) {  // infinities and NaN stay what they are, and take nothing from their neighbours
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint32_t size = v[c] & 0x7FFFFFFFu;
      most[c] = __reduce_max_sync(0xffffffffu, size < 0x7F800000u ? size : 0u);
    }
  }
}
template <typename Staged>
__device__ __forceinline__ void finish_y_half(const uint32_t (&v)[16], const uint32_t (&most)[16], const ExpertArgs& a,
                                              int d, int64_t row, int lane, int own, bool there, uint8_t* y) {
  uint32_t exponents[4] = {0u, 0u, 0u, 0u};
  float f[16], least = INFINITY;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const uint32_t exponent = max(15u, most[c] >> 23);
    exponents[c / 4] |= exponent << (8 * (c & 3));
    f[c] = __uint_as_float((268u - exponent) << 23) * __uint_as_float(v[c]);
    least = fminf(least, fabsf(f[c]));
  }
  uint32_t wide = 0u;  // the rows in bf16
  if (__any_sync(0xffffffffu, least < 0x1p-14f)) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (__any_sync(0xffffffffu, (v[c] & 0x7FFFFFFFu) != 0u && fabsf(f[c]) < 0x1p-14f)) {
        wide |= 1u << c;
        exponents[c / 4] &= ~(0xFFu << (8 * (c & 3)));
      }
  }
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    uint32_t word = pack_pair(f[c], f[c + 1], OUT_F16);
    if (wide) {
      const uint32_t plain = pack_pair(__uint_as_float(v[c]), __uint_as_float(v[c + 1]), OUT_BF16);
      const uint32_t mask = (wide >> c & 1u ? 0xFFFFu : 0u) | (wide >> (c + 1) & 1u ? 0xFFFF0000u : 0u);
      word = (word & ~mask) | (plain & mask);
    }
    Staged::put(y, word, c, own, lane);
  }
  if (there && lane < 16 && d - lane < a.ldy) {
    const uint32_t word = lane < 8 ? (lane < 4 ? exponents[0] : exponents[1]) : (lane < 12 ? exponents[2] : exponents[3]);
    a.y_exponent[(row / 16 * (a.ldy / 32) + d / 32) * 16 + lane] = static_cast<uint8_t>(word >> (8 * (lane & 3)));
  }
}

// A weight's gradient: this warp's 32 rows of M, its 128 columns of N.  `sums`: 0 for
// an expert without rows.
__device__ __forceinline__ void finish_weight(uint32_t tcol, bool sums, const ExpertArgs& a, int expert, int row0, int M,
                                              int col0, int N, float f, const CUtensorMap* mapC, uint8_t* buf, int lane) {
  if (row0 >= M) return;
  const int fmt = a.bf16 ? OUT_BF16 : OUT_F16;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int col = col0 + c * 64;
    if (col >= N) break;
    uint32_t w[32];
    if (sums) {
      uint32_t lo[32], hi[32];
      ptx::tmem_ld_32x32b_x32(tcol + c * 64, lo);
      ptx::tmem_ld_32x32b_x32(tcol + c * 64 + 32, hi);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = pack_pair(f * __uint_as_float(lo[2 * i]), f * __uint_as_float(lo[2 * i + 1]), fmt);
        w[16 + i] = pack_pair(f * __uint_as_float(hi[2 * i]), f * __uint_as_float(hi[2 * i + 1]), fmt);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
    }
    if (a.store_granule == 0)
      store_words(w, mapC, col, row0, expert, buf, lane);
    else
      store_words_plain(w, static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(expert) * M + row0) * a.ld_out + col,
                        a.ld_out, M - row0, N - col, a.store_granule, buf, lane);
  }
}

template <int MODE, int PARTS, bool GATHER>
__global__ void __launch_bounds__(expert_threads(PARTS), 1)
    expert_kernel(const __grid_constant__ ExpertMaps maps, const __grid_constant__ ExpertArgs args) {
  const CUtensorMap &mapA = maps.a, &mapB = maps.b, &mapC = maps.c;
  constexpr int STAGES = expert_stages(MODE, PARTS);
  constexpr bool GRADIENT = weight_gradient(MODE);
  static_assert(!GRADIENT || PARTS == 2, "staging of stores");
  constexpr int ACC = 256;
  constexpr uint32_t TMEM_COLS = 512;
  static_assert(expert_smem(MODE, PARTS) <= kSmemLimit, "shared memory per CTA");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sC = smem + STAGES * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(sC + expert_epi_bytes(MODE, PARTS));
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  static_assert((2 * STAGES + 5) * 8 + 8 <= kBarrierBytes, "barrier area");
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(ptx::cluster_ctarank() & 1u);
  const bool leader = cta == 0;
  const int worker = blockIdx.x / 2, workers = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&acc_full[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&acc_empty[b]), 2 * 4 * PARTS);
    }
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&mapA);
    ptx::tma_prefetch_desc(&mapB);
    if (!GRADIENT && !GATHER) {
      ptx::tma_prefetch_desc(&maps.b32);
      ptx::tma_prefetch_desc(&maps.b16);
    }
    if (MODE != EXPERT_DH) ptx::tma_prefetch_desc(&mapC);
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
  const ExpertUnits<MODE> units(args);

  if (warp == 0) {
    // ------------------------------------------------ bulk-tensor producer
    // As few instructions a stage as it takes: they queue behind the epilogues', and
    // with n = 256 a stage's MMAs last 512 cycles.  Lane 0 copies the weight, lanes 1..
    // the tokens' boxes.
    const uint32_t full0 = ptx::smem_u32(&full[0]), empty0 = ptx::smem_u32(&empty[0]);
    const uint32_t full0_leader = ptx::mapa_shared(full0, 0), ring = ptx::smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    ExpertUnit next = units.get(args, worker);
    for (int i = worker; ok && i < units.count; i += workers) {
      const ExpertUnit u = next;
      next = units.get(args, i + workers);
      const int stages = units.stages(args, u);
      const int half = GRADIENT ? kTileM : u.n / 2;  // this CTA's columns
      const uint32_t bytes = 2u * (kSub + static_cast<uint32_t>(half) * 128u);
      // a CTA's columns in as few boxes as add up to them (each costs the copy engine
      // some 20 cycles beside its bytes): lane 1 + b's box
      const int wide = half / 64, b = lane - 1;
      const bool mid = (half & 32) != 0, small = (half & 16) != 0;
      const bool copies_b = GRADIENT ? lane == 1 : GATHER ? 4 * lane < half : lane >= 1 && b < wide + (mid ? 1 : 0) + (small ? 1 : 0);
      const CUtensorMap* box = GRADIENT || b < wide ? &mapB : b == wide && mid ? &maps.b32 : &maps.b16;
      const int box0 = GRADIENT ? 0 : b < wide ? 64 * b : b == wide ? 64 * wide : 64 * wide + 32;
      const int m0 = u.mb * 256 + cta * kTileM;  // 128 of the 256 of M
      const int f0 = u.mb * kTileM + cta * 64;   // UP: 64 features
      const int row = u.row0 + cta * half + box0;
      int4 rows = make_int4(0, 0, 0, 0);
      if (GATHER && copies_b)
        rows = __ldcg(reinterpret_cast<const int4*>(args.rows.token + u.row0 + cta * half + 4 * lane));
      int k0 = 0;  // past the k axis: zeros (gradients: other rows, which no MMA reads)
      for (int it = 0; it < stages; ++it, k0 += kTileK) {
        ok = wait_bounded(empty0 + 8 * stage, phase ^ 1u, ctl, SITE_PRODUCER_EMPTY);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t fb = full0_leader + 8 * stage, sa = ring + stage * kStage, sb = sa + kSub;
        if (lane == 0) {
          if (leader) ptx::mbar_arrive_expect_tx(full0 + 8 * stage, bytes);
          if constexpr (MODE == EXPERT_UP) {
            if (!args.split)
              ptx::tma_load_5d_pair(sa, &mapA, k0, 0, 0, f0 / 16, u.expert, fb);
            else
              for (int q = 0; q < 4; ++q) ptx::tma_load_3d_pair(sa + q * 4096, &mapA, k0, f0 + q * 16, 2 * u.expert, fb);
          } else if constexpr (MODE == EXPERT_DOWN) {
            ptx::tma_load_3d_pair(sa, &mapA, k0, m0, u.expert, fb);
          } else if constexpr (GRADIENT) {
            ptx::tma_load_3d_pair(sa, &mapA, 0, u.row0 + k0, m0 / 64, fb);
          } else if (!args.split) {
            ptx::tma_load_4d_pair(sa, &mapA, 0, k0, m0 / 64, u.expert, fb);
          } else {
            for (int q = 0; q < 2; ++q) ptx::tma_load_3d_pair(sa + q * 8192, &mapA, m0 + q * 64, k0, u.expert, fb);
          }
        }
        if (copies_b) {
          if constexpr (GRADIENT)
            ptx::tma_load_3d_pair(sb, &mapB, 0, u.row0 + k0, u.nb * 4 + cta * 2, fb);
          else if constexpr (GATHER)
            tma_gather4_pair(sb + lane * 512, &mapB, k0, rows, fb);
          else
            ptx::tma_load_3d_pair(sb + box0 * 128, box, k0, row, 0, fb);
        }
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
    // loads in flight land before shared memory is released (see tc_gemm_2sm.cu)
    if (lane == 0) {
      for (uint32_t s = 0; s < STAGES; ++s)
        if (issued > s) {
          const uint32_t par = (issued - s - 1) / STAGES & 1u;  // of the stage's last use
          wait_teardown(ptx::smem_u32(leader ? &full[s] : &empty[s]), par, ctl, SITE_TEARDOWN);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------ MMA issuer (leader CTA only)
    if (leader && lane == 0) {
      const uint32_t ab = args.bf16 ? 1u : 0u;
      const uint32_t fixed = (1u << 4) | (ab << 7) | (ab << 10) | (expert_a_m_major(MODE) ? 1u << 15 : 0u) |
                             (expert_b_n_major(MODE) ? 1u << 16 : 0u) |
                             (static_cast<uint32_t>((2 * kTileM) >> 4) << 24);
      // the first stage's operands; a stage and a step of 16 are constants further
      const uint64_t a_desc = expert_a_m_major(MODE) ? sw128_desc(ptx::smem_u32(smem), 8192, 1024)
                                                     : sw128_desc(ptx::smem_u32(smem), 16, 1024);
      const uint64_t b_desc = expert_b_n_major(MODE) ? sw128_desc(ptx::smem_u32(smem) + kSub, 8192, 1024)
                                                     : sw128_desc(ptx::smem_u32(smem) + kSub, 16, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      ExpertUnit next = units.get(args, worker);
      for (int i = worker; ok && i < units.count; i += workers) {
        const ExpertUnit u = next;
        next = units.get(args, i + workers);
        const int stages = units.stages(args, u);
        const uint32_t idesc = fixed | (static_cast<uint32_t>((GRADIENT ? 256 : u.n) >> 3) << 17);
        for (int lo = 0; ok && lo < stages; lo += args.chunk) {
          if (!wait_bounded(ptx::smem_u32(&acc_empty[acc]), acc_phase ^ 1u, ctl, SITE_MMA_ACC_EMPTY)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * ACC);
          const int end = min(lo + args.chunk, stages);
          for (int it = lo; it < end; ++it) {
            if (!wait_bounded(ptx::smem_u32(&full[stage]), phase, ctl, SITE_MMA_FULL)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after_sync();
            const uint64_t da = a_desc + static_cast<uint64_t>(stage * (kStage >> 4));
            const uint64_t db = b_desc + static_cast<uint64_t>(stage * (kStage >> 4));
            // steps of 16: the expert's rows end at one, what follows is another's
            const int steps = GRADIENT ? min(kTileK / 16, (u.n - it * kTileK) / 16) : kTileK / 16;
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k)
              if (!GRADIENT || k < steps)
                ptx::tc_mma_f16_pair(d_tmem, da + k * ((expert_a_m_major(MODE) ? 2048 : 32) >> 4),
                                     db + k * ((expert_b_n_major(MODE) ? 2048 : 32) >> 4), idesc,
                                     (it != lo || k != 0) ? 1u : 0u);
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
    const int quarter = warp & 3;          // tensor-memory lanes of this warp
    const int part = (warp - 2) / 4;       // its share of the columns
    uint8_t* buf = sC + (warp - 2) * 4096;
    constexpr bool STAGED = !GRADIENT && MODE != EXPERT_DH;
    using Staged = StagedRows<staged_buffers(MODE), staged_bytes(MODE)>;
    Staged staged{sC + part * staged_buffers(MODE) * staged_bytes(MODE), 0, part, quarter};
    const int fmt = args.bf16 ? OUT_BF16 : OUT_F16;
    const bool pairs = (args.F & 1) == 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const auto taken = [&]() {
      ok = warp_wait(ptx::smem_u32(&acc_full[acc]), acc_phase, ctl, SITE_EPI_ACC_FULL);
      ptx::tc_fence_after_sync();
      return tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * ACC);
    };
    const auto given_back = [&]() {
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&acc_empty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    };
    ExpertUnit next = units.get(args, worker);
    for (int i = worker; ok && i < units.count; i += workers) {
      const ExpertUnit u = next;
      const int stages = units.stages(args, u);
      // this warp's blocks of 16 columns: of a weight's gradient 128 neighbours, else every PARTS-th
      constexpr int STEP = GRADIENT ? 1 : PARTS, MOST = 16 / PARTS;
      const int block0 = GRADIENT ? part * MOST : part;
      const int blocks = GRADIENT ? MOST : (u.n / 16 - part + PARTS - 1) / PARTS;
      uint32_t tcol = 0;
      if (!GRADIENT || stages > 0) {
        tcol = taken() + block0 * 16;
        int lo = args.chunk;  // end of the chunk at hand
        if (lo < stages && ok) {
          uint32_t sum[MOST][16];
          first_sums<STEP, MOST>(tcol, sum);
          given_back();
          for (lo += args.chunk;; lo += args.chunk) {
            tcol = taken() + block0 * 16;
            if (!ok) break;
            more_sums<STEP, MOST>(tcol, sum);
            if (lo >= stages) {
              whole_sums<STEP, MOST>(tcol, sum);
              break;
            }
            given_back();
          }
        }
      }
      if constexpr (STAGED) ok = part_agrees(ok, part);
      if (!ok) break;
      next = units.get(args, i + workers);  // under this epilogue; no register is its beside the sums
      float unscale = 1.0f;  // of the expert's fp16 gradients
      if ((GRADIENT || MODE == EXPERT_DX) && args.largest)
        unscale = expert_unscale(__ldcg(args.largest + 2 * u.expert + (MODE == EXPERT_DOUT ? 1 : 0)));
      if constexpr (GRADIENT) {
        const int M = MODE == EXPERT_DIN ? 2 * args.F : args.D, N = MODE == EXPERT_DIN ? args.D : args.F;
        finish_weight(tcol, stages > 0, args, u.expert, u.mb * 256 + cta * kTileM + quarter * 32, M,
                      u.nb * 256 + part * 128, N, unscale, &mapC, buf, lane);
        if (stages > 0) given_back();
      } else {
        const int m0 = MODE == EXPERT_UP ? u.mb * kTileM + cta * 64 + quarter * 16 + (lane & 15)
                                         : u.mb * 256 + cta * kTileM + quarter * 32 + lane;
        // the weight of each of a block's rows, a lane each, a block ahead
        const auto weight_of = [&](int b) {
          const int c = (part + b * PARTS) * 16 + lane;
          return lane < 16 && b < blocks && c < u.valid
                     ? __ldg(args.weights + __ldcg(args.rows.place + u.row0 + c))
                     : 0.0f;
        };
        float ahead = MODE == EXPERT_DH ? weight_of(0) : 0.0f;
        uint32_t most[2] = {0u, 0u};
        constexpr bool JOINED = MODE == EXPERT_DOWN || MODE == EXPERT_DX;
        if (JOINED && args.bf16) {
          // two blocks at a time: their chains of reductions and exchanges run side by side
          const int x0 = u.mb * 256 + cta * kTileM;
#pragma unroll 1
          for (int b = 0; b < blocks; b += 2) {
            const bool both = b + 1 < blocks;
            const int row = u.row0 + (part + b * PARTS) * 16, other = row + PARTS * 16;
            uint32_t v[16], w[16], v_most[16], w_most[16];
            ptx::tmem_ld_32x32b_x16(tcol + b * PARTS * 16, v);
            ptx::tmem_ld_32x32b_x16(tcol + (both ? b + 1 : b) * PARTS * 16, w);
            ptx::tmem_wait_ld();
            row_sizes(v, v_most);
            row_sizes(w, w_most);
            staged.acquire(lane);
            finish_y_half<Staged>(v, v_most, args, m0, row, lane, m0 - x0, true, staged.block(m0 - x0));
            finish_y_half<Staged>(w, w_most, args, m0, other, lane, m0 - x0, both, staged.block(m0 - x0, 1));
            staged.store(&mapC, x0, args.D - x0, row, both ? 2 : 1, other, lane);
          }
        }
#pragma unroll 1
        for (int b = JOINED && args.bf16 ? blocks : 0; b < blocks; ++b) {
          const int c0 = (part + b * PARTS) * 16;
          const int valid = u.valid - c0;
          if constexpr (MODE == EXPERT_DH) {
            const float mine = ahead;
            ahead = weight_of(b + 1);
#pragma unroll
            for (int half = 0; half < 16; half += 8) {
              uint32_t v[8];
              ptx::tmem_ld_32x32b_x8(tcol + b * PARTS * 16 + half, v);
              ptx::tmem_wait_ld();
              const int dot = (u.mb * 2 + cta) * 4 + quarter;
              if (args.v)
                finish_v(v, args, m0, u.row0 + c0 + half, valid - half, lane, mine, half, dot, args.m_blocks * 8, most);
              else if (pairs)
                finish_dh<true>(v, args, m0, u.row0 + c0 + half, valid - half, fmt, lane, mine, half, dot, args.m_blocks * 8);
              else
                finish_dh<false>(v, args, m0, u.row0 + c0 + half, valid - half, fmt, lane, mine, half, dot, args.m_blocks * 8);
            }
          } else {
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(tcol + b * PARTS * 16, v);
            ptx::tmem_wait_ld();
            if constexpr (MODE == EXPERT_UP) {
              const int x0 = u.mb * kTileM + cta * 64;  // the CTA's first feature
              finish_up(v, args, m0, u.row0 + c0, valid, fmt, lane, m0 - x0, staged);
              staged.store(&mapC, x0, min(64, args.F - x0), u.row0 + c0, 1, 0, lane);
            } else {
              finish_y(v, args, m0, u.row0 + c0, valid, unscale);
            }
          }
        }
        given_back();
        if (MODE == EXPERT_DH && args.v) {  // a maximum is the same in whatever order
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t all = __reduce_max_sync(0xffffffffu, most[i]);
            if (lane == 0 && all) atomicMax(args.largest + 2 * u.expert + i, all);
          }
        }
      }
    }
    if ((GRADIENT || STAGED) && lane == 0) ptx::bulk_wait_group_read<0>();
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

template <int MODE, int PARTS, bool GATHER = false>
cudaError_t launch_expert(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  return launch_pairs(expert_kernel<MODE, PARTS, GATHER>, expert_smem(MODE, PARTS), expert_threads(PARTS), done_mask, pairs,
                      stream, maps, args);
}

}  // namespace
}  // namespace tgemm
