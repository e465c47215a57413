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
// fp32 operands come as three bf16 planes (loss_rows.cu), and a stage of the k
// axis is then six stages, one per pair of planes, the small terms first: the
// last sixth alone adds to a sum of full size, so the adder's truncation is
// that of a 16-bit product.  DH and DW, whose k axes are long, move their sums
// out of tensor memory every `chunk` stages and add them in fp32 with rounding
// to nearest, each element by the one thread that owns it.
//
// with k2 = scale log2(e), so that one fused multiply-add and one 2^x serve
// each logit.  H and W are read K-major (their rows are the k axis) by STATS
// and DZ; W as the N-major B of DH; dz as the M-major A and H as the N-major B
// of DW: no operand is ever transposed in memory.
//
// Roles (both CTAs unless noted):
//   warp 0      bulk-tensor producer of this CTA's 128 rows of A and 128
//               columns of B; completion on the leader CTA's full barrier
//   warp 1      tensor-memory allocation; MMA issue by one thread of the leader
//   warps 2..   epilogue of this CTA's 128 rows, one row per thread: four warps
//               for STATS; eight for the gradients, half of the columns each,
//               since their stores can outlast a short k axis
//
// The number of gathered rows is known on the device only (rows that do not
// count are not gathered), so every role derives the tile list from it.  Every
// wait is bounded (tc_common.cuh).
#include <atomic>
#include <climits>

#include "loss_internal.h"
#include "tc_common.cuh"

namespace tgemm {
namespace {

constexpr int kSub = kTileM * kTileK * 2;        // 16 KB: one CTA's share of A or B in one stage
constexpr int kStage = 2 * kSub;
// Warps per quarter of the rows in the epilogue, each with 4 KB to stage stores.
constexpr int head_halves(int mode) { return mode == HEAD_STATS ? 1 : 2; }
constexpr int head_threads(int mode) { return 32 * (2 + 4 * head_halves(mode)); }
constexpr int head_epi_bytes(int mode) { return mode == HEAD_STATS ? 0 : 4 * head_halves(mode) * 4096; }
constexpr int head_stages(int mode) {
  return (kSmemLimit - 1024 - head_epi_bytes(mode) - kBarrierBytes) / kStage;
}
constexpr int head_smem(int mode) {
  return 1024 + head_stages(mode) * kStage + head_epi_bytes(mode) + kBarrierBytes;
}
constexpr bool a_m_major(int mode) { return mode == HEAD_DW; }
constexpr bool b_n_major(int mode) { return mode == HEAD_DH || mode == HEAD_DW; }

// Pairs of planes in the order they are summed: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0).
constexpr int plane_terms(int planes) { return planes == 1 ? 1 : 6; }
__device__ __forceinline__ int plane_a(int term) { return (0x001102 >> (4 * term)) & 0xF; }
__device__ __forceinline__ int plane_b(int term) { return (0x010120 >> (4 * term)) & 0xF; }

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

// The tile list of a launch, derived from the gathered row count.
struct Tiles {
  int m, n, units, k_blocks;
};

template <int MODE>
__device__ __forceinline__ Tiles head_tiles(const HeadArgs& a, int rows) {
  Tiles t;
  t.m = ((MODE == HEAD_DW ? a.cols : rows) + kHeadTile - 1) / kHeadTile;
  t.n = ((MODE == HEAD_DH || MODE == HEAD_DW ? a.D : a.cols) + kHeadTile - 1) / kHeadTile;
  t.k_blocks = MODE == HEAD_DW ? (rows + kTileK - 1) / kTileK : a.k_blocks;
  t.units = t.m * t.n * (MODE == HEAD_DH ? a.splits : 1);
  return t;
}

struct HeadUnit {
  int mb, nb, split, lo, hi;
};

// Unit -> tile and k-stage range: groups of group_m block-rows are walked
// column by column (as the plain product does), split after split.
template <int MODE>
__device__ __forceinline__ HeadUnit head_unit(const HeadArgs& a, const Tiles& t, int u) {
  HeadUnit w;
  const int per = t.m * t.n;
  w.split = MODE == HEAD_DH ? u / per : 0;
  const int i = MODE == HEAD_DH ? u - w.split * per : u;
  const int per_group = a.group_m * t.n;
  const int g = i / per_group;
  const int first = g * a.group_m;
  const int gsz = min(t.m - first, a.group_m);
  const int r = i - g * per_group;
  w.mb = first + r % gsz;
  w.nb = r / gsz;
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
  __device__ __forceinline__ void start(const HeadArgs& a, int row, int n, int first) {
    K = pos = 0;
    next = INT_MAX;
    ids = nullptr;
    q = nullptr;
    one = a.mass;
    if (row >= n) return;
    const int t = a.source ? a.source[row] : row;
    if (a.targets) {
      const int64_t y = a.targets[t];
      if (y >= first && y < a.V) next = static_cast<int>(y);
      return;
    }
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

// Statistics of this thread's row over the tile's columns.
__device__ __forceinline__ void epilogue_stats(uint32_t tbase, int row, int n, int nb, const HeadArgs& a) {
  const int first = a.col0 + nb * kHeadTile;  // vocabulary entry of the tile's first column
  const int width = a.cols - nb * kHeadTile;
  Walk walk;
  walk.start(a, row, n, first);
  float m = -INFINITY, s = 0.0f, dot = 0.0f, zs = 0.0f;
#pragma unroll 1
  for (int c = 0; c < kHeadTile / 32; ++c) {
    const int limit = width - c * 32;
    if (limit <= 0) break;
    uint32_t raw[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, raw);
    ptx::tmem_wait_ld();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
    if (limit < 32) {  // columns past the piece are no entries
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = i < limit ? v[i] : -INFINITY;
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
    const float m_new = fmaxf(m, top);
    const float ref = m_new == -INFINITY ? 0.0f : m_new;  // nothing but -inf so far: every term is 0
    const float off = -ref * a.k2;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i) part[i & 3] += exp2_fast(fmaf(v[i], a.k2, off));
    s = fmaf(s, exp2_fast((m - ref) * a.k2), (part[0] + part[1]) + (part[2] + part[3]));
    m = m_new;
    if (a.flat != 0.0f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) zs += i < limit ? v[i] : 0.0f;
    }
    const int base = first + c * 32;
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
  if (row < n) {
    const int64_t at = static_cast<int64_t>(a.tile0 + nb) * a.T + row;
    a.ms[at] = make_float2(m * a.k2, s);
    a.dot[at] = fmaf(a.flat, zs, dot);
  }
}

// 32 logits of a row -> their gradient.
__device__ __forceinline__ void gradient_chunk(uint32_t (&raw)[32], int base, int limit, const float4& k,
                                               const HeadArgs& a, Walk& walk) {
  const float flat = k.y * a.flat;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float p = exp2_fast(fmaf(__uint_as_float(raw[i]), a.k2, -k.z));
    raw[i] = __float_as_uint(fmaf(k.x, p, -flat));
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
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    if (r >= rows) break;
    uint16_t* row = dst + r * ld;
    if (granule >= 4) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(buf + sw128_offset(r, lane * 4));
      if (2 * lane + 2 <= cols)
        reinterpret_cast<uint32_t*>(row)[lane] = v;
      else if (2 * lane < cols)
        row[2 * lane] = static_cast<uint16_t>(v & 0xFFFFu);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        if (c < cols) row[c] = *reinterpret_cast<const uint16_t*>(buf + sw128_offset(r, c * 2));
      }
    }
  }
  __syncwarp();
}

template <int PLANES>
__device__ __forceinline__ void epilogue_dz(uint32_t tbase, int row0, int n, int nb, int half, const HeadArgs& a,
                                            const CUtensorMap* mapC, uint8_t* buf, int lane) {
  if (row0 >= a.T) return;
  const int c0 = half * (kHeadTile / 128), c1 = c0 + kHeadTile / 128;
  const int row = row0 + lane;
  const int first = a.col0 + nb * kHeadTile;
  const int width = a.cols - nb * kHeadTile;
  Walk walk;
  walk.start(a, row, n, first + c0 * 64);
  const float4 k = row < n ? a.coef[row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int fmt = a.bf16 ? OUT_BF16 : OUT_F16;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    if (c * 64 >= width) break;
    uint32_t lo[32], hi[32], w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 64, lo);
    ptx::tmem_ld_32x32b_x32(tbase + c * 64 + 32, hi);
    ptx::tmem_wait_ld();
    gradient_chunk(lo, first + c * 64, width - c * 64, k, a, walk);
    gradient_chunk(hi, first + c * 64 + 32, width - c * 64 - 32, k, a, walk);
    if (row >= n) {  // rows past the count: zeros, which the products read
#pragma unroll
      for (int i = 0; i < 32; ++i) lo[i] = hi[i] = 0u;
    }
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        uint32_t* v = i < 16 ? &lo[2 * i] : &hi[2 * i - 32];
        const float x = __uint_as_float(v[0]), y = __uint_as_float(v[1]);
        w[i] = pack_pair(x, y, PLANES == 1 ? fmt : OUT_BF16);
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

// 32 fp32 values of a row: stored, or added to what is there.  The same thread
// writes an element in every chunk, so the order of the additions is fixed.
__device__ __forceinline__ void store_row_f32(float* dst, const float (&v)[32], int valid, bool vec, bool add) {
  if (vec && valid >= 32) {
    float4* d = reinterpret_cast<float4*>(dst);
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = add ? __ldcg(d + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __stcg(d + i, make_float4(o[i].x + v[4 * i], o[i].y + v[4 * i + 1], o[i].z + v[4 * i + 2], o[i].w + v[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < valid) __stcg(dst + i, add ? __ldcg(dst + i) + v[i] : v[i]);
  }
}

// fp32 DH and DW: one chunk's sums of this thread's row, times f.
__device__ __forceinline__ void epilogue_f32(uint32_t tbase, float* row, bool valid_row, int nb, int half, int cols,
                                             float f, bool vec, bool add) {
  const int c0 = half * (kHeadTile / 64), c1 = c0 + kHeadTile / 64;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int col = nb * kHeadTile + c * 32;
    if (col >= cols) break;
    uint32_t w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, w);
    ptx::tmem_wait_ld();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = f * __uint_as_float(w[i]);
    if (valid_row) store_row_f32(row + col, v, cols - col, vec, add);
  }
}

__device__ __forceinline__ void epilogue_dh(uint32_t tbase, int row0, const HeadUnit& u, int half, const HeadArgs& a,
                                            const CUtensorMap* mapC, uint8_t* buf, int lane) {
  if (row0 >= a.T) return;
  const int c0 = half * (kHeadTile / 64), c1 = c0 + kHeadTile / 64;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const int col = u.nb * kHeadTile + c * 32;
    if (col >= a.D) break;
    uint32_t w[32];
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, w);
    ptx::tmem_wait_ld();
    stage_row(buf, lane, w);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (a.reduce)
        tma_reduce_add_3d(mapC, col, row0, u.split, ptx::smem_u32(buf));
      else
        ptx::tma_store_3d(mapC, col, row0, u.split, ptx::smem_u32(buf));
      ptx::bulk_commit_group();
    }
  }
}

__device__ __forceinline__ void epilogue_dw(uint32_t tbase, int row0, int nb, int half, const HeadArgs& a,
                                            const CUtensorMap* mapC, uint8_t* buf, int lane) {
  if (row0 >= a.cols) return;
  const float f = *a.factor;
  const int fmt = a.bf16 ? OUT_BF16 : OUT_F16;
  const int c0 = half * (kHeadTile / 128), c1 = c0 + kHeadTile / 128;
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

template <int MODE, int PLANES>
__global__ void __launch_bounds__(head_threads(MODE), 1)
    head_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ CUtensorMap mapC, const HeadArgs args) {
  constexpr int STAGES = head_stages(MODE);
  constexpr int TERMS = plane_terms(PLANES);
  constexpr int ACC = 256;
  constexpr uint32_t TMEM_COLS = 512;
  static_assert(head_smem(MODE) <= kSmemLimit, "shared memory per CTA");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sC = smem + STAGES * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(sC + head_epi_bytes(MODE));
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  static_assert((2 * STAGES + 5) * 8 + 8 <= kBarrierBytes, "barrier area");
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(ptx::cluster_ctarank() & 1u);  // which 128 rows of the pair's tile
  const bool leader = cta == 0;
  const int worker = blockIdx.x / 2;
  const int workers = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&acc_full[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&acc_empty[b]), 2 * 4 * head_halves(MODE));
    }
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
  // stages summed in tensor memory at a time: all of a unit's, or a chunk
  const int chunk = PLANES > 1 && (MODE == HEAD_DH || MODE == HEAD_DW) ? args.chunk : INT_MAX / 2;

  if (warp == 0) {
    // ------------------------------------------------ bulk-tensor producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, last_parity = 0;
      bool ok = true;
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
            const int term = PLANES == 1 ? 0 : it / span;
            const int k0 = (lo + it - term * span) * kTileK;  // stages past the k axis load zeros
            const int pa = PLANES == 1 ? 0 : plane_a(term), pb = PLANES == 1 ? 0 : plane_b(term);
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
    const int half = (warp - 2) / 4;           // its half of the tile's columns
    uint8_t* buf = sC + (warp - 2) * 4096;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = worker; ok && i < tiles.units; i += workers) {
      const HeadUnit u = head_unit<MODE>(args, tiles, i);
      const int row0 = u.mb * kHeadTile + cta * kTileM + quarter * 32;
      for (int lo = u.lo; lo < u.hi; lo += chunk) {
        if (!warp_wait(ptx::smem_u32(&acc_full[acc]), acc_phase, ctl, SITE_EPI_ACC_FULL)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after_sync();
        const uint32_t tbase =
            tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * ACC);
        if constexpr (MODE == HEAD_STATS) {
          if (row0 < n) epilogue_stats(tbase, row0 + lane, n, u.nb, args);
        } else if constexpr (MODE == HEAD_DZ) {
          epilogue_dz<PLANES>(tbase, row0, n, u.nb, half, args, &mapC, buf, lane);
        } else if constexpr (PLANES > 1) {
          // a chunk's sum of the full-size terms took 4 steps a stage
          const float put_back = 1.0f + kStepLoss * static_cast<float>(4 * min(chunk, u.hi - lo));
          const int row = row0 + lane;
          float* out = static_cast<float*>(args.out);
          if constexpr (MODE == HEAD_DH) {
            if (row0 < n)
              epilogue_f32(tbase, out + u.split * args.split_stride + static_cast<int64_t>(row) * args.ld_out, row < n,
                           u.nb, half, args.D, put_back, true, args.reduce || lo > u.lo);
          } else if (row0 < args.cols) {
            epilogue_f32(tbase, out + static_cast<int64_t>(args.out_row0 + row) * args.ld_out, row < args.cols, u.nb,
                         half, args.D, put_back * *args.factor, args.store_granule == 16, lo > u.lo);
          }
        } else if constexpr (MODE == HEAD_DH) {
          epilogue_dh(tbase, row0, u, half, args, &mapC, buf, lane);
        } else {
          epilogue_dw(tbase, row0, u.nb, half, args, &mapC, buf, lane);
        }
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&acc_empty[acc]), 0));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
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

template <int MODE, int PLANES>
cudaError_t launch(const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap& mC, const HeadArgs& args,
                   int pairs, cudaStream_t stream) {
  constexpr int smem = head_smem(MODE);
  auto kernel = head_kernel<MODE, PLANES>;
  static std::atomic<uint64_t> done_mask{0};
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
  cfg.blockDim = dim3(head_threads(MODE), 1, 1);
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
  return cudaLaunchKernelEx(&cfg, kernel, mA, mB, mC, args);
}

}  // namespace

cudaError_t launch_head(int mode, int planes, const CUtensorMap& mapA, const CUtensorMap& mapB,
                        const CUtensorMap& mapC, const HeadArgs& args, int pairs, cudaStream_t stream) {
#define TGEMM_HEAD(MODE)                                                                  \
  case MODE:                                                                              \
    return planes == 1 ? launch<MODE, 1>(mapA, mapB, mapC, args, pairs, stream)           \
                       : launch<MODE, kPlanes>(mapA, mapB, mapC, args, pairs, stream)
  switch (mode) {
    TGEMM_HEAD(HEAD_STATS);
    TGEMM_HEAD(HEAD_DZ);
    TGEMM_HEAD(HEAD_DH);
    TGEMM_HEAD(HEAD_DW);
    default: return cudaErrorInvalidValue;
  }
#undef TGEMM_HEAD
}

}  // namespace tgemm
