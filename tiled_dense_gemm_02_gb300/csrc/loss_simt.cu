// Row statistics of 9 to 32 fp32 rows on the CUDA cores (what STATS of
// loss_gemm.cuh does with planes of H and W and 256-row tiles, mostly empty here).
//
// A block computes a tile of TE entries x RT rows; a thread eight entries x four
// rows, k in pairs, so that a fused multiply-add of two serves each: 12 loads of 16
// bytes from shared memory for 128 multiply-adds.  32-column pieces of W and H
// arrive by asynchronous copies, a stage ahead; W is read once, as it lies, in
// fp32, and H by every block.  The finished tile goes to shared memory, where a
// warp takes a row: its maximum, its sum and its targets.
//
// Bound by the latency of shared memory at 8 to 16 warps an SM: 0.48 of the fp32
// rate with 32 rows, 3.5 TB/s of W with 16.  Against passes of eight rows over W
// (loss_few.cuh) and the tensor cores, 65536 x 4096: 16 rows 305, 416 and 1028 us;
// 32 rows 479, 828 and 1028 us.  32 rows of 131072 x 2048: 413, 823 and 965 us.
// Tiles of 64 rows for 33 to 64 took 850 us (1290 us unaligned, against 1150 of the
// tensor cores) and 66 us against 33 for 8192 x 512: not kept.  Nor was a
// gradient epilogue: a backward call needs W's planes for dH in any case, and dz
// from them takes no longer (2322 us against 1791 for 32 rows in all).
#include "loss_few.cuh"

namespace tgemm {
namespace {

constexpr int kSimtK = 32, kSimtPitch = kSimtK + 4;  // pitch: eight rows, eight banks' worth

template <int RT>
struct SimtTile {
  static constexpr int R = 4;                           // rows a thread
  static constexpr int RG = RT / R;                     // groups of rows
  static constexpr int EG = RT == 16 ? 32 : 16;         // groups of entries
  static constexpr int THREADS = RG * EG;
  static constexpr int TE = 8 * EG;                     // entries a block
  static constexpr int STAGE = (TE + RT) * kSimtPitch;  // floats
  static constexpr int BLOCKS = RT == 16 ? 2 : 4;       // an SM
  static constexpr int STAGES = 2;
  static constexpr int ZP = TE + 4;
  static constexpr int SMEM = (STAGES * STAGE > RT * ZP ? STAGES * STAGE : RT * ZP) * 4;
};

// Four elements of a row from column c on; past column D, and where not `on`, zeros.
template <bool VEC>
__device__ __forceinline__ void copy_piece(float* dst, const float* row, int c, int D, bool on) {
  const uint32_t to = ptx::smem_u32(dst);
  if constexpr (VEC) {
    const int n = on ? min(max(D - c, 0), 4) : 0;
    ptx::cp_async<16>(to, row + (n ? c : 0), static_cast<uint32_t>(4 * n));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = on && c + i < D;
      ptx::cp_async<4>(to + 4 * i, row + (in ? c + i : 0), in ? 4u : 0u);
    }
  }
}

template <int RT, bool VEC>
__global__ void __launch_bounds__(SimtTile<RT>::THREADS, SimtTile<RT>::BLOCKS) simt_stats_kernel(const HeadSimtArgs s) {
  using Tile = SimtTile<RT>;
  constexpr int R = Tile::R, RG = Tile::RG, EG = Tile::EG, TE = Tile::TE, STAGES = Tile::STAGES, ZP = Tile::ZP;
  constexpr int STEP = Tile::THREADS / 8;  // rows of a stage copied at a time
  extern __shared__ __align__(16) float s_mem[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const HeadArgs& a = s.head;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = blockIdx.x * TE;  // in the piece
  const int limit = min(TE, a.cols - v0);

  // this thread's share of a stage: column piece tid % 8 of rows tid / 8 + STEP i
  const int piece = (tid & 7) * 4, prow = tid >> 3;
  const float* h_row[RT / STEP];
#pragma unroll
  for (int i = 0; i < RT / STEP; ++i) {
    const int r = prow + STEP * i;
    h_row[i] = r < a.T ? s.H + r * s.ldh : nullptr;
  }
  const int chunks = (a.D + kSimtK - 1) / kSimtK;
  const auto load = [&](int c) {
    if (c < chunks) {
      float* dst = s_mem + (c % STAGES) * Tile::STAGE + prow * kSimtPitch + piece;
      const int col = c * kSimtK + piece;
#pragma unroll
      for (int i = 0; i < TE / STEP; ++i) {
        const int v = v0 + min(prow + STEP * i, limit - 1);  // past the piece: its last entry again
        copy_piece<VEC>(dst + STEP * i * kSimtPitch, s.W + static_cast<int64_t>(v) * s.ldw, col, a.D, true);
      }
#pragma unroll
      for (int i = 0; i < RT / STEP; ++i)
        copy_piece<VEC>(dst + (TE + STEP * i) * kSimtPitch, h_row[i] ? h_row[i] : s.H, col, a.D, h_row[i] != nullptr);
    }
    ptx::cp_async_commit();
  };

  const int eg = tid % EG, rg = tid / EG;  // entries eg + EG i, rows rg + RG j
  float2 acc[8][R];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < STAGES - 1; ++c) load(c);
  for (int c = 0; c < chunks; ++c) {
    ptx::cp_async_wait<STAGES - 2>();
    __syncthreads();  // stage c has come, and all are done with stage c - 1
    load(c + STAGES - 1);
    const float* w = s_mem + (c % STAGES) * Tile::STAGE + eg * kSimtPitch;
    const float* h = s_mem + (c % STAGES) * Tile::STAGE + (TE + rg) * kSimtPitch;
#pragma unroll 2
    for (int k = 0; k < kSimtK; k += 4) {
      float4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const float4*>(w + EG * i * kSimtPitch + k);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(h + RG * j * kSimtPitch + k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y.x, y.y), acc[i][j]);
          acc[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y.z, y.w), acc[i][j]);
        }
      }
    }
  }
  ptx::cp_async_wait<0>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) s_mem[(rg + RG * j) * ZP + eg + EG * i] = acc[i][j].x + acc[i][j].y;
  __syncthreads();

  const int first = a.col0 + v0;
  for (int r = warp; r < min(RT, a.T); r += Tile::THREADS / 32) {
    float* z = s_mem + r * ZP;
    const int64_t list = static_cast<int64_t>(r) * a.K;
    const int64_t y = a.target ? a.target[r] : -1;
    float m = -INFINITY, sum = 0.0f, zs = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < TE / 32; ++i)
      if (lane + 32 * i < limit) m = fmaxf(m, z[lane + 32 * i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float off = m == -INFINITY ? 0.0f : -m * a.k2;
#pragma unroll
    for (int i = 0; i < TE / 32; ++i)
      if (lane + 32 * i < limit) {
        sum += exp2f(fmaf(z[lane + 32 * i], a.k2, off));
        zs += z[lane + 32 * i];
      }
    if (a.target) {
      if (lane == 0 && y >= first && y < first + limit) dot = a.mass * z[y - first];
    } else {
      for (int p = lane; p < a.K; p += 32) {
        const int id = a.ids[list + p];
        if (id >= first && id < first + limit) dot = fmaf(a.q[list + p], z[id - first], dot);
      }
    }
    if (a.flat != 0.0f) dot = fmaf(a.flat, zs, dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (lane == 0) {
      const int64_t at = (static_cast<int64_t>(a.tile0) + blockIdx.x) * a.T + r;
      a.ms[at] = make_float2(m * a.k2, sum);
      a.dot[at] = dot;
    }
  }
}

template <int RT, bool VEC>
cudaError_t launch_tile(const HeadSimtArgs& s, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  using Tile = SimtTile<RT>;
  static_assert(Tile::SMEM <= kFewSmem && Tile::BLOCKS * (Tile::SMEM + 1024) <= 228 * 1024, "blocks an SM");
  return launch_few_kernel(simt_stats_kernel<RT, VEC>, s, dim3((s.head.cols + Tile::TE - 1) / Tile::TE),
                           Tile::THREADS, Tile::SMEM, done_mask, stream);
}

template <bool VEC>
cudaError_t launch_rows(const HeadSimtArgs& s, cudaStream_t stream) {
  if (s.head.T <= 16) return launch_tile<16, VEC>(s, stream);
  return launch_tile<32, VEC>(s, stream);
}

}  // namespace

int head_simt_tile(int64_t T) { return T <= 16 ? SimtTile<16>::TE : SimtTile<32>::TE; }

cudaError_t launch_head_simt(const HeadSimtArgs& s, bool aligned, cudaStream_t stream) {
  return aligned ? launch_rows<true>(s, stream) : launch_rows<false>(s, stream);
}

}  // namespace tgemm
