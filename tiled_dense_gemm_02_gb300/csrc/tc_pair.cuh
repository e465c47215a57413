// What the CTA-pair products of the losses and of the experts share: their ring's
// stage, 16-bit results on their way to memory, and the launch.
#pragma once

#include <atomic>

#include "tc_common.cuh"

namespace tgemm {
namespace {

constexpr int kSub = kTileM * kTileK * 2;        // 16 KB: one CTA's share of A or B in one stage
constexpr int kStage = 2 * kSub;

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

}  // namespace
}  // namespace tgemm
