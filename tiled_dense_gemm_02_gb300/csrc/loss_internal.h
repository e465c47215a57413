// Internal interfaces of the vocabulary-head losses (loss_api.cu, loss_gemm.cu,
// loss_rows.cu) and the services of api.cu that they use.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tgemm_internal.h"

namespace tgemm {

// ---------------------------------------------------- services of api.cu
// SMs, resident CTA pairs and status word of the current device; a status code.
int host_device(int* sms, int* pairs, unsigned int** status);
// Records a failed CUDA call's text and returns TGEMM_ERR_LAUNCH.
int host_cuda_fail(cudaError_t e, const char* what);
// Cached tensor maps, 128-byte swizzle, zero fill (after host_device).
// type: 0 bf16, 1 f16, 2 f32.
int host_map_2d(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t pitch_bytes,
                uint32_t box_cols, uint32_t box_rows);
int host_map_3d(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t depth,
                int64_t pitch_bytes, int64_t depth_bytes, uint32_t box_cols, uint32_t box_rows);
// fp32 product C = A . B + beta C on the CUDA cores.
int host_gemm_f32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B, int64_t ldb, float* C,
                  int64_t ldc, float beta, cudaStream_t stream);
// Adds tensor-core launches to the host counters.
void host_count_launches(int n);
bool host_ranges_overlap(uint64_t a0, uint64_t a1, uint64_t b0, uint64_t b1);
int host_granule(const void* p, int64_t ld, int es);

// --------------------------------------------------- rows that count
// What the row kernels leave for the products, all in the workspace.  Row r of
// the gathered matrix (r < *count) is row source[r] of H; place[t] is its
// inverse (-1: row t does not count).  Row t's targets are ids[t*K .. t*K+K),
// ascending, with masses q; unused places come last with id INT_MAX.
struct HeadRows {
  int* count;         // rows that count
  float* factor;      // what the gradient products' sums are multiplied with
  int* source;        // T
  int* place;         // T
  int* ids;           // T x K
  float* q;           // T x K
  float* own;         // T: sum q log q (distillation), else null
  unsigned char* flags;  // T (distillation), else null
  float4* coef;       // T, gathered: {c_p, c_q, lse * log2(e), lse} (backward), else null
  void* h;            // gathered rows, pitch ldh elements
  int64_t ldh;
};

constexpr unsigned char kRowIgnored = 0, kRowCounts = 1, kRowBad = 2;
// Gathered rows are zero-filled up to a multiple of this (and at least one such block), capped at T.
constexpr int kRowBlock = 256;

struct GatherArgs {
  int T, V, D, K;
  int es;                    // bytes of an element of H
  const void* H;
  int64_t ldh;
  int granule;               // alignment of H's rows (16, 8, 4 or 2 bytes)
  const int64_t* targets;    // cross entropy, else null
  int64_t ignore_index;
  float smoothing, z_loss, scale;
  float range;               // power of two that 16-bit gradients are scaled with (0: fp32, no normalisation)
  int zero_rows;             // 1: zero every gathered row past the count, 0: up to the next block
  const float* lse;          // backward: the forward call's, else null
  const float* grad;         // backward
  float* loss_out;           // forward: rows that do not count are written here
  float* lse_out;
  HeadRows rows;
};
cudaError_t launch_distill_lists(const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits, int T,
                                 int V, int K, float scale, const HeadRows& rows, cudaStream_t stream);
cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream);

// Row statistics of `tiles` column tiles: ms[i * T + r] = {max, sum of
// 2^(y - max)} of y = z log2(e) over tile i, dot[i * T + r] = its share of
// sum q z / scale.
cudaError_t launch_combine(const float2* ms, const float* dot, int tiles, int T, float scale, float z_loss,
                           const HeadRows& rows, float* loss, float* lse, cudaStream_t stream);
// dH row t = factor * sum over splits of acc[s][place[t]], or 0.
cudaError_t launch_finish_dh(const float* acc, int64_t ld_acc, int64_t split_stride, int splits, int T, int D,
                             const HeadRows& rows, int type, void* dH, int64_t lddh, cudaStream_t stream);
// fp32 path: statistics of one piece of logits Z [T x cols], and their
// gradient in place.
cudaError_t launch_stats_f32(const float* Z, int64_t ldz, int cols, int col0, int T, int K, float k2, float flat,
                             const HeadRows& rows, float2* ms, float* dot, cudaStream_t stream);
cudaError_t launch_dz_f32(float* Z, int64_t ldz, int cols, int col0, int T, int K, float scale, float flat,
                          const HeadRows& rows, cudaStream_t stream);

// ------------------------------------------------------- pair products
enum HeadMode : int {
  HEAD_STATS = 0,  // logits tile -> row statistics
  HEAD_DZ = 1,     // logits tile -> gradient of the logits (16-bit)
  HEAD_DH = 2,     // dz . W      -> fp32 sums
  HEAD_DW = 3      // dz^T . H    -> dW (16-bit)
};

struct HeadArgs {
  const int* count;
  int T, V, K;
  int cols;       // columns of this piece (logits), or their number rounded up to 64-deep stages' extent (DH: K)
  int col0;       // vocabulary entry of the piece's column 0
  int b_row0;     // STATS, DZ: row of the weight map for column 0; DH: the same along K
  int D;
  int k_blocks;   // 64-deep stages (DW: from the count)
  int splits, k_per_split;  // DH
  int reduce;     // DH: add to the sums instead of storing them
  int group_m;
  int bf16;
  float k2;       // scale * log2(e)
  float flat;     // eps / V (cross entropy), else 0
  const int* source;
  const int* ids;
  const float* q;
  float2* ms;     // STATS
  float* dot;
  int tile0;      // STATS: index of the piece's first column tile
  const float4* coef;     // DZ
  const float* factor;    // DW
  void* out;              // DW
  int64_t ld_out;
  int store_granule;      // DW: 0 bulk-tensor stores, else the granule of per-thread stores
  int out_row0;           // DW: row of dW for the piece's column 0
  unsigned long long timeout_ns;
  unsigned int* status;
};

// Output tile of every mode: 256 x 256 per CTA pair.
constexpr int kHeadTile = 256;
cudaError_t launch_head(int mode, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                        const HeadArgs& args, int pairs, cudaStream_t stream);

}  // namespace tgemm
