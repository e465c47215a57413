// Internal interfaces of the vocabulary-head losses (loss_api.cu, loss_gemm.cuh,
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
// Cached 3-D tensor map, 128-byte swizzle, zero fill (after host_device).
// type: 0 bf16, 1 f16, 2 f32.
int host_map_3d(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t depth,
                int64_t pitch_bytes, int64_t depth_bytes, uint32_t box_cols, uint32_t box_rows);
// Adds tensor-core launches to the host counters.
void host_count_launches(int n);
bool host_ranges_overlap(uint64_t a0, uint64_t a1, uint64_t b0, uint64_t b1);
int host_granule(const void* p, int64_t ld, int es);

// --------------------------------------------------- rows that count
// What the row kernels leave for the products, all in the workspace.  Row r of
// the gathered matrix (r < *count) is row source[r] of H; place[t] is its
// inverse (-1: row t does not count).  Distillation: row t's list is ids[t*K ..
// t*K+K), ascending, with masses q; unused places come last with id INT_MAX.
// Forward calls that read H in place have no gathered rows: count, source and
// place are then null, and row r is row r of H.
struct HeadRows {
  int* count;         // rows that count
  float* factor;      // what the gradient products' sums are multiplied with
  int* source;        // T
  int* place;         // T
  int64_t* target;    // T (cross entropy): the gathered rows' targets
  int* ids;           // T x K (distillation)
  float* q;           // T x K
  float* own;         // T: sum q log q (distillation), else null
  unsigned char* flags;  // T (distillation), else null
  float4* coef;       // T, gathered: {c_p, c_q, lse * log2(e), the row's own scale} (backward), else null
  int* spread;        // whether rows have scales of their own (fp16, backward), else null
  void* h;            // gathered rows, pitch ldh 16-bit elements
  int64_t ldh;
  int64_t plane;      // elements between the planes of fp32 rows
};

// fp32 operands are split into three bf16 planes, x = hi + mid + lo: 3 x 8
// significant bits hold all 24 of x.  A product of two of them is then six
// plane products (those of relative size 2^-24 and below are left out).
constexpr int kPlanes = 3;

// fp16 gradients of the logits: dW's product sums over the rows and needs one
// scale for all of them, by which a row of small weight falls among fp16's
// subnormal numbers: at 2^-20 of the largest gradient, a probability of 2^-17 has
// three bits left.  The bits that dW loses are below its largest terms' last; dH's
// rows, each a sum of its own, would lose them whole.  Where a row that counts is
// below this part of the largest, DZ stores dz twice, the second time with each row
// scaled to the top of the range, for DH, and the last step of dH takes the row's
// scale back.  At 2^-6 and above probabilities of 2^-22 are still normal numbers.
constexpr float kSpread = 1.0f / 64;

constexpr unsigned char kRowIgnored = 0, kRowCounts = 1, kRowBad = 2;
// Gathered rows are zero-filled up to a multiple of this (and at least one such block), capped at T.
constexpr int kRowBlock = 256;

// Whether row t counts, from its target (targets not null) or its list's flag.
struct RowRule {
  const int64_t* targets;    // cross entropy, else null
  int64_t ignore_index;
  const unsigned char* flags;
  int V;
};

struct GatherArgs {
  int T, D;
  int es;                    // bytes of an element of H
  const void* H;
  int64_t ldh;
  int granule;               // alignment of H's rows (16, 8, 4 or 2 bytes)
  RowRule rule;
  float z_loss, scale;
  float range;               // power of two that the stored gradients are scaled with
  const float* lse;          // backward: the forward call's, else null
  const float* grad;         // backward
  float* loss_out;           // forward: rows that do not count are written here
  float* lse_out;
  HeadRows rows;
};
cudaError_t launch_distill_lists(const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits, int T,
                                 int V, int K, float scale, const HeadRows& rows, cudaStream_t stream);
cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream);

// Row statistics of `tiles` parts of the columns: ms[i * T + r] = {max, sum of
// 2^(y - max)} of y = z log2(e) over part i, dot[i * T + r] = its share of
// sum q z / scale.  Without gathered rows it also writes those that do not count.
cudaError_t launch_combine(const float2* ms, const float* dot, int tiles, int T, float scale, float z_loss,
                           const HeadRows& rows, const RowRule& rule, float* loss, float* lse, cudaStream_t stream);
// dH row t = factor / its own scale * sum over splits of acc[s][place[t]], or 0.  Without
// gathered rows: of acc[s][t], factor 1.
cudaError_t launch_finish_dh(const float* acc, int64_t ld_acc, int64_t split_stride, int splits, int T, int D,
                             const HeadRows& rows, const RowRule& rule, int type, void* dH, int64_t lddh,
                             cudaStream_t stream);
// The three planes of an fp32 matrix (vec: 16-byte aligned rows); each plane
// has pitch ld_out, a multiple of 8.
cudaError_t launch_split(const float* W, int64_t ldw, void* out, int64_t ld_out, int64_t plane, int rows, int cols,
                         bool vec, cudaStream_t stream);

// ------------------------------------------------------- pair products
enum HeadMode : int {
  HEAD_STATS = 0,  // logits tile -> row statistics
  HEAD_DZ = 1,     // logits tile -> gradient of the logits (16-bit, or its three planes)
  HEAD_DH = 2,     // dz . W      -> fp32 sums
  HEAD_DW = 3      // dz^T . H    -> dW
};

struct HeadArgs {
  const int* count;
  int T, V, K, D;
  int cols;       // entries of this piece of the vocabulary
  int col0;       // vocabulary entry of the piece's column 0
  int b_row0;     // STATS, DZ, DH: row of the weight map for the piece's column 0
  int k_blocks;   // 64-deep stages of the k axis (DW: were every row to count)
  int splits, k_per_split;  // DH: ranges of the k axis summed apart
  int chunk;      // stages of the k axis summed in tensor memory, at most, before they are added in fp32
  int reduce;     // DH: add to the sums instead of storing them
  int bf16;
  float k2;       // scale * log2(e)
  float flat;     // eps / V (cross entropy), else 0
  const int64_t* target;    // cross entropy: the target of row r, with mass `mass`
  float mass;
  const int* source;        // null: row r is row r of H, and count is null
  const int* ids;           // distillation
  const float* q;
  float2* ms;     // STATS
  float* dot;
  int tile0;      // STATS: index of the piece's first column tile
  int parts;      // STATS: epilogue warps per quarter of a tile's rows, 1 or 2
  const float4* coef;     // DZ
  const int* spread;      // DZ, DH: not null and not 0: dz is there a second time, for DH
  const float* factor;    // DW
  void* out;              // DW
  int64_t ld_out;
  int store_granule;      // DW: 0 bulk-tensor stores, else the granule of per-thread stores
  int out_row0;           // DW: row of dW for the piece's column 0
  unsigned long long timeout_ns;
  unsigned int* status;
};

// Output tile of every product: 256 x 256 per CTA pair.
constexpr int kHeadTile = 256;
// planes: 1 (16-bit operands), 2 (the same, with dz in two planes) or 3 (fp32).
cudaError_t launch_head_stats(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                              const HeadArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_head_dz(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                           const HeadArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_head_dh(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                           const HeadArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_head_dw(int planes, const CUtensorMap& mapA, const CUtensorMap& mapB, const CUtensorMap& mapC,
                           const HeadArgs& args, int pairs, cudaStream_t stream);

// dH by dh_pairs pairs and dW by dw_pairs, side by side.
struct HeadLaunch {
  CUtensorMap a, b, c;
  HeadArgs args;
};
cudaError_t launch_head_both(int planes, const HeadLaunch& dh, int dh_pairs, const HeadLaunch& dw, int dw_pairs,
                             cudaStream_t stream);

// ---------------------------------------------- 9 to 32 fp32 rows
// STATS of rows read in place on the CUDA cores, one part per head_simt_tile(T) entries.
struct HeadSimtArgs {
  HeadArgs head;
  const float* H;
  int64_t ldh;
  const float* W;  // the piece's first entry
  int64_t ldw;
};
constexpr int64_t kHeadSimtRows = 32;
int head_simt_tile(int64_t T);
cudaError_t launch_head_simt(const HeadSimtArgs& args, bool aligned, cudaStream_t stream);

// ------------------------------------------------------------- few rows
// Statistics of a few rows of H, read in place, in one pass over W on the CUDA
// cores; few_blocks(T, V) parts.
struct FewArgs {
  int T, V, D, K;
  const void* H;
  int64_t ldh;
  const void* W;
  int64_t ldw;
  float k2, flat;
  const int64_t* targets;
  float mass;
  const int* ids;
  const float* q;
  float2* ms;
  float* dot;
  int64_t ld_stats;  // rows of all passes
  // backward
  RowRule rule;
  float scale, z_loss;
  const float* lse;
  const float* grad;
  float* dz;         // V x rows_held(T)
};
constexpr int kFewRows = 8;   // held in shared memory at a time
// 9 to 32 fp32 rows take passes of eight over vocabularies below this, whose tiles
// would leave most SMs idle.  Forward calls, passes and tiles: 4096 x 4096, 9 rows
// 52 and 187 us, 32 rows 110 and 160 us; 16384 x 2048, 84 and 98, 148 and 86 us.
constexpr int64_t kFewSimtV = 16384;
constexpr int kFewSmem = 160 * 1024;
constexpr int kFewSms = 152;
// Whether these rows take it (`aligned`: W's rows on the 16-byte grid).
bool few_rows(bool backward, int64_t T, int64_t V, int64_t D, bool f32, bool aligned);
int few_blocks(int64_t T, int64_t V);
// Backward of a few rows: dz first, then dW and dH in one pass over W (each block
// a share of the vocabulary and up to 256 16-byte pieces of the columns), dH as
// one sum per share.
struct FewGradArgs {
  int T, V, D;
  const void* H;
  int64_t ldh;
  const void* W;
  int64_t ldw;
  const float* dz;
  RowRule rule;
  void* dW;            // null: not wanted
  int64_t lddw;
  int store_granule;   // alignment of dW's rows in bytes
  float* acc;          // shares x T x ld_acc; null: dH is not wanted
  int64_t ld_acc;
  int shares;
};
int few_held(int64_t T);  // rows of dz: T rounded up to a power of two
int few_shares(int64_t V, int64_t D, bool f32);
cudaError_t launch_few_grad(const FewArgs& f, const FewGradArgs& g, int type, bool aligned, int blocks,
                            cudaStream_t stream);
// type: 0 bf16, 1 f16, 2 f32; granule: alignment of W's rows in bytes
cudaError_t launch_few_stats(const FewArgs& args, int type, int granule, int blocks, cudaStream_t stream);

}  // namespace tgemm
