// Internal interfaces of the experts' products (experts_api.cu, experts_rows.cu,
// experts_gemm.cuh).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "loss_internal.h"

namespace tgemm {

// ------------------------------------------------- rows in their experts' order
// A place is one (token, j) of ids [T, k], numbered t * k + j; a used place is a row
// of the sorted matrices.  Each expert's rows are neighbours, in the order of
// their places, and fill up to a multiple of kRowPad rows; the filling has the
// token of the expert's first row and no place, and is 0 in the sorted matrices.  Token tiles are the
// products' columns: an expert's rows in even parts of at most kTokenTile.
constexpr int kRowPad = 32;
constexpr int kTokenTile = 256;
constexpr int kMaxExperts = 1024;
constexpr int kPlaceBlock = 2048;  // places of one block of the sort, at most

struct ExpertRows {
  int* head;       // {tiles, rows with the filling}
  int* count;      // E: rows of each expert
  int* first;      // E + 1: its first row
  int4* tiles;     // {expert, first row, rows with the filling, rows}
  int* token;      // of each row
  int* place;      // of each row; -1: filling
  int* row;        // of each place; -1: unused, -2: no such expert
  int* partial;    // blocks x E, for many places
};

struct OrderArgs {
  const int64_t* ids;
  int64_t places;
  int T, E, k;
  ExpertRows rows;
};
int order_blocks(int64_t places);
cudaError_t launch_order(const OrderArgs& a, cudaStream_t stream);

// E x rows rows of cols 16-bit elements copied from pitch ld_from to ld_to (elements; whole
// 16-byte words, as `to`), of the experts with a count; rows = 0: nothing.  used: such
// experts, at most.
struct WeightCopy {
  const void* from;
  void* to;
  int64_t ld_from, ld_to;
  int rows, cols;
};
cudaError_t launch_copy_weights(const int* count, int E, int64_t used, const WeightCopy& in, const WeightCopy& out, int sms,
                                cudaStream_t stream);

// out[r] (pitch ld_out, 16-byte aligned) = the row of x of sorted row r's token; the
// filling is 0.  granule: alignment of x's rows in bytes.  zeros (or null): `words` words
// that become 0.
cudaError_t launch_gather_rows(const ExpertRows& rows, int64_t most_rows, const void* x, int64_t ldx, int granule, int D,
                               void* out, int64_t ld_out, unsigned int* zeros, int words, int sms, cudaStream_t stream);

// fp16 gradients on their way into the products: from v = W_out^T grad in fp32 (as DH leaves
// it), g and u, the rows of dg, du and weight * h in halves, times the powers of two of their
// expert (expert_scale).  The filling is 0.
struct RoundArgs {
  int E, F;
  ExpertRows rows;
  const float* weights;          // of each place
  const float* gu;               // [row / 4][g, u][feature, pitch ldg][row % 4]
  const float* v;                // [row / 4][feature, pitch ldg][row % 4]
  int64_t ldg;
  const unsigned int* largest;   // of each expert: {|dg|, |du|; |weight h|}, floats' bits
  void* dgu;
  int64_t ld_dgu;
  void* h;
  int64_t ldh;
};
cudaError_t launch_round_gradients(const RoundArgs& a, int64_t most_rows, cudaStream_t stream);
// The exponent of the power of two that brings the largest of some finite values (a float's bits)
// into [2^14, 2^15), as far as it and its reciprocal are floats with all bits.
__host__ __device__ inline int expert_exponent(unsigned int largest) {
  const int e = 14 + 127 - static_cast<int>(largest >> 23);
  return e < 126 ? e : 126;
}
#ifdef __CUDACC__
__device__ __forceinline__ float expert_scale(unsigned int largest) {
  return __uint_as_float(static_cast<unsigned int>(127 + expert_exponent(largest)) << 23);
}
__device__ __forceinline__ float expert_unscale(unsigned int largest) {
  return __uint_as_float(static_cast<unsigned int>(127 - expert_exponent(largest)) << 23);
}
#endif

// out[t] = sum over t's rows of weight * y[row] (weights null: of y[row]), rounded
// to type (0 bf16, 1 f16); a place of no such expert: NaN.  dots not null: d_weights
// of each place = the sum of its row's `parts` dots (0 where unused).
struct JoinArgs {
  const ExpertRows* rows;
  const float* weights;
  int64_t T;
  int k, D;
  const void* y;        // fp32, or (type 0) halves times 2^(e - 141), e = y_exponent of 32 columns; e = 0: bf16
  const uint8_t* y_exponent;
  int64_t ldy;
  int type;
  void* out;
  int64_t ld_out;
  const float* dots;
  int parts;
  float* d_weights;
};
cudaError_t launch_join(const JoinArgs& a, cudaStream_t stream);

// ------------------------------------------------------------- a few places
// Forward for a few places on the CUDA cores; x's and the weights' rows are 16-byte
// aligned.
struct ExpertFewArgs {
  int T, E, k, D, F;
  const void* x;
  int64_t ldx;
  const void* w_in;
  int64_t ld_in;
  const void* w_out;
  int64_t ld_out;
  const int64_t* ids;
  const float* weights;
  float* h;              // places x F
  int64_t ldh;           // a multiple of 4
  void* out;
  int64_t ldo;
};
cudaError_t launch_experts_few(const ExpertFewArgs& a, bool bf16, cudaStream_t stream);

// ---------------------------------------------------------------- products
// M is a weight's axis, N the tokens' (the gradients of the weights: M and N the
// weight's two axes, K the expert's rows).
enum ExpertMode : int {
  EXPERT_UP = 0,    // W_in x -> h (and g, u)
  EXPERT_DOWN = 1,  // W_out h -> y
  EXPERT_DH = 2,    // W_out^T d_out -> dg, du, weight * h, dots
  EXPERT_DX = 3,    // W_in^T (dg, du) -> y
  EXPERT_DIN = 4,   // (dg, du)^T x -> dW_in
  EXPERT_DOUT = 5   // d_out^T (weight * h) -> dW_out
};

struct ExpertArgs {
  int E, D, F, T;
  int m_blocks, n_blocks;  // 256-row (UP: 128-feature) blocks of M; gradients of the weights: 256-column blocks of N
  int k_blocks;            // 64-deep stages (gradients of the weights: the rows')
  int chunk;               // stages summed in tensor memory, at most
  int bf16;
  int gather;              // UP: rows of x where they lie
  int split;               // A comes in several boxes
  ExpertRows rows;
  void* h;                 // UP: h; DH: weight * h
  int64_t ldh;
  float* gu;               // UP: g and u where kept, else null; DH: read.  [row / 4][g, u][feature, pitch ldg][row % 4]
  int64_t ldg;
  void* dgu;               // DH
  int64_t ld_dgu;
  float* dots;             // DH: m_blocks * 8 per row
  const float* weights;    // DH: of each place
  // fp16, else null: DH leaves v = W_out^T grad in fp32 and each expert's largest finite numbers
  // (RoundArgs), from which launch_round_gradients makes dgu and h; DX, DIN and DOUT take the
  // powers of two back
  float* v;
  unsigned int* largest;
  void* y;                 // DOWN, DX: fp32, or (bf16) halves with an exponent for each 32 columns (JoinArgs)
  int64_t ldy;             // a multiple of 64
  uint8_t* y_exponent;     // [row / 16][column / 32][row % 16]: a warp's 16 bytes lie together
  void* out;               // DIN, DOUT
  int64_t ld_out;
  int store_granule;       // 0 bulk-tensor stores, else the granule of per-thread stores
  unsigned long long timeout_ns;
  unsigned int* status;
};

// Operands A and B (token products: boxes of 64, 32 and 16 rows), and where all but DH
// store.  Axes of a, from the innermost: UP {k, feature % 16, gate or up, feature /
// 16, expert}, or where args.split {k, feature, 2 expert + (gate or up)}; DOWN {k, row,
// expert}; DH and DX {column % 64, row, column / 64, expert}, or where args.split {column,
// row, expert}.  DIN's and DOUT's a and b: {column % 64, row, column / 64}.
struct ExpertMaps {
  CUtensorMap a, b, b32, b16, c;
};
cudaError_t launch_expert_up(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_expert_down(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_expert_dh(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_expert_dx(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_expert_din(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);
cudaError_t launch_expert_dout(const ExpertMaps& maps, const ExpertArgs& args, int pairs, cudaStream_t stream);

}  // namespace tgemm
