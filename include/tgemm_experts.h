/*
 * tgemm experts -- the operators of a sparse layer, whose tokens each go to a few
 * of many experts, on NVIDIA GB300 (sm_103a).  Part of libtgemm.so; same
 * conventions as tgemm.h: plain integers and pointers, status codes of enum
 * tgemm_status, a stream as `void*`, nothing allocated, asynchronous on `stream`,
 * safe to call from several host threads.
 *
 * Routing (tgemm_route_*): T rows of E logits x -> k experts and weights a row.
 *
 *   score_e = softmax(x)_e, or sigmoid(x_e)
 *   key_e   = score_e (+ bias_e)                       what experts are picked by
 *   weight  = scale * score (/ the sum of the picked scores, where renormalize)
 *
 * The bias (one float32 per expert, to balance their load) has no part in the
 * weights and no gradient.  With `groups` > 1 the experts are groups of E / groups
 * neighbours; the top_groups groups of the largest value stay, a group's value
 * being its largest key or the sum of its two largest.  Of equal keys, and of
 * equal groups, the one with the lowest index is first; picks are listed by
 * falling key.
 *
 * Picks are those of real arithmetic on the given numbers: without a bias, and
 * without sums of keys, logits are compared as they are; else keys are computed in
 * fp32, and rows in which two that decide come within fp32's error of one
 * another again in fp64.
 *
 * A logit of -inf masks its expert (as does a bias of -inf): it is never picked.
 * Where fewer than k are left, the places left over hold id -1 and weight 0.  A NaN
 * logit ranks first, and makes NaN of the weights that it takes part in.
 *
 * The experts' products (tgemm_experts_*): with e = ids[t][j]
 *
 *   (g, u) = W_in[e] x_t,   h = g sigmoid(g) u   (F each)
 *   out_t  = sum_j weights[t][j] W_out[e] h
 *
 *   x: T x D, x[t*ldx + d]
 *   W_in: E x 2F x D, row r of expert e at W_in[(e*2F + r)*ld_in]: F gates, F ups
 *   W_out: E x D x F, row d of expert e at W_out[(e*D + d)*ld_out]
 *   ids, weights: T x k, dense; int64 and float32
 *
 * x, W_in, W_out and what is computed from them are bf16 or fp16; products run on
 * the tensor cores with fp32 sums, h is rounded to the operands' type on its way
 * into the second product, and out, summed in fp32, is rounded once.  A place whose
 * id is below 0 is unused; a row without a used place gives 0 (and x may hold
 * anything there, NaN included).  An id of E or more is an error in the data: its
 * row of out is NaN, and so are its row of dx and its place of dweights; it has no
 * part in any other gradient.  An expert listed twice counts twice.
 *
 * Results do not depend on timing: every sum has a fixed order, no atomics.
 */
#ifndef TGEMM_EXPERTS_H
#define TGEMM_EXPERTS_H

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TGEMM_ROUTE_MAX_EXPERTS 1024
#define TGEMM_ROUTE_MAX_K 32
#define TGEMM_ROUTE_MAX_GROUPS 32

enum tgemm_route_scoring { TGEMM_ROUTE_SOFTMAX = 0, TGEMM_ROUTE_SIGMOID = 1 };
enum tgemm_route_group_score { TGEMM_ROUTE_GROUP_MAX = 0, TGEMM_ROUTE_GROUP_TOP2 = 1 };

/* Options of the routing; NULL means softmax scores, no groups, weights as they
 * are.  Zero-initialise and set what you need. */
typedef struct tgemm_route_options {
  int scoring;      /* enum tgemm_route_scoring */
  int renormalize;  /* 0 or 1 */
  float scale;      /* factor of the weights, finite, >= 0; 0 means 1 */
  int groups;       /* 0 means 1; divides E */
  int top_groups;   /* 0 means 1; at most groups, and k at most top_groups * E / groups */
  int group_score;  /* enum tgemm_route_group_score */
  int reserved[2];  /* must be 0 */
} tgemm_route_options;

/*
 * Routing, forward.  logits: T x E, row pitch ld >= E, of dtype TGEMM_F32, TGEMM_F16
 * or TGEMM_BF16.  bias: E float32, or NULL.  ids, weights: T x k, dense.
 *
 * Errors: TGEMM_ERR_INVALID_VALUE for T < 0, E < 1, k < 1, k > E, a short pitch, a
 * null pointer with T > 0, a bad option; TGEMM_ERR_UNSUPPORTED_DTYPE;
 * TGEMM_ERR_MISALIGNED for a pointer not aligned to its element; TGEMM_ERR_ALIAS
 * when an output overlaps an input or another output; TGEMM_ERR_TOO_LARGE for E,
 * k or groups above the limits here, T >= 2^31 - 256 or ld >= 2^31.  They are
 * returned before any CUDA call.  T == 0 does nothing.
 */
TGEMM_API int tgemm_route_forward(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ld, int dtype,
               const float* bias, const tgemm_route_options* opts, int64_t* ids, float* weights, void* stream);

/* Routing, backward: d_logits (T x E, pitch ld_out >= E, dtype as logits) of
 * sum(grad * weights), for the forward call's ids; grad: T x k float32, dense
 * (places with an id below 0 are not read; an id of E or more is left out). */
TGEMM_API int tgemm_route_backward(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ld, int dtype,
               const int64_t* ids, const float* grad, const tgemm_route_options* opts, void* d_logits,
               int64_t ld_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_EXPERTS_H */
