/*
 * tgemm losses -- a language model's vocabulary head fused with its loss, on
 * NVIDIA GB300 (sm_103a).  Part of libtgemm.so; same conventions as tgemm.h:
 * plain integers and pointers, status codes of enum tgemm_status, a stream as
 * `void*`, nothing allocated, asynchronous on `stream`, safe to call from
 * several host threads.
 *
 * The head's product  z[t][v] = scale * sum_d H[t][d] W[v][d]  is computed tile
 * by tile, and the T x V logits are never written out: a tile leaves only the
 * maximum, the sum of exponentials and the weighted sum of each of its rows.
 * The backward pass computes the logits again, in pieces of the vocabulary,
 * and keeps one piece of their gradient (in the workspace) at a time.
 *
 *   H: T x D hidden states, element (t, d) at H[t*ldh + d], ldh >= D
 *   W: V x D head weight, one row per vocabulary entry, W[v*ldw + d], ldw >= D
 *
 * Two losses, float32, one value per row t, with
 * lse_t = log sum_v exp(z[t][v]):
 *
 * Cross entropy (tgemm_xent_*): with the target y_t, eps = label_smoothing and
 * q = (1 - eps) [v = y_t] + eps / V
 *     loss_t = lse_t - sum_v q_v z[t][v] + z_loss * lse_t^2.
 * A row whose target is ignore_index is ignored.
 *
 * Distillation from a teacher's top logits (tgemm_distill_*): row t lists K
 * entries ids[t][k] with the teacher's logits[t][k]; an id below 0 marks an
 * unused place.  With q = softmax over the row's used places of
 * scale * logits (scale = 1 / temperature, on both sides),
 *     loss_t = sum_k q_k log q_k + lse_t - sum_k q_k z[t][ids[t][k]],
 * the divergence of the student's distribution from the teacher's renormalised
 * top-K (the scale is applied to differences from the row's largest logit, so
 * logits may be the type's lowest or largest).  An entry listed twice counts with both masses; a logit of -inf has
 * no mass.  A row with no used place, or whose used logits are all -inf, is
 * ignored.  K <= TGEMM_DISTILL_MAX_K.
 *
 * Ignored rows have loss 0, lse 0 and no part in any gradient, whatever H
 * holds there (NaN included).  Where rows are gathered they cost no product
 * work; calls that read H in place compute them and drop them: forward calls
 * of up to 256 16-byte-aligned 16-bit rows or 32 fp32 rows, and the few rows
 * below.  A row with a target or an id outside [0, V) that is neither ignored
 * nor unused is an error in the data: its loss is NaN and it has no part in
 * any gradient.
 *
 * Gradients, for g[t] = the gradient of the result with respect to loss_t:
 *     dz = g ((1 + 2 z_loss lse) exp(z - lse) - q)
 *     dH = scale * dz W,  dW = scale * dz^T H
 * in H's and W's type, each sum held in float32 and rounded once.  dH and dW are
 * overwritten.  Results do not depend on timing: every sum has a fixed order.
 *
 * Numbers.  Products run on the tensor cores, whose adder truncates: its sums
 * are moved and added in fp32 with rounding to nearest often enough to keep a
 * logit within 7.6e-6 (fp32: 3.8e-6), and a 16-bit gradient's sum within 3.1e-5,
 * of its sum of magnitudes whatever D, V and T; with mixed signs an eighth of
 * that.  Sums that fp32 holds exactly stay exact.  A few rows take the CUDA
 * cores: forward one 16-bit row, eight whose W is off the 16-byte grid, 32 of
 * fp32; backward two aligned 16-bit rows, eight of fp32.
 * dz on its way into the two products:
 *   - few rows on the CUDA cores: float32;
 *   - fp32: three bf16 planes (24 bits), as H and W: six products, errors of
 *     4 to 8e-7 of the norm.  Finite values keep their size up to the type's
 *     largest; an infinite element of H or W makes NaN of its logits;
 *   - 16-bit, T up to 32 (ignored rows among them): two planes, dH and dW as
 *     exact as their own last rounding;
 *   - 16-bit, T above 32: rounded to H's type.  dH and dW are 1.2 to 1.5 times
 *     as far off, in the norm, as their own last rounding makes them (measured
 *     1.24 to 1.48), single rows of dH up to 1.6 times where few rows count.
 * fp16 scales dz by the largest |g| that counts; where other rows' are below
 * 1/64 of it, dH's product reads dz with each row scaled by its own, so dH's
 * rows keep their accuracy.  dW, which sums over the rows, resolves 2^-39 of the
 * largest |g| times |h|.
 */
#ifndef TGEMM_LOSS_H
#define TGEMM_LOSS_H

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TGEMM_DISTILL_MAX_K 256

/* Options of both losses; NULL means the defaults.  Zero-initialise and set
 * what you need (ignore_index 0 is a vocabulary entry like any other: set it
 * to -100, the default, or to what your targets use). */
typedef struct tgemm_loss_options {
  float scale;           /* factor of the logits, finite, >= 0; 0 means 1 */
  float label_smoothing; /* eps in [0, 1]; cross entropy only */
  float z_loss;          /* weight of lse^2, finite, >= 0; cross entropy only */
  int piece;             /* vocabulary entries per piece of the gradient, a
                            multiple of 256 (0: chosen by the library) */
  int64_t ignore_index;  /* cross entropy only; default -100 */
  int wait_timeout_us;   /* bound of every in-kernel wait (0 = 2 s) */
  int reserved[3];       /* must be 0 */
} tgemm_loss_options;

/* Bytes of workspace a call needs: device memory owned by the caller, 256-byte
 * aligned, no initialisation needed, contents unspecified afterwards.  Calls
 * that may run at the same time must not share one.  backward: 0 for the
 * forward calls, 1 for the backward calls; K: 0 for the cross entropy.  W and
 * ldw tell whether the weight's rows are 16-byte aligned (pieces of it are
 * copied to an aligned pitch when they are not; only W's value modulo 16 is
 * looked at).  Needs no GPU.
 *
 * What it holds, beside up to 40 bytes a row and 8 a place of the lists:
 *   - H's rows, gathered: 2 bytes an element, 6 for fp32;
 *   - forward: 12 bytes per row and 256 entries (1.6 GB for 131072 rows of a
 *     vocabulary of 262144);
 *   - a piece of W where it is copied: 2 bytes an element, 6 for fp32;
 *   - backward: a piece of dz, 2 bytes an element and plane (fp16 twice as many),
 *     and 4 bytes an element of dH, several times for few rows (up to 256 MB).
 * Unless `piece` says otherwise, a piece of dz and of W takes 256 MB each, but at
 * least 2048 entries; W copied for up to 256 rows at least 19456 entries (a whole
 * round of tiles: 478 MB for fp32 at D = 4096). */
TGEMM_API int tgemm_loss_workspace_size(int backward, int64_t T, int64_t V, int64_t D, int64_t K,
               const void* W, int64_t ldw, int dtype, const tgemm_loss_options* opts, size_t* bytes);

/*
 * Cross entropy, forward: loss[T] and lse[T] (lse is what the backward call
 * takes; it may be used as is for scoring).  dtype: TGEMM_BF16, TGEMM_F16 or
 * TGEMM_F32.  targets: T int64 on the device.
 *
 * Errors: TGEMM_ERR_INVALID_VALUE for T < 0, V < 1, D < 1, a short leading
 * dimension, a null pointer with T > 0, a bad option, a workspace that is
 * misaligned or smaller than tgemm_loss_workspace_size;
 * TGEMM_ERR_UNSUPPORTED_DTYPE; TGEMM_ERR_MISALIGNED for a pointer not aligned
 * to its element; TGEMM_ERR_ALIAS when an output overlaps an input, another
 * output or the workspace; TGEMM_ERR_TOO_LARGE for T, V >= 2^31 - 256, D >=
 * 2^28, a leading dimension >= 2^31, or K > TGEMM_DISTILL_MAX_K.  They are returned before any
 * CUDA call.  T == 0: the forward calls do nothing, the backward calls zero dW.
 */
TGEMM_API int tgemm_xent_forward(int64_t T, int64_t V, int64_t D,
               const void* H, int64_t ldh, const void* W, int64_t ldw,
               const int64_t* targets, int dtype, const tgemm_loss_options* opts,
               float* loss, float* lse,
               void* workspace, size_t workspace_bytes, void* stream);

/* Cross entropy, backward.  lse: the forward call's.  grad: T float32, the
 * gradient of the result with respect to each loss (only rows that count are
 * read).  dH (T x D, lddh >= D) and dW (V x D, lddw >= D): either may be NULL
 * when it is not wanted. */
TGEMM_API int tgemm_xent_backward(int64_t T, int64_t V, int64_t D,
               const void* H, int64_t ldh, const void* W, int64_t ldw,
               const int64_t* targets, const float* lse, const float* grad,
               int dtype, const tgemm_loss_options* opts,
               void* dH, int64_t lddh, void* dW, int64_t lddw,
               void* workspace, size_t workspace_bytes, void* stream);

/* Distillation, forward.  ids: T x K int64, row pitch ld_ids >= K; logits:
 * T x K float32, row pitch ld_logits >= K.  K >= 1. */
TGEMM_API int tgemm_distill_forward(int64_t T, int64_t V, int64_t D, int64_t K,
               const void* H, int64_t ldh, const void* W, int64_t ldw,
               const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits,
               int dtype, const tgemm_loss_options* opts,
               float* loss, float* lse,
               void* workspace, size_t workspace_bytes, void* stream);

/* Distillation, backward; lse, grad, dH and dW as in tgemm_xent_backward.  The
 * teacher's logits get no gradient. */
TGEMM_API int tgemm_distill_backward(int64_t T, int64_t V, int64_t D, int64_t K,
               const void* H, int64_t ldh, const void* W, int64_t ldw,
               const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits,
               const float* lse, const float* grad,
               int dtype, const tgemm_loss_options* opts,
               void* dH, int64_t lddh, void* dW, int64_t lddw,
               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_LOSS_H */
