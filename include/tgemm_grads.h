/*
 * tgemm gradients -- the norm over all gradients of a training step, and their
 * clipping, on NVIDIA GB300 (sm_103a).  Part of libtgemm.so; same conventions as
 * tgemm.h: plain integers and pointers, status codes of enum tgemm_status, a
 * stream as `void*`, nothing allocated, asynchronous on `stream`, safe to call
 * from several host threads.
 *
 * The n gradients are given by their first elements (device pointers, aligned to
 * their element), their numbers of elements (dense, any shape) and their types:
 * TGEMM_F32, TGEMM_F16 or TGEMM_BF16, mixed as you like.  The lists themselves are host memory, read during
 * the call only.
 *
 *     norm = sqrt(sum over all elements of x^2)
 *
 * Squares are added in fp32 a few at a time and from there in fp64, in a fixed
 * order (no atomics: the same call gives the same bits); squares that leave
 * fp32's range are taken in fp64.  norm is one float32 on the device.
 *
 * Clipping writes x * (max_norm / norm) where norm > max_norm, else x: the factor
 * is one fp32 number, the product is rounded once to the output's type.  A norm
 * that is infinite or NaN as it is returned (also one past fp32's largest number) scales
 * nothing (x as it is): look at norm, and skip the step.
 *
 * Errors: TGEMM_ERR_INVALID_VALUE for n < 0, a negative count, a null list or
 * pointer (of a tensor that has elements), a max_norm that is negative or NaN, a
 * workspace that is null, not 256-byte aligned or too small;
 * TGEMM_ERR_UNSUPPORTED_DTYPE; TGEMM_ERR_MISALIGNED; TGEMM_ERR_ALIAS where what is
 * written (outputs, norm, workspace) overlaps anything else of the call, but for
 * an output that is its own input; TGEMM_ERR_TOO_LARGE for n > TGEMM_GRAD_MAX_TENSORS
 * or 2^40 elements.  They are returned before any CUDA call.
 */
#ifndef TGEMM_GRADS_H
#define TGEMM_GRADS_H

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TGEMM_GRAD_MAX_TENSORS 1048576

/* Bytes of workspace both calls need for n tensors: device memory owned by the
 * caller, 256-byte aligned, no initialisation needed.  Calls that may run at the
 * same time must not share one.  Needs no GPU. */
TGEMM_API int tgemm_grad_workspace_size(int64_t n, size_t* bytes);

TGEMM_API int tgemm_grad_norm(int64_t n, const void* const* grads, const int64_t* counts, const int* dtypes,
               float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* outputs: where each scaled gradient goes, same count and type; NULL: in place
 * (a list may also name a gradient itself).  In place nothing is written where
 * nothing is scaled.  A gradient may be listed once only where it is written. */
TGEMM_API int tgemm_grad_clip(int64_t n, const void* const* grads, const int64_t* counts, const int* dtypes,
               void* const* outputs, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_GRADS_H */
