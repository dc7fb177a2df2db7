/*
 * tcl_dense.h — a language model's dense path on bf16 matrices: the gated feed-forward block and
 * the cross entropy over a vocabulary, both with their gradients, and the norm and clipping of
 * gradients.
 *
 * Part of the library that tcl_gemm.h describes: its statuses, streams and CUDA graphs hold here
 * too, with these differences.
 *   Sizes: tokens may be 0 (nothing is read; the gradients of weights are zeros); widths are at
 *     least 1; all are below 2^31 - 2^16, and a product has fewer than 2^30 tiles of 256 × 128 (the
 *     block's first one of 256 × 64; TCL_ERR_DIMS otherwise). What a sum runs over is at most 2^25:
 *     hidden and inner; for the gradients also the vocabulary and the block's tokens.
 *   Memory: nothing is allocated and nothing kept between calls. A call that needs a workspace
 *     gets it from the caller: *workspace_bytes is the size of what `workspace` points to (256-byte
 *     aligned; 0 and NULL: none). Where a call needs more, it launches nothing, writes the size
 *     into *workspace_bytes and returns TCL_ERR_WORKSPACE; the size depends on the sizes, the
 *     leading dimensions and the alignment of the operands. A workspace may be used again as soon
 *     as the call's work on the stream is done.
 *   Waits inside the kernels end after 1 s and are reported by tcl_last_device_error() (codes 1 to 4
 *     as in tcl_gemm.h).
 *
 * Matrices are bf16, row-major, leading dimensions in elements; weights as a layer stores them,
 * outputs × inputs. Bases have to be aligned to their element (TCL_ERR_ALIGN). Operands whose
 * base is not 16-byte aligned or whose leading dimension is not a multiple of 8 are copied into the
 * workspace first. Results may have any leading dimension (rows on 16-byte pieces are stored
 * fastest); what lies between their rows is left as it was. They overlap neither operands nor one another.
 *
 * Products run on the tensor cores with fp32 sums, of which every result is rounded once; what is
 * rounded to bf16 between two products of a call, and what clipping rounds, is named there.
 */
#ifndef TCL_DENSE_H
#define TCL_DENSE_H

#include <stddef.h>

#include "tcl_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(g): g·sigmoid(g); g·Phi(g), Phi the normal distribution; its tanh form
 * g·(1 + tanh(sqrt(2/pi)·(g + 0.044715·g^3)))/2 */
typedef enum { TCL_ACT_SILU = 0, TCL_ACT_GELU = 1, TCL_ACT_GELU_TANH = 2 } tcl_act_t;

/* out = h · Wdown^T,  h = act(gate) * up,  gate = X · Wgate^T,  up = X · Wup^T.
 * X, out: tokens × hidden; Wgate, Wup: inner × hidden; Wdown: hidden × inner.
 * h (tokens × inner, bf16) is written in any case: the second product reads it. gate and up,
 * both or neither (NULL), are written in bf16 for tcl_gated_ffn_grad. All three share ld_kept, a
 * multiple of 8 that is at least inner, and are 16-byte aligned; the columns of their rows from
 * inner to the next multiple of 8 are overwritten. */
TCL_API int tcl_gated_ffn(int tokens, int hidden, int inner, const void* X, int ldx, const void* Wgate, int ld_gate,
                          const void* Wup, int ld_up, const void* Wdown, int ld_down, int act, void* gate, void* up, void* h,
                          int ld_kept, void* out, int ldo, void* workspace, size_t* workspace_bytes, cudaStream_t stream);

/* Gradients of the same from `grad`, that of out (tokens × hidden), and what the forward pass kept:
 *   dh = grad · Wdown,  dgate = dh * up * act'(gate),  dup = dh * act(gate)   (both bf16)
 *   dX = dgate · Wgate + dup · Wup,  dWgate = dgate^T · X,  dWup = dup^T · X,  dWdown = grad^T · h
 * dX is bf16, the weights' gradients are all of type w_type (TCL_OUT_BF16 or TCL_OUT_F32). */
TCL_API int tcl_gated_ffn_grad(int tokens, int hidden, int inner, const void* grad, int ld_grad, const void* X, int ldx,
                               const void* Wgate, int ld_gate, const void* Wup, int ld_up, const void* Wdown, int ld_down,
                               int act, const void* gate, const void* up, const void* h, int ld_kept, void* dX, int ld_dx,
                               void* dWgate, int ld_dgate, void* dWup, int ld_dup, void* dWdown, int ld_ddown, int w_type,
                               void* workspace, size_t* workspace_bytes, cudaStream_t stream);

/* With logits l = X · W^T (tokens × vocab, never stored) and for each token t
 *   lse[t] = log sum over v of exp(l[t][v]),  loss[t] = lse[t] - l[t][target[t]],
 * both fp32. Targets are int32 or int64 (target_bytes 4 or 8); one outside 0 .. vocab-1 drops its
 * token: its loss is 0. A logit beyond ±2^30 counts as infinite: above it lse is infinity, below it the word has
 * no weight. X: tokens × hidden, W: vocab × hidden. */
TCL_API int tcl_cross_entropy(int tokens, int hidden, int vocab, const void* X, int ldx, const void* W, int ldw,
                              const void* targets, int target_bytes, float* loss, float* lse, void* workspace,
                              size_t* workspace_bytes, cudaStream_t stream);

/* The same and the gradients of sum over t of grad[t]·loss[t] (grad: fp32):
 *   d[t][v] = grad[t]·(exp(l[t][v] - lse[t]) - [v = target[t]]),  dX = d · W (bf16),  dW = d^T · X
 * (w_type). Dropped tokens add nothing, whatever their rows hold, and their rows of dX are zeros; one that is
 * not dropped and has a logit that is infinity, beyond 2^30 or NaN makes its row of dX and all of dW NaN.
 * The exponentials are computed once, kept in bf16 for a piece of the tokens at a time (at most
 * 2 GiB, or 256 tokens) and read by both products; the rows of X for dW are rounded to bf16 again
 * after their scaling by grad[t] / (sum of the exponentials). Pieces of dW are added in fp32. */
TCL_API int tcl_cross_entropy_grad(int tokens, int hidden, int vocab, const void* X, int ldx, const void* W, int ldw,
                                   const void* targets, int target_bytes, const float* grad, float* loss, float* lse,
                                   void* dX, int ld_dx, void* dW, int ld_dw, int w_type, void* workspace,
                                   size_t* workspace_bytes, cudaStream_t stream);

/* norm = sqrt of the sum of the squares of all elements of `count` tensors (host arrays of their
 * addresses, lengths and types, TCL_OUT_F32 or TCL_OUT_BF16), fp32 on the GPU. Tensors may be empty.
 * Squares are added in fp32 for 32 elements at a time, in fp64 beyond that, in an order that the lengths
 * and addresses fix. */
TCL_API int tcl_grad_norm(int count, const void* const* tensors, const long long* lengths, const int* types, float* norm,
                          void* workspace, size_t* workspace_bytes, cudaStream_t stream);

/* The same, and to[i] = from[i] · f with f = bound/norm where norm > bound; else, and where the
 * norm is infinite or NaN, to[i] = from[i]. f is worked out in fp64 and rounded to fp32, the product to fp32
 * and from there to bf16 where that is the type. to[i] may be from[i]; otherwise a
 * result overlaps no other tensor (TCL_ERR_CONFIG). bound >= 0. */
TCL_API int tcl_clip_gradients(int count, const void* const* from, void* const* to, const long long* lengths,
                               const int* types, float bound, float* norm, void* workspace, size_t* workspace_bytes,
                               cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif
