/*
 * tcl_fp8.h — products of 8-bit floating point (e4m3) matrices with one fp32
 * scale for each 128 values, and the sorting of tokens by expert around them.
 *
 * Part of the library that tcl_gemm.h describes: its statuses, memory and
 * ownership, streams and CUDA graphs hold here too, with these differences.
 *   Sizes: a count of rows or tokens may be 0 (nothing is launched, or what has
 *     no rows is written as zeros); widths and K are at least 1, and either is
 *     below 2^31 - 2^16 (TCL_ERR_DIMS otherwise; widths of rows that are quantised
 *     along them, gathered or combined end at 67,107,840).
 *   Nothing is kept between calls but library scratch, which only operands that
 *     miss the alignment below use.
 *   Reported by tcl_last_device_error(): code 7, the experts' offsets do not
 *     ascend from 0 within the rows (or are off the multiples of 128 where
 *     those are asked for); such a launch writes nothing. Waits inside the
 *     products' kernels end after 1 s (codes 1 to 4 as in tcl_gemm.h).
 *
 * Values: a group of 128 numbers x has the scale s = max(max|x| / 448, 2^-126)
 *   and holds q = e4m3(x · (1/s)), rounded to nearest even; q·s stands for x. A
 *   group that is cut off by the matrix' end holds fewer numbers. A NaN makes its
 *   whole group NaN, an infinity a group of NaN and of 0 times infinity: either
 *   comes out of every product with the group as NaN. The 4-byte scales of a
 *   matrix of R rows and G groups lie at scale[row * s_row + group * s_group]
 *   with any strides, in elements; kernels read them fastest with s_row = 1.
 *
 * Products: C = A · B^T, A[M][K] and B[N][K] both with K contiguous (a layer's
 *   weights as they are stored, outputs × inputs),
 *     C[i][j] = sum over groups g of (SA[i][g] · SB[j][g]) · sum over k in g of
 *               A[i][k] · B[j][k],
 *   a group's sum on the tensor cores in fp32, scales (their product too, which
 *   over- and underflows as one) and the sum over groups in fp32, C rounded once. C is fp32 (TCL_OUT_F32) or bf16 (TCL_OUT_BF16) and is
 *   overwritten. Leading dimensions are in elements.
 *
 * Alignment: scales 4 bytes, fp32 and bf16 matrices their element size. e4m3
 *   operands whose base is not 16-byte aligned, or whose leading dimension or
 *   (experts' matrices) distance from one another is not a multiple of 16, are
 *   copied into library scratch first, every matrix of them, a byte at a time and
 *   on every call (64 matrices of 4096 × 2048: 2.2 ms before a product of 50 us).
 *   The scratch grows on demand (TCL_ERR_CAPTURE if that would be inside a
 *   capture). K itself is free.
 */
#ifndef TCL_FP8_H
#define TCL_FP8_H

#include "tcl_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { TCL_X_BF16 = 0, TCL_X_F32 = 1 } tcl_x_t;

/* A side's scales: one scale row per matrix row, or per 128 rows. */
typedef enum { TCL_SCALE_ROWS = 0, TCL_SCALE_BLOCKS = 1 } tcl_scale_t;

/* Most experts of one call. */
#define TCL_MAX_EXPERTS 1024

/* Q[i][c], scale[i][c/128] = X[i][c] in groups along the rows (activations as
 * operands of a product over their columns). X: rows × cols, bf16 or fp32.
 * The bytes of Q's rows between cols and the next multiple of 16 are written as
 * zeros where ldq has room for them.
 * With `position` (tokens sorted by expert, tcl_sort_by_expert): rows = tokens,
 * and token t's row goes to each of the rows position[t*top + j] >= 0 of Q; the
 * rows r < out_rows with source[r] < 0 are written as a group of zeros is.
 * Without: top, source and out_rows are ignored. */
TCL_API int tcl_quantize_fp8_rows(int x_type, int rows, int cols, const void* X, int ldx, const int32_t* position,
                                  int top, const int32_t* source, int out_rows, void* Q, int ldq, float* scale,
                                  long long s_row, long long s_group, cudaStream_t stream);

/* Groups of 128 down a column, the result stored transposed (operands of a
 * weight gradient, a product over the rows): Q[c][i], scale[c][i/128] (at
 * c*s_row + i/128*s_group) from X[i][c]. With `source`: Q has out_rows columns,
 * column r from row source[r] / top of X, zeros where source[r] < 0 (or beyond
 * X's rows). The bytes of Q's rows between its columns and the next multiple of
 * 16 are written as zeros where ldq has room. */
TCL_API int tcl_quantize_fp8_columns(int x_type, int rows, int cols, const void* X, int ldx, const int32_t* source,
                                     int top, int out_rows, void* Q, int ldq, float* scale, long long s_row,
                                     long long s_group, cudaStream_t stream);

/* One scale for each block of 128 × 128 (weights), for `batch` matrices X at
 * x_batch elements from one another. Q[i][c] and scale[i/128][c/128], or with
 * transpose Q[c][i] and scale[c/128][i/128] (for the gradient of the inputs; the
 * same values and scales); scale contiguous for each matrix, one after another;
 * Q's matrices q_batch bytes apart. Padding as above. */
TCL_API int tcl_quantize_fp8_blocks(int x_type, int batch, int rows, int cols, const void* X, int ldx,
                                    long long x_batch, int transpose, void* Q, int ldq, long long q_batch,
                                    float* scale, cudaStream_t stream);

/* C = A · B^T. SA: scale rows for A's rows. SB: sb_kind TCL_SCALE_ROWS, for B's
 * rows, or TCL_SCALE_BLOCKS, for each 128 of them. M >= 0. */
TCL_API int gemm_fp8(int M, int N, int K, const void* A, int lda, const float* SA, long long sa_row,
                     long long sa_group, const void* B, int ldb, const float* SB, int sb_kind, long long sb_row,
                     long long sb_group, void* C, int ldc, int out, cudaStream_t stream);

/* Rows of A sorted by expert, each expert's times its own matrix: expert e's
 * rows are offsets[e] .. offsets[e+1]-1 (experts + 1 ascending numbers in device
 * memory, from 0 to at most rows, any alignment), C[r] = A[r] · B[e]^T with
 * B[e] (N × K) at e*b_expert bytes and its scales at e*sb_expert elements. Rows
 * from offsets[experts] on are written as zeros. */
TCL_API int gemm_fp8_experts(int rows, int experts, int N, int K, const void* A, int lda, const float* SA,
                             long long sa_row, long long sa_group, const void* B, int ldb, long long b_expert,
                             const float* SB, int sb_kind, long long sb_expert, long long sb_row,
                             long long sb_group, const int32_t* offsets, void* C, int ldc, int out,
                             cudaStream_t stream);

/* The experts' weight gradients: C[e] = sum over expert e's rows r of
 * A[n][r] · B[k][r], for A (N × rows) and B (K × rows) quantised down the sorted
 * rows and stored transposed (tcl_quantize_fp8_columns). offsets are multiples
 * of 128 (tcl_sort_by_expert's align), so that no group spans two experts.
 * C[e] (N × K) at e*c_expert elements; an expert without rows gets zeros. */
TCL_API int gemm_fp8_experts_wgrad(int rows, int experts, int N, int K, const void* A, int lda, const float* SA,
                                   long long sa_row, long long sa_group, const void* B, int ldb, const float* SB,
                                   long long sb_row, long long sb_group, const int32_t* offsets, void* C, int ldc,
                                   long long c_expert, int out, cudaStream_t stream);

/* Order of the slots (tokens × top expert choices) by expert, and within an
 * expert by slot. ids: tokens × top contiguous, 4 or 8 bytes each (id_bytes);
 * a choice outside 0 .. experts-1 is dropped.
 *   offsets[experts + 1]: expert e's first row; each expert's length is rounded
 *     up to a multiple of align (1 .. 128).
 *   position[tokens * top]: the slot's row, -1 for a dropped one.
 *   source[rows]: the row's slot, -1 for a row that no slot has. rows is at least
 *     tokens*top + min(experts, tokens*top)*(align-1), rounded down to a multiple
 *     of align (TCL_ERR_DIMS otherwise).
 * Stable and without atomics whose order could show: the same ids give the same
 * order. */
TCL_API int tcl_sort_by_expert(int tokens, int top, const void* ids, int id_bytes, int experts, int align, int rows,
                               int32_t* offsets, int32_t* position, int32_t* source, cudaStream_t stream);

/* Y[r] = X[source[r] / top], zeros where source[r] < 0; X: tokens × cols, Y:
 * rows × cols, both of x_type. Its gradient is tcl_combine without weights. */
TCL_API int tcl_gather_rows(int x_type, int tokens, int top, int rows, int cols, const void* X, int ldx,
                            const int32_t* position, const int32_t* source, void* Y, int ldy, cudaStream_t stream);

/* out[t] = sum over j of weights[t*top + j] · Y[position[t*top + j]], in fp32 in
 * the order of j, rounded once; dropped slots add nothing. weights NULL: ones.
 * Y: rows × cols, out: tokens × cols, both of x_type. */
TCL_API int tcl_combine(int x_type, int tokens, int top, int rows, int cols, const void* Y, int ldy,
                        const float* weights, const int32_t* position, void* out, int ldo, cudaStream_t stream);

/* Gradients of tcl_combine from the gradient G (tokens × cols) of its output:
 *   DY[position[t*top + j]] = weights[t*top + j] · G[t], zeros in the rows r with
 *   source[r] < 0;  DW[t*top + j] = sum over columns of G[t] · Y[position], 0 for a
 *   dropped slot, in fp32. Either of DY and DW may be NULL (not computed); Y is
 *   read only for DW. */
TCL_API int tcl_combine_grad(int x_type, int tokens, int top, int rows, int cols, const void* G, int ldg,
                             const void* Y, int ldy, const float* weights, const int32_t* position,
                             const int32_t* source, void* DY, int lddy, float* DW, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TCL_FP8_H */
