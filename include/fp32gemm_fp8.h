/*
 * fp32gemm_fp8 -- matrices held in 8-bit floating point (e4m3) with one
 * binary32 scale for each block of 128: quantisation, and the product of two
 * such matrices on the matrix cores of gfx950.
 *
 * Same conventions as fp32gemm.h: row-major matrices with leading dimensions
 * in elements, device pointers owned by the caller, work enqueued on `stream`
 * without synchronising on the current device, errors reported through
 * fg_status / fg_last_bad_arg() / fg_last_error(), nothing enqueued when an
 * argument is rejected, no allocation.
 *
 * Codes. e4m3 (1 sign, 4 exponent, 3 mantissa bits, bias 7; largest value
 * 448, no infinities, 0x7F and 0xFF are NaN), one byte each. Rows of a matrix
 * of codes start at multiples of 16 bytes (base address and leading
 * dimension); a row's bytes up to the next multiple of 16 may be read, and
 * have no effect.
 *
 * Scales. A matrix of codes with R rows and C columns has ceil(C / 128)
 * column blocks, and its scales are stored block by block:
 *   FG_BLOCK_ROW   S[b * lds + i]        for row i, columns [128 b, 128 b + 128)
 *   FG_BLOCK_TILE  S[b * lds + i / 128]  for rows [128 (i / 128), ... + 128)
 * with lds >= R (FG_BLOCK_ROW) or >= ceil(R / 128) (FG_BLOCK_TILE). Element
 * (i, c) stands for code(i, c) * S of its block.
 */
#ifndef FP32GEMM_FP8_H
#define FP32GEMM_FP8_H

#include "fp32gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of these entry points' matrices. */
typedef enum fg_type {
    FG_TYPE_F32 = 0,
    FG_TYPE_BF16 = 1,
    FG_TYPE_E4M3 = 2 /* codes with block scales */
} fg_type;

/* Which elements share a scale. */
typedef enum fg_block {
    FG_BLOCK_ROW = 0, /* 1 x 128 */
    FG_BLOCK_TILE = 1 /* 128 x 128 */
} fg_block;

/*
 * fg_quantize_fp8: X (M x N, binary32 or bfloat16) to codes and scales, in
 * its own order (Q, S) and/or transposed (QT, ST), X read once for both.
 *
 * For every block: s = max(fl32(max|x| / 448), 2^-126) over the block's
 * finite elements, and each code is the e4m3 value nearest to the exact
 * quotient x / s, ties to even. NaN and infinities become a NaN code and do
 * not enter the scale. Q is M x N with blocks along the rows of X; QT is
 * N x M, the codes of X's transpose with blocks along the columns of X (128
 * rows of X), as the product that sums over X's rows needs them. With
 * FG_BLOCK_TILE both have the same 128 x 128 blocks.
 *
 * Arguments (positions used by fg_last_bad_arg):
 *   1 type            : FG_TYPE_F32 or FG_TYPE_BF16
 *   2 block           : fg_block
 *   3 M, 4 N          : >= 0
 *   5 X, 6 ldx        : ldx >= max(1, N), any alignment of the type
 *   7 Q, 8 ldq        : NULL, or M rows of codes, ldq >= N, multiple of 16
 *   9 S, 10 lds       : Q's scales (non-NULL with Q)
 *   11 QT, 12 ldqt    : NULL, or N rows of codes, ldqt >= M, multiple of 16
 *   13 ST, 14 ldst    : QT's scales (non-NULL with QT)
 *   15 stream
 * At least one of Q and QT must be given (else bad argument 7). Bytes of a
 * row past its last code are not written. M == 0 or N == 0: FG_OK, nothing
 * enqueued.
 */
fg_status fg_quantize_fp8(fg_type type, fg_block block, int64_t M, int64_t N, const void* X,
                          int64_t ldx, uint8_t* Q, int64_t ldq, float* S, int64_t lds,
                          uint8_t* QT, int64_t ldqt, float* ST, int64_t ldst,
                          hipStream_t stream);

/*
 * fg_gemm_fp8: C = alpha * A * B^T + beta * C for A (M x K) and B (N x K)
 * in codes, both stored with K along the rows:
 *
 *   C(i,j) = alpha * sum_b SA[b*ldsa + i] * SB(b,j) *
 *                    sum_{k in block b} A(i,k) * B(j,k)  +  beta * C(i,j)
 *
 * Products are exact and sums binary32, whatever C's type. SA * SB of a block
 * is rounded to binary32 first, but where that would be infinite or lose bits
 * below the smallest normal number. A's scales are FG_BLOCK_ROW, B's either kind. A linear
 * layer's three products are all of this form: Y = X W^T (X by rows, W by
 * tiles), dX = dY W (W's transposed codes), dW = dY^T X (both transposed
 * codes, by rows; beta = 1 adds to what is there).
 *
 * Arguments (positions used by fg_last_bad_arg):
 *   1 M, 2 N, 3 K     : >= 0
 *   4 alpha
 *   5 A, 6 lda        : lda >= K, multiple of 16; A 16-byte aligned
 *   7 SA, 8 ldsa      : ldsa >= M
 *   9 B, 10 ldb       : ldb >= K, multiple of 16; B 16-byte aligned
 *   11 SB, 12 ldsb    : ldsb >= N or ceil(N / 128)
 *   13 block_b        : fg_block of B's scales
 *   14 beta
 *   15 C, 16 ldc      : ldc >= N
 *   17 type_c         : FG_TYPE_F32 or FG_TYPE_BF16 (rounded once)
 *   18 workspace      : NULL, or device memory, 16-byte aligned, that no call
 *                       that may run at the same time uses
 *   19 workspace_bytes: its size; fg_gemm_fp8_workspace_size gives what the
 *                       call can use (less is never an error: the sum over K
 *                       is split among fewer workgroups, or not at all)
 *   20 stream
 * Quick returns and the treatment of alpha == 0, K == 0 and beta == 0 are
 * those of fg_sgemm; M and N are at most 2^30, and C has fewer than 2^23 tiles
 * of 256 x 128 (else FG_ERR_UNSUPPORTED). Repeated calls with the same arguments and workspace
 * size give identical bits. Leading dimensions up to FG_MAX_LD.
 */
fg_status fg_gemm_fp8(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t* A,
                      int64_t lda, const float* SA, int64_t ldsa, const uint8_t* B, int64_t ldb,
                      const float* SB, int64_t ldsb, fg_block block_b, float beta, void* C,
                      int64_t ldc, fg_type type_c, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

/* Workspace bytes fg_gemm_fp8 can use for this shape (0: none). Host only. */
size_t fg_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* FP32GEMM_FP8_H */
