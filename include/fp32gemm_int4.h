/*
 * fp32gemm_int4 -- products of a few rows (a decode step) with weights of 4 bits
 * and a scale for each group of columns, plain and as the gated half of a
 * feed-forward block.
 *
 * Same conventions as fp32gemm.h and fp32gemm_fp8.h.
 *
 * Weights. A matrix of N rows and K columns is N rows of ceil(K / 2) bytes: column
 * c of a row is in byte c / 2, an even one in its low half, an odd one in its high
 * half, as q = 0 .. 15. Rows start at multiples of 16 bytes (base address and
 * leading dimension); a row's bytes up to the next multiple of 16 may be read, and have
 * no effect. Each group of `group` columns of a row has a scale s and a zero point z
 * (8 where there are no zero points), stored group by group: S[b * lds + n] and
 * Z[b * ldz + n] for columns [b group, (b + 1) group) of row n. Element (n, c)
 * stands for s * (q - z).
 */
#ifndef FP32GEMM_INT4_H
#define FP32GEMM_INT4_H

#include "fp32gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FG_INT4_MAX_ROWS 64 /* rows of x of one call */

typedef struct fg_int4 {
    const uint8_t* q; /* N rows of ceil(K / 2) bytes */
    int64_t ldq;      /* bytes, >= ceil(K / 2), multiple of 16 */
    const void* s;    /* ceil(K / group) rows of N scales */
    int64_t lds;      /* >= N */
    const uint8_t* z; /* ceil(K / group) rows of N zero points, 0 .. 255, or NULL */
    int64_t ldz;      /* >= N */
} fg_int4;

/*
 * fg_gemm_int4:  out = x W^T.   fg_gated_int4:  out = act(x gate^T) * (x up^T).
 *
 * Arguments (positions used by fg_last_bad_arg):
 *   1 T          : rows of x, 0 .. FG_INT4_MAX_ROWS
 *   2 N, 3 K     : >= 0
 *   4 group      : 32, 64 or 128
 *   5 type       : x and out: FG_TYPE_F32 or FG_TYPE_BF16
 *   6 scale_type : FG_TYPE_F32 or FG_TYPE_BF16
 *   7 x, 8 ldx   : T rows of K elements, starting at multiples of 16 bytes; a row's
 *                  bytes up to the next multiple of 16 may be read, and have no effect
 *   9 w (gate)   : N x K
 *   10 up        : N x K (fg_gated_int4 only; the positions after it stay the same)
 *   11 activation: fg_activation (fg_gated_int4 only)
 *   12 out       : T rows of N elements, no overlap with the inputs
 *   13 ldo       : >= N
 *   14 stream
 * Products with the codes are exact and sums binary32 for either type. FG_TYPE_F32: the
 * sum over a group is of (q - z) x, and its part of the result s times that; of an x below
 * 2^-109 in magnitude the bits under 2^-133 do not count. FG_TYPE_BF16: the sum is taken of
 * q x and of x, and its part is s (sum q x - z sum x); errors are binary32 roundings of
 * s (q + z) |x|, below those of a bfloat16 result unless an x some 10^5 times the others
 * meets its zero point. (Where a sum is not finite it is taken again, of (q - z) x times
 * 2^-20.) Scales are finite, and 0 or of a magnitude between 2^-100 and 2^100; scales and
 * zero points of a matrix reach over less than 2 GiB each (else FG_ERR_UNSUPPORTED).
 * T == 0 or N == 0: FG_OK,
 * nothing enqueued. K == 0: zeros. Repeated calls give identical bits. No workspace.
 */
fg_status fg_gemm_int4(int64_t T, int64_t N, int64_t K, int32_t group, fg_type type,
                       fg_type scale_type, const void* x, int64_t ldx, const fg_int4* w, void* out,
                       int64_t ldo, hipStream_t stream);
fg_status fg_gated_int4(int64_t T, int64_t N, int64_t K, int32_t group, fg_type type,
                        fg_type scale_type, const void* x, int64_t ldx, const fg_int4* gate,
                        const fg_int4* up, int32_t activation, void* out, int64_t ldo,
                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP32GEMM_INT4_H */
