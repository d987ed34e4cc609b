/*
 * fp32gemm_gated -- a gated feed-forward block for any number of tokens, in
 * training and serving: both projections, the activation and their product in
 * one call, what the backward pass needs kept in the block's type or in 8 bits,
 * and the gradients.
 *
 *   G = x gate^T,   U = x up^T,   h = act(G) * U
 *
 * x is T x H (tokens by hidden size), gate and up are I x H (inner by hidden
 * size), h is T x I. The block's last product, h down^T, is a plain one.
 *
 * Same conventions as fp32gemm.h and fp32gemm_fp8.h: row-major matrices with
 * leading dimensions in elements, device pointers owned by the caller, work
 * enqueued on `stream` without synchronising on the current device, errors
 * reported through fg_status / fg_last_bad_arg() / fg_last_error(), nothing
 * enqueued when an argument is rejected, no allocation.
 *
 * Rows of x, gate and up start at multiples of 16 bytes (base address and
 * leading dimension); a row's bytes up to the next multiple of 16 may be read,
 * and have no effect. All other matrices may begin at any element. No output
 * may overlap an input or another output, except as stated.
 *
 * Types. FG_TYPE_F32: products and sums in binary32. FG_TYPE_BF16: x, gate, up,
 * h, the gradients and what is kept are bfloat16; products are exact, sums and
 * the activation binary32, every output is rounded once. The gradients of G and U
 * are rounded to the block's type before they meet gate, up and x, as tensors
 * of that type would be.
 *
 * Activations are binary32 with the hardware's exponential and reciprocal: act(v) of silu
 * and gelu is off by at most (|v| + 8) 2^-23 max(|act(v)|, |v| / 4), their slopes by
 * (2 |v| + 16) 2^-23 (gelu's erf is a polynomial, off by 4e-7). Sums of the products are
 * binary32, n roundings of a sum of n terms at most; dx in binary32 is two sums, added.
 * Infinities and NaN follow the formulas: silu and gelu of -inf are NaN (-inf times 0) and
 * their slopes 0, of +inf infinite and 1.
 */
#ifndef FP32GEMM_GATED_H
#define FP32GEMM_GATED_H

#include "fp32gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How G and U are kept for the backward pass. */
typedef enum fg_save {
    FG_SAVE_NONE = 0, /* not at all */
    FG_SAVE_SAME = 1, /* in the block's type */
    FG_SAVE_E4M3 = 2  /* as e4m3 codes with a scale for each 1 x 128 block
                         (FG_BLOCK_ROW of fp32gemm_fp8.h): s = max(fl32(max|v| /
                         448), 2^-126) over the block's finite binary32 sums, the
                         code nearest to the exact v / s, ties to even; NaN and
                         infinities are NaN codes */
} fg_save;

/* One block; the numbers are the positions fg_last_bad_arg() reports. */
typedef struct fg_gated_block {
    int64_t tokens;      /* 1: T >= 0 */
    int64_t hidden;      /* 2: H >= 0 */
    int64_t inner;       /* 3: I >= 0 */
    int32_t type;        /* 4: FG_TYPE_F32 or FG_TYPE_BF16 */
    int32_t activation;  /* 5: fg_activation */
    const void* x;       /* 6: T rows of H elements */
    int64_t ldx;         /* 7 */
    const void* gate;    /* 8: I rows of H elements */
    int64_t ldgate;      /* 9 */
    const void* up;      /* 10: I rows of H elements */
    int64_t ldup;        /* 11 */
    int32_t save;        /* 12: fg_save */
    void* g;             /* 13: G as kept, T rows of I elements or codes (rows of
                                codes as in fp32gemm_fp8.h, at multiples of 16) */
    int64_t ldg;         /* 14 */
    void* u;             /* 15: U as kept */
    int64_t ldu;         /* 16 */
    float* sg;           /* 17: FG_SAVE_E4M3: G's scales, sg[b * ldsg + token] */
    int64_t ldsg;        /* 18: >= T */
    float* su;           /* 19: U's scales */
    int64_t ldsu;        /* 20: >= T */
    void* h;             /* 21: T rows of I elements */
    int64_t ldh;         /* 22: >= I */
} fg_gated_block;

/*
 * fg_gated: h, and what is kept of G and U. Arguments after the block's:
 *   23 workspace       : NULL, or device memory, 16-byte aligned, that no call
 *                        that may run at the same time uses; nothing in it is kept
 *   24 workspace_bytes : its size; fg_gated_workspace_size gives what the call can
 *                        use (less is never an error: a long sum of a small result
 *                        is split among fewer workgroups)
 *   25 stream
 * T == 0 or I == 0: FG_OK, nothing enqueued. H == 0: zeros. Repeated calls with
 * the same arguments and workspace size give identical bits.
 */
fg_status fg_gated(const fg_gated_block* block, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/* The gradients; the numbers are the positions fg_last_bad_arg() reports. */
typedef struct fg_gated_grads {
    const void* dh;      /* 23: gradient of h, T rows of I elements */
    int64_t lddh;        /* 24: >= I */
    void* dx;            /* 25: gradient of x, T rows of H elements, or NULL */
    int64_t lddx;        /* 26: >= H */
    void* dgate;         /* 27: gradient of gate, I rows of H elements, or NULL */
    int64_t lddgate;     /* 28: >= H */
    void* dup;           /* 29: gradient of up; given exactly when dgate is */
    int64_t lddup;       /* 30: >= H */
    float beta;          /* 31: dgate and dup are added to beta times what is there
                                (0: not read) */
} fg_gated_grads;

/*
 * fg_gated_backward: from dh and what fg_gated kept (block->save, g, u, sg, su,
 * here inputs; not FG_SAVE_NONE):
 *
 *   dU = dh * act(G),  dG = dh * U * act'(G),  h = act(G) * U
 *   dx = dG gate + dU up,  dgate = dG^T x + beta dgate,  dup = dU^T x + beta dup
 *
 * with G and U as they were kept. block->h is an output, or NULL: a block that
 * kept G and U need not keep h for the gradient of down. gate and up are read for
 * dx only, x for dgate and dup only (else NULL is allowed). relu' is 0 at 0.
 *   32 workspace       : device memory, 16-byte aligned, that no call that may run
 *                        at the same time uses; nothing in it is kept
 *   33 workspace_bytes : at least fg_gated_backward_min_workspace_size; more is used
 *                        up to fg_gated_backward_workspace_size
 *   34 stream
 * T == 0: the products are empty sums. Repeated calls with the same arguments and
 * workspace size give identical bits.
 */
fg_status fg_gated_backward(const fg_gated_block* block, const fg_gated_grads* grads,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes (0 if a size or the type is out of range). Host only. */
size_t fg_gated_workspace_size(int64_t tokens, int64_t hidden, int64_t inner, int32_t type);
size_t fg_gated_backward_min_workspace_size(int64_t tokens, int64_t inner, int32_t type);
size_t fg_gated_backward_workspace_size(int64_t tokens, int64_t hidden, int64_t inner,
                                        int32_t type);

#ifdef __cplusplus
}
#endif

#endif /* FP32GEMM_GATED_H */
