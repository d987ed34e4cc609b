/*
 * fp32gemm_moe -- a mixture-of-experts layer for a few tokens (a decode
 * step): router, top-k, the chosen experts' gated products and their weighted
 * sum, for weights in binary32, bfloat16 or block-scaled e4m3 codes.
 *
 *   logits(t,e) = sum_h x(t,h) * router(e,h)
 *   ids(t,0..k-1)     = the experts with the k largest logits, descending,
 *                       ties to the lowest expert
 *   weights(t,s)      = softmax over the k chosen logits (renormalize) or
 *                       over all of them
 *   out(t,:) = sum_s weights(t,s) * down_e (act(gate_e x(t,:)) * (up_e x(t,:))),
 *              e = ids(t,s)
 *
 * Same conventions as fp32gemm.h and fp32gemm_fp8.h.
 */
#ifndef FP32GEMM_MOE_H
#define FP32GEMM_MOE_H

#include "fp32gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FG_MOE_MAX_TOKENS 64   /* tokens of one call */
#define FG_MOE_MAX_TOP_K 16    /* experts of one token */
#define FG_MOE_MAX_EXPERTS 512 /* experts of the layer */
#define FG_MOE_MAX_DIM 65536   /* hidden and inner size */

/* The experts' matrices of one kind: expert e's is `rows` rows of `ld`
 * elements at w + e * stride. Rows start at multiples of 16 bytes (w, ld and
 * stride); a row's bytes up to the next multiple of 16 may be read, and have
 * no effect. Codes have FG_BLOCK_TILE scales, expert e's at scales +
 * e * scale_stride with leading dimension lds (NULL for the other types). */
typedef struct fg_experts {
    const void* w;
    int64_t ld;
    int64_t stride;
    const float* scales;
    int64_t lds;
    int64_t scale_stride;
} fg_experts;

/* One call; the numbers are the positions fg_last_bad_arg() reports. */
typedef struct fg_moe_layer {
    int32_t tokens;       /* 1: T, 0 .. FG_MOE_MAX_TOKENS */
    int32_t experts;      /* 2: E, 1 .. FG_MOE_MAX_EXPERTS */
    int32_t top_k;        /* 3: k, 1 .. min(E, FG_MOE_MAX_TOP_K) */
    int32_t hidden;       /* 4: H, 1 .. FG_MOE_MAX_DIM */
    int32_t inner;        /* 5: I, 1 .. FG_MOE_MAX_DIM */
    int32_t type;         /* 6: x and out: FG_TYPE_F32 or FG_TYPE_BF16 */
    int32_t weight_type;  /* 7: gate, up and down: any fg_type */
    int32_t activation;   /* 8: fg_activation (FG_ACT_SILU for the usual layer) */
    int32_t renormalize;  /* 9: 0 or 1 */
    const void* x;        /* 10: T rows of H elements */
    int64_t ldx;          /* 11: >= H */
    fg_experts gate;      /* 12: I x H each */
    fg_experts up;        /* 13: I x H each */
    fg_experts down;      /* 14: H x I each */
    const void* router;   /* 15: E rows of H elements, or NULL: ids and weights
                                 are inputs */
    int64_t ldr;          /* 16: >= H */
    int32_t router_type;  /* 17: FG_TYPE_F32 or FG_TYPE_BF16 */
    int32_t* ids;         /* 18: T x k, written with a router, else read; an id
                                 outside 0 .. E-1 is a slot that adds nothing
                                 (its weight is not used) */
    float* weights;       /* 19: T x k, written with a router, else read */
    void* out;            /* 20: T rows of H elements, must not overlap the
                                 inputs */
    int64_t ldo;          /* 21: >= H */
} fg_moe_layer;

/*
 * fg_moe: the layer on `stream`. Arguments after the layer's:
 *   22 workspace       : device memory, 16-byte aligned, that no call that may
 *                        run at the same time uses; nothing in it is kept
 *   23 workspace_bytes : at least fg_moe_workspace_size(T, k, E, H, I)
 *   24 stream
 * Products are exact and sums and activations binary32 for every type: an
 * operand that one bfloat16 does not hold is split into the three that hold its
 * 24 bits (of values below 2^-110 those down to 2^-133). Logits are summed in binary64, so near ones are not exchanged. A
 * token whose slots are all empty gets zeros. tokens == 0: FG_OK, nothing
 * enqueued. Repeated calls give identical bits. An expert chosen twice by one
 * token counts with the sum of the two weights.
 */
fg_status fg_moe(const fg_moe_layer* layer, void* workspace, size_t workspace_bytes,
                 hipStream_t stream);

/* Workspace bytes of fg_moe (0 if an argument is out of range). Host only. */
size_t fg_moe_workspace_size(int32_t tokens, int32_t top_k, int32_t experts, int32_t hidden,
                             int32_t inner);

#ifdef __cplusplus
}
#endif

#endif /* FP32GEMM_MOE_H */
