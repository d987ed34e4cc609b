// Internal interface between the host side of the 8-bit and mixture-of-experts
// entry points (fg_lowp_api.cpp) and their kernels. Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fg {

constexpr int kScaleBlock = 128;  // elements along k that share a scale

enum : int32_t { TYPE_F32 = 0, TYPE_BF16 = 1, TYPE_E4M3 = 2 };

// Quantisation of X (M x N) to e4m3 codes in its own order (q, s) and/or
// transposed (qt, st); null pointers leave an order out.
struct QuantParams {
    const void* x;
    int64_t ldx;
    int32_t M, N;
    uint8_t* q;
    int64_t ldq;
    float* s;
    int64_t lds;
    uint8_t* qt;
    int64_t ldqt;
    float* st;
    int64_t ldst;
    int32_t bf16;   // X is bfloat16
    int32_t tile;   // 128 x 128 blocks
};
hipError_t launch_quantize_fp8(const QuantParams& p, hipStream_t stream);

// Block-scaled product (see fp32gemm_fp8.h).
struct Fp8Params {
    const uint8_t* A;
    const uint8_t* B;
    const float* SA;
    const float* SB;
    void* C;
    int64_t lda, ldsa, ldb, ldsb, ldc;
    int32_t M, N, K;
    int32_t kb;            // 128-blocks along K
    int32_t kb_per_split;  // blocks of one slice
    int32_t splits;
    float alpha, beta;
    int32_t c_bf16;
    float* ws;             // partial sums (splits > 1): slice s at s * M * N
};
// Tile kernels' shapes: index into the table of gemm_fp8.hip.
struct Fp8Shape {
    int bm, bn;             // rows of A and of B per workgroup
    float start_us;         // of a round of 256 workgroups
    float block_us;         // of a block of K in it
    float far_us;           // at least, from beyond the L2s and one workgroup per CU
};
int fp8_num_shapes();
Fp8Shape fp8_shape(int shape);
hipError_t launch_gemm_fp8(int shape, bool b_tile, const Fp8Params& p, hipStream_t stream);
// C = alpha * sum of the p.splits slices of p.ws + beta * C (splits == 0: no
// product).
hipError_t launch_fp8_finish(const Fp8Params& p, hipStream_t stream);

// Mixture-of-experts layer (see fp32gemm_moe.h).
struct ExpertMatrix {
    const void* w;
    int64_t ld, stride;
    const float* s;
    int64_t lds, s_stride;
};
// A group of tokens that share an expert: their pairs (token * k + first slot
// that chose it) and weights (summed over the slots that did).
struct MoeGroup {
    int32_t expert, count;
    int16_t pair[16];
    float weight[16];
    int32_t unused[2];  // (whole 16-byte pieces)
};
static_assert(sizeof(MoeGroup) == 112, "copied in 16-byte pieces");
struct MoePlan {
    int32_t total_x, total_h;  // groups in the two lists
    int32_t ticket;            // top-k workgroups that have finished
};
struct MoeParams {
    int32_t T, E, k, H, I;
    int32_t x_bf16, wtype, act, renorm;
    int32_t vec_x;              // rows of x start 16-byte aligned
    const void* x;
    int64_t ldx;
    ExpertMatrix gate, up, down;
    const void* router;
    int64_t ldr;
    int32_t router_bf16, vec_r;
    int32_t* ids;
    float* weights;
    void* out;
    int64_t ldo;
    double* logits;             // T x E
    // act(gate x) * (up x) of pair (token * k + slot): rows of h_ld elements
    // (zeros past I) in planes of bfloat16 terms, or binary32 for binary32 weights
    uint16_t* h;
    int64_t h_plane, h_bytes;
    int32_t h_ld;
    // x as the experts' products read it: rows of xs_ld elements, xs_cols of them
    // (a multiple of 8; zeros past H) valid, in planes of bfloat16 terms, or
    // binary32 for binary32 weights. x itself, or made by the call (xs_made).
    void* xs;
    int64_t xs_plane, xs_bytes;
    int32_t xs_ld, xs_cols, xs_made;
    // The plan: groups of at most gx (for gate and up) and gh tokens (for down;
    // the same list when gh == gx), and upper bounds on their numbers.
    MoePlan* plan;
    MoeGroup *groups_x, *groups_h;
    int32_t gx, gh, most_x, most_h;
    // down: workgroups per tile of output rows, how many have finished, their pieces
    int32_t down_wgs;
    int32_t* tickets;
    float* pieces;
};
// Tokens in a group whose values have `terms` terms; workgroups per output tile.
int moe_group_size(int terms);
int moe_down_workgroups(int wtype, int H, int I, int most_groups);
// Router logits, top-k and the plan; prepares x too when p.xs_made is set.
hipError_t launch_moe_route(const MoeParams& p, hipStream_t stream);
// The plan, and x (a call without a router).
hipError_t launch_moe_plan(const MoeParams& p, hipStream_t stream);
hipError_t launch_moe_experts(const MoeParams& p, hipStream_t stream);

}  // namespace fg
