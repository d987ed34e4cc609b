// Internal interface between the host side of the gated feed-forward and 4-bit
// entry points (fg_gated_api.cpp) and their kernels. Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fg_lowp_kernels.h"

namespace fg {

enum : int32_t { SAVE_NONE = 0, SAVE_SAME = 1, SAVE_E4M3 = 2 };

// ---- a few rows of x beside weights that are streamed once -------------------

// A matrix of weights, N x K: values of x's type, or 4-bit codes with a scale (and
// a zero point, or 8) for each `group` columns of a row.
struct RowsWeights {
    const uint8_t* w;
    int64_t ld;            // bytes
    const void* s;         // S[b * lds + n]
    int64_t lds;
    const uint8_t* z;      // Z[b * ldz + n], or null
    int64_t ldz;
};
struct RowsParams {
    int32_t T, N, K;
    int32_t x_bf16;
    int32_t act;           // gated only
    int32_t group;         // 4-bit codes; 0: weights of x's type
    int32_t s_bf16;
    int32_t matrices;      // 1: out = x W^T; 2: out = act(x W0^T) * (x W1^T)
    const void* x;
    int64_t ldx;           // elements
    RowsWeights w[2];
    void* out;
    int64_t ldo;
    void* save[2];         // both products in x's type, or null
    int64_t ld_save[2];
};
// Rows of x beside weights of its type. More of them, or one tile of 32 rows: 4096 x 8192
// in bfloat16, 16 rows 33 us here and 30 in a tile, 17 rows 51 and 30; 2048 x 1408 7 and 9,
// 16 and 9; binary32 11 and 26, 29 and 26.
constexpr int kRowsMaxTokens = 16;
constexpr int kInt4MaxRows = 64;   // FG_INT4_MAX_ROWS
// launch_rows_<4-bit><bfloat16 x><matrices>, each a translation unit of few_rows.hip
hipError_t launch_rows_002(const RowsParams& p, hipStream_t stream);
hipError_t launch_rows_012(const RowsParams& p, hipStream_t stream);
hipError_t launch_rows_101(const RowsParams& p, hipStream_t stream);
hipError_t launch_rows_102(const RowsParams& p, hipStream_t stream);
hipError_t launch_rows_111(const RowsParams& p, hipStream_t stream);
hipError_t launch_rows_112(const RowsParams& p, hipStream_t stream);
inline hipError_t launch_rows(const RowsParams& p, hipStream_t stream) {
    if (p.T < 1 || p.T > (p.group ? kInt4MaxRows : kRowsMaxTokens)) return hipErrorInvalidValue;
    if (!p.group) {
        if (p.matrices != 2) return hipErrorInvalidValue;
        return p.x_bf16 ? launch_rows_012(p, stream) : launch_rows_002(p, stream);
    }
    if (p.matrices == 1) return p.x_bf16 ? launch_rows_111(p, stream) : launch_rows_101(p, stream);
    return p.x_bf16 ? launch_rows_112(p, stream) : launch_rows_102(p, stream);
}


// ---- many rows: tile kernels ---------------------------------------------------

// The three products of the gated block. Two matrices each of what differs between
// gate and up; K and the steps below count one of them.
//   FORWARD  G = A B0^T, U = A B1^T, C[0] = act(G) * U; A is T x H, B I x H
//   DX       C[0] = A0 B0 + A1 B1; A (the gradients of G and U) T x I, B I x H
//   DW       C[i] = Ai^T B0 + beta C[i]; A T x I, B0 (x) T x H
enum : int32_t { GATED_FORWARD = 0, GATED_DX = 1, GATED_DW = 2 };
constexpr int kGradRow = 128;   // rows of dG and dU are a multiple of it, and end with zeros
struct GatedTileParams {
    const void* A[2];
    const void* B[2];
    int64_t lda, ldb[2];   // elements
    int32_t M, N, K;       // rows and columns of C, length of one sum
    void* C[2];
    int64_t ldc[2];
    float beta;
    // FORWARD: what is kept of G and U (values, or codes with their scales)
    int32_t act, save;
    void* saved[2];
    int64_t ld_saved[2];
    float* scales[2];
    int64_t ld_scales[2];
    // Slices of the sum: slice s takes steps [s * per_split, (s + 1) * per_split),
    // its partial sums of matrix i are the dense M x N ws + (2 s + i) M N (DX: one
    // matrix, ws + s M N).
    int32_t steps, per_split, splits;
    float* ws;
};
struct GatedShape {
    int bm, bn;            // rows and columns of C per workgroup
    int kb;                // bytes of k per step
    int per_cu;            // workgroups that run on a CU together
    float start_us;        // of a round: one workgroup on a CU, or per_cu
    float step_us;         // of a step of one workgroup alone on its CU
    float full_us;         // of a step of per_cu workgroups
};
int gated_num_shapes(int op, bool bf16);
GatedShape gated_shape(int op, bool bf16, int shape);
hipError_t launch_gated_tile(int op, bool bf16, int shape, const GatedTileParams& p,
                             hipStream_t stream);
// dx and dgate and dup (one slice) in one launch. bfloat16: dx in one of its two smallest
// tiles and one slice, dgate and dup in tile kPairDw; each alone is a chain of latencies on a
// part of the CUs. binary32: tiles of 64 x 128.
constexpr int kPairDx32 = 4, kPairDx64 = 3, kPairDw = 1;
constexpr int kPairDxF32 = 1, kPairDwF32 = 2;
// dx's tile in bfloat16, or -1: where all tiles are at most two to a CU, the smaller if
// either leaves them so, or where dx's smallest are.
int gated_pair(int64_t T, int64_t H, int64_t I);
hipError_t launch_gated_pair(bool bf16, int dx_shape, const GatedTileParams& dx, const GatedTileParams& dw,
                             hipStream_t stream);
// What follows a launch with several slices.
hipError_t launch_gated_finish(int op, bool bf16, const GatedTileParams& p, hipStream_t stream);

// Gradients of G and U from h's: du = dh * act(g), dg = dh * u * act'(g), both T x I
// with rows of ld_d elements (a multiple of kGradRow, zeros past I), and h = act(g) * u
// (or null).
struct GatedGradParams {
    int32_t T, I, act, save;   // SAVE_SAME or SAVE_E4M3
    const void* dh;
    int64_t lddh;
    const void* saved[2];
    int64_t ld_saved[2];
    const float* scales[2];
    int64_t ld_scales[2];
    void *dg, *du;
    int64_t ld_d;
    void* h;
    int64_t ldh;
};
hipError_t launch_gated_grad(bool bf16, const GatedGradParams& p, hipStream_t stream);

}  // namespace fg
