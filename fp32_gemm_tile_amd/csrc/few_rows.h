// A few rows of x (64, or 16 beside weights of x's type) and weights that are streamed once:
//
//   out = x W^T          or          out = act(x W0^T) * (x W1^T)
//
// for weights of x's type (binary32, bfloat16) or of 4 bits, w = s (q - z).
//
// Bound by HBM: every weight is used T times only, so the weights come straight
// from memory into the registers of the wave that uses them, 16 bytes per lane,
// 64 bytes of each of 16 rows per load, the next UN units in flight while one is
// used. A workgroup owns 16 or 32 rows of W, its waves share the columns (each takes a
// contiguous part of every row) and their sums are joined through LDS in wave order.
// The products run on the matrix cores with x's rows as the instruction's rows and
// W's as its columns: a lane holds one column of out, and so one scale of each
// group, and rows 4 e + g of it (rows of x are given to the instruction in that
// order, so that up to four rows of x leave one value per lane to be scaled). x, which
// every workgroup reads, comes from the L2s.
//
// 4-bit codes. A byte 0x0q is the e4m3 number q 2^-9 for every q from 0 to 15, so the
// hardware's conversion of e4m3 with a scale of 2^9 makes two codes bfloat16 at a
// time, exactly. A 32-column piece of the sum has to stay within one group of
// columns, so the four dwords of a lane's load are exchanged between the wave's four
// 16-lane rows (a 4 x 4 transpose, two swaps each way). With t = sum q x over a group
// and X = sum x, its part of the result is s (t - z X), where X is one more matrix
// instruction, shared by all rows. Sums are binary32; a binary32 x is three bfloat16
// terms that hold its 24 bits.
#pragma once

#include <type_traits>

#include "fg_device.h"
#include "fg_gated_kernels.h"
#include "fg_lds_tile.h"

namespace fg {
namespace {

typedef unsigned u2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mfma_bf16(i4v a, i4v b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
#else
    (void)a, (void)b;
    return c;
#endif
}
__device__ __forceinline__ f4 mfma_f32(i4v a, i4v b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    const f4 fa = __builtin_bit_cast(f4, a), fb = __builtin_bit_cast(f4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[e], fb[e], c, 0, 0, 0);
#else
    (void)a, (void)b;
#endif
    return c;
}

// Rows 0-15, 16-31, 32-47 and 48-63 of the wave's lanes hold rows of a 4 x 4 matrix
// of dwords: its transpose.
__device__ __forceinline__ i4v transpose_rows(i4v v) {
#if defined(__HIP_DEVICE_COMPILE__)
    const u2v a = __builtin_amdgcn_permlane32_swap((unsigned)v[0], (unsigned)v[2], false, false);
    const u2v b = __builtin_amdgcn_permlane32_swap((unsigned)v[1], (unsigned)v[3], false, false);
    const u2v c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const u2v d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return i4v{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
#else
    return v;
#endif
}

// Eight codes as bfloat16, columns 0 2 4 6 1 3 5 7.
__device__ __forceinline__ i4v codes_to_bf16(int w) {
    i4v v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const int lo = w & 0x0F0F0F0F, hi = (int)(((unsigned)w >> 4) & 0x0F0F0F0Fu);
    v[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
    v[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
    v[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
    v[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
#else
    (void)w;
#endif
    return v;
}
// The two halves' upper 16 bits in one dword (lo in the lower half).
__device__ __forceinline__ int upper_halves(uint32_t lo, uint32_t hi) {
#if defined(__HIP_DEVICE_COMPILE__)
    return (int)__builtin_amdgcn_perm(hi, lo, 0x07060302u);
#else
    return (int)((lo >> 16) | (hi & 0xFFFF0000u));
#endif
}
__device__ __forceinline__ int lower_halves(uint32_t lo, uint32_t hi) {
#if defined(__HIP_DEVICE_COMPILE__)
    return (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u);
#else
    return (int)((lo & 0xFFFFu) | (hi << 16));
#endif
}
// The codes minus the row's zero point, exactly (whole numbers of at most 255).
__device__ __forceinline__ i4v codes_minus(int w, float z) {
    i4v v{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = i < 2 ? 4 * i : 4 * (i - 2) + 1;   // columns e and e + 2
        const float a = (float)((w >> (4 * e)) & 15) - z;
        const float b = (float)((w >> (4 * (e + 2))) & 15) - z;
        v[i] = upper_halves(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
    return v;
}

enum : int { W_F32 = 0, W_BF16 = 1, W_INT4 = 2 };

// Columns of a unit: 64 bytes of a row of weights.
template <int WT>
constexpr int kUnit = WT == W_F32 ? 16 : (WT == W_BF16 ? 32 : 128);

__device__ __forceinline__ float bf16_value(uint32_t code) {
    return __builtin_bit_cast(float, code << 16);
}

// Elements [0, left) of a 16-byte piece, zeros after them.
template <int SIZE>
__device__ __forceinline__ i4v keep(i4v v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if constexpr (SIZE == 4) {
            if (d >= left) v[d] = 0;
        } else {
            if (2 * d >= left) v[d] = 0;
            else if (2 * d + 1 >= left) v[d] &= 0xFFFF;
        }
    }
    return v;
}

// Kinds of weights: WT; GP 32-column pieces in a group of 4-bit codes; SB: its scales
// are bfloat16.
template <int WT_, int GP_ = 4, bool SB_ = false>
struct Kind {
    static constexpr int WT = WT_, GP = GP_;
    static constexpr bool SB = SB_;
};

// XB: x and out are bfloat16. NM matrices, RT tiles of 16 rows of each, CT tiles of 16
// rows of x, of which a lane has NE (the rows 4 e + g, e < NE), UN units in flight.
template <typename KIND, bool XB, int NM, int RT, int CT, int NE, int UN>
__global__ void __launch_bounds__(512) rows_kernel(RowsParams p) {
    constexpr int WT = KIND::WT, GP = KIND::GP;
    constexpr int U = kUnit<WT>;
    constexpr int kXPieces = WT == W_INT4 ? (XB ? 4 : 8) : 1;   // 16 bytes of x per unit
    constexpr int XS = XB ? 2 : 4, kXPer32 = XB ? 1 : 2;
    constexpr int kTerms = WT == W_INT4 && !XB ? 3 : 1;
    constexpr int NG = WT == W_INT4 ? 4 / GP : 1;               // groups of a unit
    // Up to four rows of x beside codes: the wave's part of x is split into its terms
    // once and kept in LDS, p.x_units units of it at a time.
    constexpr bool kXKept = WT == W_INT4 && NE == 1;
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * (16 * RT);
    const int units = (p.K + U - 1) / U;
    const int per = (units + waves - 1) / waves;
    const int first = wave * per, end = first + per < units ? first + per : units;
    // units without an edge (kept x ends with zeros, and so has none)
    const int whole_end = p.K % U && !kXKept ? (end < units ? end : units - 1) : end;

    // Buffers over the workgroup's rows of W and over x: rows past the matrix read as
    // zeros, a unit's place is a scalar offset.
    const int rows = p.N - n0 < 16 * RT ? p.N - n0 : 16 * RT;
    const int64_t w_bytes = WT == W_INT4 ? (int64_t)(p.K + 1) / 2 : (int64_t)p.K * XS;
    __amdgpu_buffer_rsrc_t wbuf[NM];
    uint32_t woff[NM][RT];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        wbuf[m] = make_rsrc_bytes(p.w[m].w + (int64_t)n0 * p.w[m].ld,
                                  (rows - 1) * p.w[m].ld + ((w_bytes + 15) & ~15ll));
#pragma unroll
        for (int r = 0; r < RT; ++r)
            woff[m][r] = (uint32_t)((16 * r + n16) * p.w[m].ld) + 16u * g;
    }
    // (extents below 2^32: at most 64 rows of FG_MAX_LD elements)
    const __amdgpu_buffer_rsrc_t xbuf =
        make_rsrc_bytes(p.x, ((p.T - 1) * p.ldx * XS + (((int64_t)p.K * XS + 15) & ~15ll)));
    uint32_t xoff[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        xoff[c] = (uint32_t)((16 * c + 4 * (n16 & 3) + (n16 >> 2)) * p.ldx * XS) +
                  (uint32_t)(WT == W_INT4 && !XB ? 32 * g : 16 * g);
    // bytes from a unit's start in a row of x to piece i, and its first column
    auto x_byte = [](int i) { return XB ? 64 * i : 128 * (i >> 1) + 16 * (i & 1); };
    auto x_col = [&](int u, int i) {
        return u * U + x_byte(i) / XS + (WT == W_INT4 || XB ? 8 : 4) * g;
    };

    // (beside several tiles of x's rows the registers hold no x ahead of its use)
    constexpr bool kXAhead = WT != W_INT4 || (CT == 1 && !kXKept);
    struct Batch {
        i4v w[NM][RT];
        i4v x[kXAhead ? CT : 1][kXPieces];
        // (as loaded: what is done to a value here is waited for here)
        typename std::conditional<KIND::SB, uint16_t, uint32_t>::type s[NM][RT][NG];
        uint8_t z[NM][RT][NG];
    };
    const int groups = WT == W_INT4 ? (p.K + 32 * GP - 1) / (32 * GP) : 0;
    constexpr int SS = KIND::SB ? 2 : 4;
    // (extents below 2^31; no zero points: a buffer without a byte)
    __amdgpu_buffer_rsrc_t sbuf[NM], zbuf[NM];
    int row[RT];   // of the workgroup's, one that is there
    if constexpr (WT == W_INT4) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sbuf[m] = make_rsrc_bytes(static_cast<const uint8_t*>(p.w[m].s) + (int64_t)n0 * SS,
                                      ((groups - 1) * p.w[m].lds + rows) * SS);
            zbuf[m] = make_rsrc_bytes(p.w[m].z + n0, p.w[m].z ? (groups - 1) * p.w[m].ldz + rows : 0);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) row[r] = 16 * r + n16 < rows ? 16 * r + n16 : rows - 1;
    }
    auto load_groups = [&](Batch& b, int u) __attribute__((always_inline)) {
        if constexpr (WT == W_INT4) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int grp = u * NG + i < groups ? u * NG + i : groups - 1;   // (past K: x is zero there)
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const uint32_t so = (uint32_t)grp * (uint32_t)p.w[m].lds * SS;
                    const uint32_t zo = (uint32_t)grp * (uint32_t)p.w[m].ldz;
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        if constexpr (KIND::SB)
                            b.s[m][r][i] = __builtin_amdgcn_raw_buffer_load_b16(sbuf[m], row[r] * 2, so, 0);
                        else
                            b.s[m][r][i] = __builtin_amdgcn_raw_buffer_load_b32(sbuf[m], row[r] * 4, so, 0);
                        b.z[m][r][i] = __builtin_amdgcn_raw_buffer_load_b8(zbuf[m], row[r], zo, 0);
                    }
                }
            }
        }
    };
    auto x_piece = [&](int u, int c, int i, bool edge) __attribute__((always_inline)) {
        // (a scalar offset is no part of the bounds check)
        const uint32_t at = u * (U * XS), in = xoff[c] + x_byte(i);
        const i4v v = edge ? __builtin_amdgcn_raw_buffer_load_b128(xbuf, in + at, 0, 0)
                           : __builtin_amdgcn_raw_buffer_load_b128(xbuf, in, at, 0);
        return edge ? keep<XS>(v, p.K - x_col(u, i)) : v;
    };
    // edge: any unit, also the one with K in it, whose elements past K are cleared.
    auto load = [&](Batch& b, int u, bool edge) __attribute__((always_inline)) {
        const int left_w = p.K - u * U - (WT == W_INT4 ? 32 : (WT == W_BF16 ? 8 : 4)) * g;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                b.w[m][r] = edge || kXKept
                    ? __builtin_amdgcn_raw_buffer_load_b128(wbuf[m], woff[m][r] + (uint32_t)u * 64, 0, 2)
                    : __builtin_amdgcn_raw_buffer_load_b128(wbuf[m], woff[m][r], u * 64, 2);
                if (WT != W_INT4 && edge) b.w[m][r] = keep<XS>(b.w[m][r], left_w);
            }
        if constexpr (kXAhead) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < kXPieces; ++i) b.x[c][i] = x_piece(u, c, i, edge);
        }
        load_groups(b, u);
    };

    // Codes: scaled sums; values: the instruction's own sums, all four rows of a lane.
    constexpr int NA = WT == W_INT4 ? NE : 4;
    float acc[NM][RT][CT][NA];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int e = 0; e < NA; ++e) acc[m][r][c][e] = 0.f;
    };
    clear();

    // x of 32 columns as bfloat16 terms in the order of the codes. WIDE: times 2^-20,
    // for sums that are not finite otherwise.
    auto terms = [&](const i4v* x, auto wide, i4v* t) __attribute__((always_inline)) {
        constexpr bool WIDE = decltype(wide)::value;
        if constexpr (XB) {
            i4v v = x[0];
            if constexpr (WIDE) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float a = bf16_value((uint32_t)v[d]) * 0x1p-20f;
                    const float b = __builtin_bit_cast(float, (uint32_t)v[d] & 0xFFFF0000u) * 0x1p-20f;
                    v[d] = upper_halves(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
                }
            }
            t[0] = i4v{lower_halves(v[0], v[1]), lower_halves(v[2], v[3]), upper_halves(v[0], v[1]),
                       upper_halves(v[2], v[3])};
        } else {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int code = x[e >> 2][e & 3];   // (a vector's element is no operand of a bit cast)
                v[e] = __builtin_bit_cast(float, code);
                if constexpr (WIDE) v[e] *= 0x1p-20f;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                auto code = [&](int e) { return __builtin_bit_cast(uint32_t, v[e]); };
                t[k] = i4v{upper_halves(code(0), code(2)), upper_halves(code(4), code(6)),
                           upper_halves(code(1), code(3)), upper_halves(code(5), code(7))};
                if (k == 2) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (what is left after the upper half, exactly)
                    float rest = v[e] - __builtin_bit_cast(float, code(e) & 0xFFFF0000u);
                    if constexpr (WIDE) rest = (code(e) & 0x7F800000u) == 0x7F800000u ? 0.f : rest;
                    v[e] = rest;
                }
            }
        }
    };

    // Kept x: 16 bytes for row t, unit u, 8 columns and term at ((t x_units + u) 16 +
    // columns / 8) kTerms + term of the wave's part.
    i4v* const keep_at = reinterpret_cast<i4v*>(red + waves * NM * RT * CT * NE * 64) +
                         wave * (p.T * p.x_units * 16 * kTerms);
    const int t0 = 4 * (n16 & 3) + (n16 >> 2);
    const i4v* const kept = keep_at + ((t0 < p.T ? t0 : 0) * p.x_units * 16 + g) * kTerms;
    int kept0 = first;   // the first unit there
    auto keep_x = [&](int u0) {
        kept0 = u0;
        constexpr int kAt = XB ? 4 : 2;   // pieces on their way at a time
        const int n = p.x_units * 16;
        for (int t = 0; t < p.T; ++t) {
            for (int k0 = lane; k0 < n; k0 += 64 * kAt) {
                i4v x[kAt][kXPer32];
#pragma unroll
                for (int q = 0; q < kAt; ++q) {
                    const int col = u0 * U + (k0 + 64 * q) * 8;
#pragma unroll
                    for (int j = 0; j < kXPer32; ++j)
                        x[q][j] = __builtin_amdgcn_raw_buffer_load_b128(
                            xbuf, k0 + 64 * q < n && col + 4 * j < p.K
                                      ? (uint32_t)(t * p.ldx * XS) + col * XS + 16 * j : 0xFFFFFFF0u, 0, 0);
                }
#pragma unroll
                for (int q = 0; q < kAt; ++q) {
                    const int k = k0 + 64 * q, col = u0 * U + k * 8;
                    i4v xt[kTerms];
#pragma unroll
                    for (int j = 0; j < kXPer32; ++j) x[q][j] = keep<XS>(x[q][j], p.K - col - 4 * j);
                    terms(x[q], Flag<false>{}, xt);
                    if (k < n) {
#pragma unroll
                        for (int j = 0; j < kTerms; ++j) keep_at[(t * n + k) * kTerms + j] = xt[j];
                    }
                }
            }
        }
    };

    auto use4 = [&](const Batch& b, int u, auto edge, auto wide) __attribute__((always_inline)) {
        constexpr bool WIDE = decltype(wide)::value;
        constexpr int kOne = 0x3F803F80;   // two bfloat16 ones
        const i4v ones = {kOne, kOne, kOne, kOne};
        const f4 zero = {0.f, 0.f, 0.f, 0.f};
        i4v w[NM][RT];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) w[m][r] = transpose_rows(b.w[m][r]);
        f4 t[NM][RT][CT], sum[CT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int grp = i / GP;
            const bool begins = i % GP == 0, ends = i % GP == GP - 1;
            i4v a[NM][RT];
            float z[NM][RT];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    z[m][r] = p.w[m].z ? (float)b.z[m][r][grp] : 8.f;
                    a[m][r] = WIDE ? codes_minus(w[m][r][i], z[m][r]) : codes_to_bf16(w[m][r][i]);
                }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                i4v xt[kTerms];
                if constexpr (kXKept && !WIDE) {
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) xt[k] = kept[((u - kept0) * 16 + i * 4) * kTerms + k];
                } else {
                    i4v x[kXPer32];
#pragma unroll
                    for (int k = 0; k < kXPer32; ++k) {
                        if constexpr (kXAhead) x[k] = b.x[c][i * kXPer32 + k];
                        else x[k] = x_piece(u, c, i * kXPer32 + k, decltype(edge)::value);
                    }
                    terms(x, wide, xt);
                }
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
                    const bool fresh = begins && k == 0;
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            t[m][r][c] = mfma_bf16(xt[k], a[m][r], fresh ? zero : t[m][r][c]);
                    if constexpr (!WIDE) sum[c] = mfma_bf16(xt[k], ones, fresh ? zero : sum[c]);
                }
            }
            if (ends) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const uint32_t code = b.s[m][r][grp];
                        const float s = __builtin_bit_cast(float, KIND::SB ? code << 16 : code);
#pragma unroll
                        for (int c = 0; c < CT; ++c)
#pragma unroll
                            for (int e = 0; e < NA; ++e) {
                                const float v = WIDE ? t[m][r][c][e]
                                                     : fmaf(-z[m][r], sum[c][e], t[m][r][c][e]);
                                acc[m][r][c][e] = fmaf(s, v, acc[m][r][c][e]);
                            }
                    }
                if constexpr (CT == 4) __builtin_amdgcn_sched_barrier(0);   // (few registers)
            }
        }
    };
    auto use = [&](const Batch& b, int u, auto edge) __attribute__((always_inline)) {
        if constexpr (WT == W_INT4) {
            use4(b, u, edge, Flag<false>{});
        } else {
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        f4 v = {acc[m][r][c][0], acc[m][r][c][1], acc[m][r][c][2], acc[m][r][c][3]};
                        v = XB ? mfma_bf16(b.x[c][0], b.w[m][r], v) : mfma_f32(b.x[c][0], b.w[m][r], v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[m][r][c][e] = v[e];
                    }
        }
    };

    // No branch around a load, so that the wait before a unit's use counts the loads
    // after it and leaves them in flight: past the end the last unit comes again.
    if (first < whole_end) {
        Batch ring[UN];
        auto next = [&](int u) { return u < whole_end ? u : whole_end - 1; };
#pragma unroll
        for (int i = 0; i < UN; ++i) load(ring[i], next(first + i), false);
        if constexpr (kXKept) keep_x(first);
        int u = first;
        for (; u + UN < whole_end; u += UN) {
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                use(ring[i], u + i, Flag<false>{});
                load(ring[i], next(u + i + UN), false);
                __builtin_amdgcn_sched_barrier(0);   // (else all units are waited for at once)
            }
            // (a multiple of UN units is kept)
            if constexpr (kXKept)
                if (__builtin_amdgcn_readfirstlane(u + UN == kept0 + p.x_units)) keep_x(u + UN);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (u + i < whole_end) use(ring[i], u + i, Flag<false>{});
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (first < end && whole_end < end) {
        Batch b;
        load(b, whole_end, true);
        use(b, whole_end, Flag<true>{});
    }

    // The waves' sums, joined in wave order.
    constexpr int kTiles = NM * RT * CT * NE;
    float* const own = red + wave * kTiles * 64 + lane;
    auto slot = [](int m, int r, int c, int e) { return (((m * RT + r) * CT + c) * NE + e) * 64; };
    float all = 0.f;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    own[slot(m, r, c, e)] = acc[m][r][c][e];
                    if constexpr (WT == W_INT4) all = fmaf(acc[m][r][c][e], 0.f, all);
                }
    if constexpr (WT == W_INT4) {
        // z X may be infinite or NaN where the result is not (an infinity beside
        // other columns, sums past the largest binary32): such sums are taken again
        // with the codes minus their zero points and x times 2^-20.
        if (__builtin_expect(__ballot(all != 0.f) != 0, false)) {
            clear();
#pragma unroll 1
            for (int u = first; u < end; ++u) {
                Batch b;
                load(b, u, true);
                use4(b, u, Flag<true>{}, Flag<true>{});
            }
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            const float o = own[slot(m, r, c, e)];
                            if (o - o != 0.f) own[slot(m, r, c, e)] = acc[m][r][c][e] * 0x1p20f;
                        }
        }
    }
    __syncthreads();
    for (int i = wave; i < RT * CT * NE; i += waves) {
        float sum[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sum[m] = red[(m * RT * CT * NE + i) * 64 + lane];
            for (int v = 1; v < waves; ++v) sum[m] += red[(v * kTiles + m * RT * CT * NE + i) * 64 + lane];
        }
        const int t = 16 * (i / NE % CT) + 4 * (i % NE) + g, n = n0 + 16 * (i / (NE * CT)) + n16;
        if (t >= p.T || n >= p.N) continue;
        auto put = [&](void* to, int64_t ld, float v) {
            if constexpr (XB) static_cast<uint16_t*>(to)[t * ld + n] = (uint16_t)bf16_code(v);
            else static_cast<float*>(to)[t * ld + n] = v;
        };
        if constexpr (NM == 2) {
            put(p.out, p.ldo, activate(sum[0], p.act) * sum[1]);
            if (p.save[0]) {
                put(p.save[0], p.ld_save[0], sum[0]);
                put(p.save[1], p.ld_save[1], sum[1]);
            }
        } else {
            put(p.out, p.ldo, sum[0]);
        }
    }
}

template <typename KIND, bool XB, int NM, int RT, int CT, int NE, int UN>
hipError_t launch(const RowsParams& p, hipStream_t stream) {
    constexpr int U = kUnit<KIND::WT>;
    const int units = (p.K + U - 1) / U;
    int waves = 8;   // two units each at least
    while (waves > 1 && waves * 2 > units) waves >>= 1;
    unsigned lds = (unsigned)(waves * NM * RT * CT * NE * 64 * 4);
    static_assert(8 * NM * RT * CT * NE * 64 * 4 <= 65536, "LDS");
    RowsParams q = p;
    if (KIND::WT == W_INT4 && NE == 1) {
        // all of a wave's x, or as many units as leave room for a second workgroup
        const int per = (units + waves - 1) / waves, unit = p.T * 256 * (XB ? 1 : 3) * waves;
        const int most = (65536 - (int)lds) / unit / UN * UN;
        q.x_units = (per + UN - 1) / UN * UN;
        if (q.x_units > most) q.x_units = most;
        lds += (unsigned)(q.x_units * unit);
    }
    const dim3 grid((unsigned)((p.N + 16 * RT - 1) / (16 * RT)));
    hipLaunchKernelGGL((rows_kernel<KIND, XB, NM, RT, CT, NE, UN>), grid, dim3((unsigned)(64 * waves)),
                       lds, stream, q);
    return hipGetLastError();
}

// Rows of W per workgroup: 32 where x costs as much as the weights (16 rows of x and
// more beside 4 bits; binary32 x, whose terms are made anew by every workgroup).
template <typename KIND, bool XB, int NM>
hipError_t launch_ct(const RowsParams& p, hipStream_t stream) {
    if constexpr (KIND::WT == W_INT4) {
        constexpr int RT = NM == 2 ? 1 : 2, UN = 2;
        if (p.T <= 4)
            return NM == 1 && p.N >= 8192 ? launch<KIND, XB, NM, RT, 1, 1, UN>(p, stream)
                                          : launch<KIND, XB, NM, 1, 1, 1, UN>(p, stream);
        if (p.T <= 16) return launch<KIND, XB, NM, RT, 1, 4, XB ? 2 : 1>(p, stream);
        if (p.T <= 32) return launch<KIND, XB, NM, RT, 2, 4, 1>(p, stream);
        return launch<KIND, XB, NM, RT, 4, 4, 1>(p, stream);
    } else {
        if (p.T <= 4) return launch<KIND, XB, NM, 1, 1, 1, 4>(p, stream);
        return launch<KIND, XB, NM, 1, 1, 4, 4>(p, stream);
    }
}

template <bool XB, int NM>
hipError_t launch_int4(const RowsParams& p, hipStream_t stream) {
    if (p.s_bf16) {
        if (p.group == 32) return launch_ct<Kind<W_INT4, 1, true>, XB, NM>(p, stream);
        if (p.group == 64) return launch_ct<Kind<W_INT4, 2, true>, XB, NM>(p, stream);
        return launch_ct<Kind<W_INT4, 4, true>, XB, NM>(p, stream);
    }
    if (p.group == 32) return launch_ct<Kind<W_INT4, 1, false>, XB, NM>(p, stream);
    if (p.group == 64) return launch_ct<Kind<W_INT4, 2, false>, XB, NM>(p, stream);
    return launch_ct<Kind<W_INT4, 4, false>, XB, NM>(p, stream);
}

}  // namespace

}  // namespace fg
