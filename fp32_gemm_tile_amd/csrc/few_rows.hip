// At most 64 rows of x beside weights that are streamed once:
//
//   out = x W^T          or          out = act(x W0^T) * (x W1^T)
//
// for weights of x's type (binary32, bfloat16) or of 4 bits, w = s (q - z).
//
// Bound by HBM: every weight is used T times only, so the weights come straight
// from memory into the registers of the wave that uses them, 16 bytes per lane,
// 64 bytes of each of 16 rows per load. A workgroup owns 16 or 32 rows of W, its waves
// share the columns (each takes a contiguous part of every row) and their sums
// are joined through LDS in wave order. The products run on the matrix cores with W's
// rows as the instruction's rows and x's as its columns: a lane then holds four
// consecutive columns of one row of out, and x, which every workgroup reads, comes
// from the L2s.
//
// 4-bit codes. A byte 0x0q is the e4m3 number q 2^-9 for every q from 0 to 15, so the
// hardware's conversion of e4m3 with a scale of 2^9 makes two codes bfloat16 at a
// time, exactly. A 32-column piece of the sum has to stay within one group of
// columns, so the four dwords of a lane's load are exchanged between the wave's four
// 16-lane rows (a 4 x 4 transpose, two swaps each way). With t = sum q x over a group
// and X = sum x, its part of the result is s (t - z X), where X is one more matrix
// instruction, shared by all rows. Sums are binary32; a binary32 x is three bfloat16
// terms that hold its 24 bits.
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

// Four scales (or as many as there are) of rows n .. n + 3.
__device__ __forceinline__ f4 scales4(const void* s, int64_t at, int left, int bf16) {
    f4 v = {0.f, 0.f, 0.f, 0.f};
    if (bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(s) + at;
        if (left >= 4) {
            uint2 u;
            __builtin_memcpy(&u, p, sizeof u);
            v = f4{bf16_value(u.x), __builtin_bit_cast(float, u.x & 0xFFFF0000u), bf16_value(u.y),
                   __builtin_bit_cast(float, u.y & 0xFFFF0000u)};
        } else {
            for (int e = 0; e < left; ++e) v[e] = bf16_value(p[e]);
        }
    } else {
        const float* p = static_cast<const float*>(s) + at;
        if (left >= 4) __builtin_memcpy(&v, p, sizeof v);
        else
            for (int e = 0; e < left; ++e) v[e] = p[e];
    }
    return v;
}
__device__ __forceinline__ f4 zeros4(const uint8_t* z, int64_t at, int left) {
    if (!z) return f4{8.f, 8.f, 8.f, 8.f};
    f4 v = {0.f, 0.f, 0.f, 0.f};
    uint32_t u = 0;
    if (left >= 4) __builtin_memcpy(&u, z + at, sizeof u);
    else
        for (int e = 0; e < left; ++e) u |= (uint32_t)z[at + e] << (8 * e);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)((u >> (8 * e)) & 0xFFu);
    return v;
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

// RT tiles of 16 rows of each matrix, CT tiles of 16 rows of x, UN units loaded
// ahead of their use.
template <int WT, bool XB, int NM, int RT, int CT, int UN>
__global__ void __launch_bounds__(512) rows_kernel(RowsParams p) {
    constexpr int U = kUnit<WT>;
    constexpr int kXPieces = WT == W_INT4 ? (XB ? 4 : 8) : 1;   // 16 bytes of x per unit
    constexpr int XS = XB ? 2 : 4;
    constexpr int kTerms = WT == W_INT4 && !XB ? 3 : 1;
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * (16 * RT);
    const int units = (p.K + U - 1) / U;
    const int per = (units + waves - 1) / waves;
    const int first = wave * per, end = first + per < units ? first + per : units;
    const int whole_end = p.K % U ? (end < units ? end : units - 1) : end;   // units without an edge

    const uint8_t* wrow[NM][RT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int n = n0 + 16 * r + n16;
            wrow[m][r] = p.w[m].w + (int64_t)(n < p.N ? n : p.N - 1) * p.w[m].ld + 16 * g;
        }
    const uint8_t* xrow[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int t = 16 * c + n16;
        xrow[c] = static_cast<const uint8_t*>(p.x) + (int64_t)(t < p.T ? t : p.T - 1) * p.ldx * XS;
    }
    // byte offset in a row of x of piece i of a unit, and its first column
    auto x_col = [&](int u, int i) {
        if constexpr (WT == W_F32) return u * 16 + 4 * g;
        else if constexpr (WT == W_BF16) return u * 32 + 8 * g;
        else if constexpr (XB) return u * 128 + 32 * i + 8 * g;
        else return u * 128 + 32 * (i >> 1) + 8 * g + 4 * (i & 1);
    };

    f4 acc[NM][RT][CT];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[m][r][c] = f4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    struct Batch {
        i4v w[NM][RT];
        i4v x[CT][kXPieces];
    };
    auto load = [&](Batch& b, int u, bool edge) __attribute__((always_inline)) {
        if (!edge) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    b.w[m][r] = __builtin_nontemporal_load(
                        reinterpret_cast<const i4v*>(wrow[m][r] + (int64_t)u * 64));
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < kXPieces; ++i)
                    b.x[c][i] = *reinterpret_cast<const i4v*>(xrow[c] + (int64_t)x_col(u, i) * XS);
            return;
        }
        // the unit with K in it: pieces past it are not read, elements cleared
        const int left_w = p.K - u * U - (WT == W_INT4 ? 32 : (WT == W_BF16 ? 8 : 4)) * g;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                i4v v = {0, 0, 0, 0};
                if (left_w > 0) v = *reinterpret_cast<const i4v*>(wrow[m][r] + (int64_t)u * 64);
                b.w[m][r] = WT == W_INT4 ? v : keep<XS>(v, left_w);
            }
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < kXPieces; ++i) {
                const int left = p.K - x_col(u, i);
                i4v v = {0, 0, 0, 0};
                if (left > 0)
                    v = *reinterpret_cast<const i4v*>(xrow[c] + (int64_t)x_col(u, i) * XS);
                b.x[c][i] = keep<XS>(v, left);
            }
    };

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

    auto use4 = [&](const Batch& b, int u, auto wide) __attribute__((always_inline)) {
        constexpr bool WIDE = decltype(wide)::value;
        constexpr int kOne = 0x3F803F80;   // two bfloat16 ones
        const i4v ones = {kOne, kOne, kOne, kOne};
        i4v w[NM][RT];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) w[m][r] = transpose_rows(b.w[m][r]);
        const int pieces = p.group >> 5;   // 32-column pieces of a group: 1, 2 or 4
        const int groups = (p.K + p.group - 1) / p.group;
        f4 t[NM][RT][CT], sum[CT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool begins = (i & (pieces - 1)) == 0, ends = (i & (pieces - 1)) == pieces - 1;
            if (begins) {
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    sum[c] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int r = 0; r < RT; ++r) t[m][r][c] = f4{0.f, 0.f, 0.f, 0.f};
                }
            }
            int grp = (u * 4 + i) / pieces;
            grp = grp < groups ? grp : groups - 1;   // (past K: x is zero there)
            i4v a[NM][RT];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    if constexpr (WIDE) {
                        const int n = n0 + 16 * r + n16 < p.N ? n0 + 16 * r + n16 : p.N - 1;
                        const float z = p.w[m].z ? (float)p.w[m].z[grp * p.w[m].ldz + n] : 8.f;
                        a[m][r] = codes_minus(w[m][r][i], z);
                    } else {
                        a[m][r] = codes_to_bf16(w[m][r][i]);
                    }
                }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                i4v xt[kTerms];
                terms(&b.x[c][i * (kXPieces / 4)], wide, xt);
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int r = 0; r < RT; ++r) t[m][r][c] = mfma_bf16(a[m][r], xt[k], t[m][r][c]);
                    if constexpr (!WIDE) sum[c] = mfma_bf16(ones, xt[k], sum[c]);
                }
            }
            if (ends) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const int n = n0 + 16 * r + 4 * g, left = p.N - n;
                        const f4 s = scales4(p.w[m].s, grp * p.w[m].lds + n, left, p.s_bf16);
                        f4 z = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (!WIDE) z = zeros4(p.w[m].z, grp * p.w[m].ldz + n, left);
#pragma unroll
                        for (int c = 0; c < CT; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float v = WIDE ? t[m][r][c][e]
                                                     : fmaf(-z[e], sum[c][e], t[m][r][c][e]);
                                acc[m][r][c][e] = fmaf(s[e], v, acc[m][r][c][e]);
                            }
                    }
            }
        }
    };
    auto use = [&](const Batch& b, int u) __attribute__((always_inline)) {
        if constexpr (WT == W_INT4) {
            use4(b, u, Flag<false>{});
        } else {
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[m][r][c] = XB ? mfma_bf16(b.w[m][r], b.x[c][0], acc[m][r][c])
                                          : mfma_f32(b.w[m][r], b.x[c][0], acc[m][r][c]);
        }
    };

    int u = first;
    for (; u + UN <= whole_end; u += UN) {
        Batch b[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) load(b[i], u + i, false);
#pragma unroll
        for (int i = 0; i < UN; ++i) use(b[i], u + i);
    }
#pragma unroll 1
    for (; u < end; ++u) {
        Batch b;
        load(b, u, u >= whole_end);
        use(b, u);
    }

    if constexpr (WT == W_INT4) {
        // z X may be infinite or NaN where the result is not (an infinity beside
        // other columns, sums past the largest binary32): such sums are taken again
        // with the codes minus their zero points and x times 2^-20.
        float all = 0.f;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) all = fmaf(acc[m][r][c][e], 0.f, all);
        if (__builtin_expect(__ballot(all != 0.f) != 0, false)) {
            f4 old[NM][RT][CT];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c) old[m][r][c] = acc[m][r][c];
            clear();
#pragma unroll 1
            for (u = first; u < end; ++u) {
                Batch b;
                load(b, u, true);
                use4(b, u, Flag<true>{});
            }
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float o = old[m][r][c][e];
                            acc[m][r][c][e] = o - o == 0.f ? o : acc[m][r][c][e] * 0x1p20f;
                        }
        }
    }

    // The waves' sums, in wave order.
    constexpr int kTiles = NM * RT * CT;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c)
                reinterpret_cast<f4*>(red)[(wave * kTiles + (m * RT + r) * CT + c) * 64 + lane] = acc[m][r][c];
    __syncthreads();
    for (int i = wave; i < RT * CT; i += waves) {
        f4 sum[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sum[m] = reinterpret_cast<const f4*>(red)[(m * RT * CT + i) * 64 + lane];
            for (int v = 1; v < waves; ++v)
                sum[m] = sum[m] + reinterpret_cast<const f4*>(red)[(v * kTiles + m * RT * CT + i) * 64 + lane];
        }
        const int t = 16 * (i % CT) + n16, n = n0 + 16 * (i / CT) + 4 * g;
        if (t >= p.T || n >= p.N) continue;
        f4 o = sum[0];
        if constexpr (NM == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = activate(sum[0][e], p.act) * sum[1][e];
        }
        auto put = [&](void* to, int64_t ld, const f4& v) {
            if (!to) return;
            const int64_t at = (int64_t)t * ld + n;
            if constexpr (XB) {
                uint16_t* q = static_cast<uint16_t*>(to) + at;
                if (n + 4 <= p.N) {
                    const uint2 w = {bf16_code(v[0]) | bf16_code(v[1]) << 16,
                                     bf16_code(v[2]) | bf16_code(v[3]) << 16};
                    __builtin_memcpy(q, &w, sizeof w);
                } else {
                    for (int e = 0; e < 3 && n + e < p.N; ++e) q[e] = (uint16_t)bf16_code(v[e]);
                }
            } else {
                float* q = static_cast<float*>(to) + at;
                if (n + 4 <= p.N) __builtin_memcpy(q, &v, sizeof v);
                else
                    for (int e = 0; e < 3 && n + e < p.N; ++e) q[e] = v[e];
            }
        };
        put(p.out, p.ldo, o);
        if constexpr (NM == 2) {
            put(p.save[0], p.ld_save[0], sum[0]);
            put(p.save[1], p.ld_save[1], sum[1]);
        }
    }
}

template <int WT, bool XB, int NM, int RT, int CT, int UN>
hipError_t launch(const RowsParams& p, hipStream_t stream) {
    const int units = (p.K + kUnit<WT> - 1) / kUnit<WT>;
    int waves = 8;
    while (waves > 1 && waves * 2 > units) waves >>= 1;
    const unsigned lds = (unsigned)(waves * NM * RT * CT * 64 * 16);
    const dim3 grid((unsigned)((p.N + 16 * RT - 1) / (16 * RT)));
    hipLaunchKernelGGL((rows_kernel<WT, XB, NM, RT, CT, UN>), grid, dim3((unsigned)(64 * waves)),
                       lds, stream, p);
    return hipGetLastError();
}

template <int WT, bool XB, int NM>
hipError_t launch_ct(const RowsParams& p, hipStream_t stream) {
    constexpr int UN = WT == W_INT4 ? 2 : 4;
    if (p.T <= 16) return launch<WT, XB, NM, 1, 1, UN>(p, stream);
    if (p.T <= 32) return launch<WT, XB, NM, 1, 2, UN / 2>(p, stream);
    return launch<WT, XB, NM, 1, 4, UN / 2>(p, stream);
}

}  // namespace

hipError_t launch_rows(const RowsParams& p, hipStream_t stream) {
    if (p.T < 1 || p.T > kRowsMaxTokens) return hipErrorInvalidValue;
    const bool two = p.matrices == 2;
    if (p.group) {
        if (p.x_bf16) return two ? launch_ct<W_INT4, true, 2>(p, stream) : launch_ct<W_INT4, true, 1>(p, stream);
        return two ? launch_ct<W_INT4, false, 2>(p, stream) : launch_ct<W_INT4, false, 1>(p, stream);
    }
    if (!two) return hipErrorInvalidValue;
    return p.x_bf16 ? launch_ct<W_BF16, true, 2>(p, stream) : launch_ct<W_F32, false, 2>(p, stream);
}

}  // namespace fg
