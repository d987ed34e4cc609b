// Quantisation to e4m3 codes with one binary32 scale per block of 128 (or
// 128 x 128) elements, in the matrix's own order and/or transposed.
//
//   s = max(fl32(max|x| / 448), 2^-126),  code = e4m3 nearest to x / s
//
// Bound by HBM: 4 or 2 bytes read and 1 written per element and order, so X is
// read once for both orders. The code is the one nearest to the exact
// quotient, which costs a handful of instructions per element:
// with s = 2^e s', s' in [1, 2), x' = x 2^-e (exact) and r = fl(1 / s'), the
// quotient q = x' r is corrected once with its exact remainder, q1 = q +
// (x' - q s') r, the binary32 value nearest to x'/s' (A. Markstein, "IA-64 and
// Elementary Functions", theorem on correctly rounded quotients). Rounding q1
// to e4m3 equals rounding x'/s' unless q1 is the middle of two codes, which
// ends in 19 zero bits; there the sign of the remainder moves q1 by one unit
// in the last place to the side the exact quotient is on.
#include "fg_device.h"
#include "fg_lowp_kernels.h"

namespace fg {
namespace {

constexpr float kTop = 448.f;

// A block's scale and what dividing by it needs.
struct Divisor {
    float f;   // 2^-e
    float s1;  // s * 2^-e, in [1, 2)
    float r;   // fl(1 / s1)
};

__device__ __forceinline__ float scale_of(float amax) {
    return fmaxf(amax / kTop, 1.17549435e-38f);
}

__device__ __forceinline__ Divisor divisor_of(float s) {
    const uint32_t u = __builtin_bit_cast(uint32_t, s);  // normal, positive, < 2^121
    Divisor d;
    d.f = __builtin_bit_cast(float, (254u << 23) - (u & 0x7F800000u));
    d.s1 = __builtin_bit_cast(float, (u & 0x007FFFFFu) | 0x3F800000u);
    d.r = 1.f / d.s1;
    return d;
}

__device__ __forceinline__ float quotient(float xf, const Divisor& d) {
    const float q = xf * d.r;
    return fmaf(fmaf(-q, d.s1, xf), d.r, q);
}

// q1 moved off the middle of two codes when the exact quotient is not there;
// a zero with x's sign, which the correction lost.
__device__ __forceinline__ float settle(float q, float xf, const Divisor& d) {
    const float rem = fmaf(-q, d.s1, xf);
    uint32_t u = __builtin_bit_cast(uint32_t, q);
    if ((u & 0x7FFFFu) == 0 && rem != 0.f)  // (a NaN's bits are not all 0)
        u += ((rem > 0.f) == (q > 0.f)) ? 1u : 0xFFFFFFFFu;
    return q == 0.f ? copysignf(0.f, xf) : __builtin_bit_cast(float, u);
}

// Codes of four elements, in one dword. d[i] divides x[i].
__device__ __forceinline__ uint32_t codes4(const f4& x, const Divisor& d0, const Divisor& d1,
                                           const Divisor& d2, const Divisor& d3) {
    const float x0 = x[0] * d0.f, x1 = x[1] * d1.f, x2 = x[2] * d2.f, x3 = x[3] * d3.f;
    float q0 = quotient(x0, d0), q1 = quotient(x1, d1), q2 = quotient(x2, d2),
          q3 = quotient(x3, d3);
    const uint32_t m0 = __builtin_bit_cast(uint32_t, q0) & 0x7FFFFu,
                   m1 = __builtin_bit_cast(uint32_t, q1) & 0x7FFFFu,
                   m2 = __builtin_bit_cast(uint32_t, q2) & 0x7FFFFu,
                   m3 = __builtin_bit_cast(uint32_t, q3) & 0x7FFFFu;
    const uint32_t a = m0 < m1 ? m0 : m1, b = m2 < m3 ? m2 : m3;
    if ((a < b ? a : b) == 0) {
        q0 = settle(q0, x0, d0);
        q1 = settle(q1, x1, d1);
        q2 = settle(q2, x2, d2);
        q3 = settle(q3, x3, d3);
    }
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q2, q3, c, true);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.f;  // NaN and infinities: 0
}

// Largest finite magnitude of four elements and m. fmaxf drops NaN by itself;
// an infinity takes the slow way.
__device__ __forceinline__ float amax4(float m, const f4& x) {
    const float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    if (a == __builtin_inff())
        return fmaxf(m, fmaxf(fmaxf(finite_abs(x[0]), finite_abs(x[1])),
                              fmaxf(finite_abs(x[2]), finite_abs(x[3]))));
    return fmaxf(m, a);
}

// Elements (row, col .. col + 3); past the matrix they read as 0.
template <bool BF16>
__device__ __forceinline__ f4 load4(const QuantParams& p, int64_t row, int col) {
    f4 v = {0.f, 0.f, 0.f, 0.f};
    if (row >= p.M || col >= p.N) return v;
    if constexpr (BF16) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx + col;
        if (p.vec && col + 4 <= p.N) {
            const uint2 u = *reinterpret_cast<const uint2*>(x);
            v[0] = __builtin_bit_cast(float, u.x << 16);
            v[1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
            v[2] = __builtin_bit_cast(float, u.y << 16);
            v[3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.N) v[i] = __builtin_bit_cast(float, (uint32_t)x[i] << 16);
        }
    } else {
        const float* x = static_cast<const float*>(p.x) + row * p.ldx + col;
        if (p.vec && col + 4 <= p.N) {
            v = *reinterpret_cast<const f4*>(x);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.N) v[i] = x[i];
        }
    }
    return v;
}

__device__ __forceinline__ void store_codes4(uint8_t* q, uint32_t c, int left) {
    if (left >= 4) {
        *reinterpret_cast<uint32_t*>(q) = c;
    } else {
        for (int i = 0; i < left; ++i) q[i] = (uint8_t)(c >> (8 * i));
    }
}

// 1 x 128 blocks, own order only: half a wave per block, 4 elements per lane,
// 32 rows by 128 columns per workgroup and step.
template <bool BF16>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantParams p) {
    const int l = threadIdx.x & 31, hw = threadIdx.x >> 5;
    const int nb = (p.N + kScaleBlock - 1) / kScaleBlock;
    const int64_t tiles = (int64_t)((p.M + 31) / 32) * nb;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row0 = t / nb * 32 + hw;
        const int b = (int)(t % nb);
        const int col = b * kScaleBlock + 4 * l;
        f4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load4<BF16>(p, row0 + 8 * i, col);
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = amax4(0.f, v[i]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], __shfl_xor(m[i], o, 64));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + 8 * i;
            const float s = scale_of(m[i]);
            const Divisor d = divisor_of(s);
            const uint32_t c = codes4(v[i], d, d, d, d);
            if (row < p.M) {
                if (col < p.N) store_codes4(p.q + row * p.ldq + col, c, p.N - col);
                if (l == 0) p.s[b * p.lds + row] = s;
            }
        }
    }
}

// A 128 x 128 tile per workgroup: half wave hw holds rows 16 hw .. 16 hw + 15,
// lane l columns 4 l .. 4 l + 3, so that a lane owns 16 consecutive bytes of
// four rows of the transposed codes; those go through LDS and leave as whole
// 128-byte rows.
template <bool BF16, bool TILE>
__global__ void __launch_bounds__(256) quant_tile_kernel(QuantParams p) {
    constexpr int kPitch = 128 + 16;
    __shared__ __attribute__((aligned(16))) uint8_t codes_t[128 * kPitch];
    __shared__ float row_part[128];
    __shared__ __attribute__((aligned(16))) float col_part[8][128];
    __shared__ float row_s[128], col_s[128];
    const int tid = threadIdx.x;
    const int l = tid & 31, hw = tid >> 5;
    const int nb = (p.N + 127) / 128, mb = (p.M + 127) / 128;
    const int64_t tiles = (int64_t)nb * mb;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int bm = (int)(t / nb), bn = (int)(t % nb);
        const int64_t row0 = (int64_t)bm * 128 + 16 * hw;
        const int col0 = bn * 128, col = col0 + 4 * l;
        f4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = load4<BF16>(p, row0 + i, col);
        f4 cm = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float m = amax4(0.f, v[i]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
            if (l == 0) row_part[16 * hw + i] = m;
#pragma unroll
            for (int j = 0; j < 4; ++j) cm[j] = fmaxf(cm[j], finite_abs(v[i][j]));
        }
        *reinterpret_cast<f4*>(&col_part[hw][4 * l]) = cm;
        __syncthreads();
        if constexpr (TILE) {
            // every thread folds the 128 row maxima (LDS broadcasts)
            float m = fmaxf(row_part[tid & 63], row_part[64 + (tid & 63)]);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
            const float s = scale_of(m);
            if (tid < 128) {
                row_s[tid] = s;
                col_s[tid] = s;
            }
            if (tid == 0) {
                if (p.q) p.s[bn * p.lds + bm] = s;
                if (p.qt) p.st[bm * p.ldst + bn] = s;
            }
        } else if (tid < 128) {
            const float s = scale_of(row_part[tid]);
            row_s[tid] = s;
            const int64_t row = (int64_t)bm * 128 + tid;
            if (p.q && row < p.M) p.s[bn * p.lds + row] = s;
        } else {
            const int c = tid - 128;
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, col_part[i][c]);
            const float s = scale_of(m);
            col_s[c] = s;
            if (p.qt && col0 + c < p.N) p.st[bm * p.ldst + col0 + c] = s;
        }
        __syncthreads();
        if (p.q) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const Divisor d = divisor_of(row_s[16 * hw + i]);
                const uint32_t c = codes4(v[i], d, d, d, d);
                if (row0 + i < p.M && col < p.N)
                    store_codes4(p.q + (row0 + i) * p.ldq + col, c, p.N - col);
            }
        }
        if (p.qt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Divisor d = divisor_of(col_s[4 * l + j]);
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f4 x = {v[4 * i][j], v[4 * i + 1][j], v[4 * i + 2][j], v[4 * i + 3][j]};
                    c[i] = codes4(x, d, d, d, d);
                }
                *reinterpret_cast<uint4*>(&codes_t[(4 * l + j) * kPitch + 16 * hw]) =
                    make_uint4(c[0], c[1], c[2], c[3]);
            }
            __syncthreads();
            const int rows_left = p.M - bm * 128;  // codes of a transposed row that exist
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = tid + 256 * i, c = u >> 3, k = (u & 7) * 16;
                const uint4 w = *reinterpret_cast<const uint4*>(&codes_t[c * kPitch + k]);
                if (col0 + c < p.N && k < rows_left) {
                    uint8_t* q = p.qt + (int64_t)(col0 + c) * p.ldqt + (int64_t)bm * 128 + k;
                    if (k + 16 <= rows_left) {
                        *reinterpret_cast<uint4*>(q) = w;
                    } else {
                        const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (k + e < rows_left) q[e] = (uint8_t)(d[e >> 2] >> (8 * (e & 3)));
                    }
                }
            }
        }
        __syncthreads();  // the next tile reuses the LDS arrays
    }
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantParams& p, hipStream_t stream) {
    const int64_t nb = ((int64_t)p.N + 127) / 128;
    constexpr int64_t kMaxGrid = 1 << 20;  // the kernels stride over the rest
    if (!p.qt && !p.tile) {
        const int64_t tiles = ((int64_t)p.M + 31) / 32 * nb;
        const dim3 g((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid));
        if (p.bf16) hipLaunchKernelGGL(quant_rows_kernel<true>, g, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL(quant_rows_kernel<false>, g, dim3(256), 0, stream, p);
    } else {
        const int64_t tiles = ((int64_t)p.M + 127) / 128 * nb;
        const dim3 g((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid));
        if (p.bf16 && p.tile)
            hipLaunchKernelGGL((quant_tile_kernel<true, true>), g, dim3(256), 0, stream, p);
        else if (p.bf16)
            hipLaunchKernelGGL((quant_tile_kernel<true, false>), g, dim3(256), 0, stream, p);
        else if (p.tile)
            hipLaunchKernelGGL((quant_tile_kernel<false, true>), g, dim3(256), 0, stream, p);
        else
            hipLaunchKernelGGL((quant_tile_kernel<false, false>), g, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace fg
