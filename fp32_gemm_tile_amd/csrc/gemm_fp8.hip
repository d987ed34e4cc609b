// Product of two block-scaled e4m3 matrices on the matrix cores:
//
//   C(i,j) = alpha * sum_b SA(b,i) SB(b,j) sum_{k in b} A(i,k) B(j,k) + beta C(i,j)
//
// Every block of 128 starts from zero and is added to the running binary32
// sum with one v_fma per element, scaled by SA * SB. B's rows are the
// instruction's rows and A's its columns, so a lane holds one row of A (one SA
// per block) and four consecutive columns of C, stored with one access.
//
// Two forms of the block's sum (FP8 below):
//   * binary32 C: the codes are converted to binary16, which holds them
//     exactly, and summed by v_mfma_f32_16x16x32_f16: products are exact and
//     sums binary32.
//   * bfloat16 C: v_mfma_f32_16x16x128_f8f6f4, twice the rate. It aligns the
//     products of a block to the largest and drops what lies 2^-14 below it
//     (measured: 448^2 + x keeps x = 8 and loses x = 4), so a block's sum is
//     off by about 3e-5 of its size on normal data, far below the 2^-9 of the
//     rounding to bfloat16; the sums over the blocks are binary32.
//
// Tiles of both operands go from memory straight to LDS (two stages, the next
// block in flight while this one is used). A 128-byte row of a tile is eight
// 16-byte chunks, chunk c of row r at position c ^ (r & 7), so the 16 rows
// that a wave's 128-bit LDS reads touch together fall on different banks.
// Rows past the matrix read as zero through the buffer's bound; the bytes of
// the last block past K are cleared when they are read from LDS.
#include "fg_device.h"
#include "fg_lowp_kernels.h"

namespace fg {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mfma_fp8(i8v a, i8v b) {
#if defined(__HIP_DEVICE_COMPILE__)
    const f4 z = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
#else
    (void)a, (void)b;
    return f4{};
#endif
}

// Eight codes as binary16, exactly.
__device__ __forceinline__ h8 codes_to_f16(int lo, int hi) {
    h8 v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
#else
    (void)lo, (void)hi;
#endif
    return v;
}

__device__ __forceinline__ f4 mfma_f16(h8 a, h8 b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#else
    (void)a, (void)b;
    return c;
#endif
}

// A lane's 32 codes as the operand of a block's sum.
template <bool FP8>
struct Operand {
    h8 v[4];
    __device__ __forceinline__ explicit Operand(i8v c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = codes_to_f16(c[2 * j], c[2 * j + 1]);
    }
    __device__ __forceinline__ f4 times(const Operand& o) const {
        f4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) t = mfma_f16(v[j], o.v[j], t);
        return t;
    }
};
template <>
struct Operand<true> {
    i8v v;
    __device__ __forceinline__ explicit Operand(i8v c) : v(c) {}
    __device__ __forceinline__ f4 times(const Operand& o) const { return mfma_fp8(v, o.v); }
};

// Bytes of a 16-byte chunk that are inside the matrix (left = how many).
__device__ __forceinline__ i4v keep_bytes(i4v v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int n = left - 4 * d;
        const uint32_t m = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
        v[d] &= (int)m;
    }
    return v;
}

// The lane's 32 codes of row r of a tile in LDS: chunks g and g + 4.
template <bool TAIL>
__device__ __forceinline__ i8v read_frag(const uint8_t* tile, int r, int g, int k_left) {
    const uint8_t* row = tile + r * 128;
    i4v lo = *reinterpret_cast<const i4v*>(row + ((g ^ (r & 7)) << 4));
    i4v hi = *reinterpret_cast<const i4v*>(row + (((g + 4) ^ (r & 7)) << 4));
    if constexpr (TAIL) {
        lo = keep_bytes(lo, k_left - 16 * g);
        hi = keep_bytes(hi, k_left - 64 - 16 * g);
    }
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                             off, 0, 0, 0);
#else
    (void)r, (void)lds, (void)off;
#endif
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4,
                                             off, 0, 0, 0);
#else
    (void)r, (void)lds, (void)off;
#endif
}

__device__ __forceinline__ void store_c(const Fp8Params& p, int64_t i, int64_t j, f4 acc) {
    const int n = p.N - j < 4 ? (int)(p.N - j) : 4;
    if (p.c_bf16) {
        uint16_t* c = static_cast<uint16_t*>(p.C) + i * p.ldc + j;
        f4 o = acc * p.alpha;
        if (p.beta != 0.f)
            for (int e = 0; e < n; ++e)
                o[e] += p.beta * __builtin_bit_cast(float, (uint32_t)c[e] << 16);
        if (n == 4 && p.vec_c) {
            uint2 u;
            u.x = bf16_code(o[0]) | bf16_code(o[1]) << 16;
            u.y = bf16_code(o[2]) | bf16_code(o[3]) << 16;
            *reinterpret_cast<uint2*>(c) = u;
        } else {
            for (int e = 0; e < n; ++e) c[e] = (uint16_t)bf16_code(o[e]);
        }
    } else {
        float* c = static_cast<float*>(p.C) + i * p.ldc + j;
        f4 o = acc * p.alpha;
        if (n == 4 && p.vec_c) {
            if (p.beta != 0.f) o = o + p.beta * *reinterpret_cast<const f4*>(c);
            *reinterpret_cast<f4*>(c) = o;
        } else {
            for (int e = 0; e < n; ++e) c[e] = p.beta != 0.f ? o[e] + p.beta * c[e] : o[e];
        }
    }
}

// Partial sums of slice `split`, dense M x N.
__device__ __forceinline__ void store_ws(const Fp8Params& p, int split, int64_t i, int64_t j,
                                         f4 acc) {
    float* c = p.ws + ((int64_t)split * p.M + i) * p.N + j;
    if ((p.N & 3) == 0) {
        *reinterpret_cast<f4*>(c) = acc;
    } else {
        for (int e = 0; e < 4; ++e)
            if (j + e < p.N) c[e] = acc[e];
    }
}

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

template <int BM, int BN, int WM, int WN, bool B_TILE, bool FP8>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN)) fp8_tile_kernel(Fp8Params p) {
    constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN;
    constexpr int TI = WM / 16, TJ = WN / 16;
    constexpr int kStage = (BM + BN) * 128;
    constexpr int kScales = BM + (B_TILE ? 0 : BN);
    __shared__ __attribute__((aligned(128))) uint8_t lds[2 * kStage];
    __shared__ __attribute__((aligned(16))) float scales[2 * kScales];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int wi = (wave % NWM) * WM, wj = (wave / NWM) * WN;
    const int tiles_m = (p.M + BM - 1) / BM;
    const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    const int split = blockIdx.y;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows_a = p.M - m0 < BM ? (int)(p.M - m0) : BM;
    const int rows_b = p.N - n0 < BN ? (int)(p.N - n0) : BN;
    const int kb0 = split * p.kb_per_split;
    const int kb1 = kb0 + p.kb_per_split < p.kb ? kb0 + p.kb_per_split : p.kb;

    const int64_t k16 = ((int64_t)p.K + 15) & ~15ll;
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc_bytes(p.A + m0 * p.lda, (int64_t)(rows_a - 1) * p.lda + k16);
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc_bytes(p.B + n0 * p.ldb, (int64_t)(rows_b - 1) * p.ldb + k16);
    // one wave's load: 8 rows, lane l row l / 8, chunk (l % 8) ^ (l / 8)
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t va = (uint32_t)((lane >> 3) * p.lda) + chunk;
    const uint32_t vb = (uint32_t)((lane >> 3) * p.ldb) + chunk;

    auto fetch = [&](int kb, int stage) {
        uint8_t* const s = lds + stage * kStage;
        float* const sc = scales + stage * kScales;
#pragma unroll
        for (int c = wave; c < BM / 8; c += NW)
            dma16(ra, s + c * 1024, va + (uint32_t)(c * 8 * p.lda) + (uint32_t)kb * 128u);
#pragma unroll
        for (int c = wave; c < BN / 8; c += NW)
            dma16(rb, s + BM * 128 + c * 1024, vb + (uint32_t)(c * 8 * p.ldb) + (uint32_t)kb * 128u);
        const __amdgpu_buffer_rsrc_t rsa =
            make_rsrc_bytes(p.SA + kb * p.ldsa + m0, (int64_t)rows_a * 4);
        for (int c = wave; c < BM / 64; c += NW) dma4(rsa, sc + c * 64, (uint32_t)(c * 64 + lane) * 4u);
        if constexpr (!B_TILE) {
            const __amdgpu_buffer_rsrc_t rsb =
                make_rsrc_bytes(p.SB + kb * p.ldsb + n0, (int64_t)rows_b * 4);
            for (int c = NW - 1 - wave; c < BN / 64; c += NW)
                dma4(rsb, sc + BM + c * 64, (uint32_t)(c * 64 + lane) * 4u);
        }
    };

    f4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

    auto use = [&](int kb, int stage, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        const int k_left = p.K - kb * 128;
        const uint8_t* const sa = lds + stage * kStage + wi * 128;
        const uint8_t* const sb = lds + stage * kStage + (BM + wj) * 128;
        const float* const sc = scales + stage * kScales;
        i8v a[TI];
        float s[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            a[i] = read_frag<TAIL>(sa, 16 * i + n16, g, k_left);
            s[i] = sc[wi + 16 * i + n16];
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const Operand<FP8> b(read_frag<TAIL>(sb, 16 * j + n16, g, k_left));
            f4 t[TI];
#pragma unroll
            for (int i = 0; i < TI; ++i) t[i] = b.times(Operand<FP8>(a[i]));
            if constexpr (B_TILE) {
                const int64_t jb = (n0 + wj + 16 * j) >> 7;
                const float sj = p.SB[kb * p.ldsb + (jb < (p.N + 127) >> 7 ? jb : 0)];
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    const float f = s[i] * sj;
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(f, t[i][e], acc[i][j][e]);
                }
            } else {
                const f4 sj = *reinterpret_cast<const f4*>(sc + BM + wj + 16 * j + 4 * g);
#pragma unroll
                for (int i = 0; i < TI; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = fmaf(s[i] * sj[e], t[i][e], acc[i][j][e]);
            }
        }
    };
    fetch(kb0, 0);
    for (int kb = kb0; kb < kb1; ++kb) {
        const int st = (kb - kb0) & 1;
        __builtin_amdgcn_s_waitcnt(0);  // this wave's part of stage st is in LDS
        __syncthreads();                // everyone's is, and stage st ^ 1 is read out
        if (kb + 1 < kb1) fetch(kb + 1, st ^ 1);
        if (p.K - kb * 128 >= 128) use(kb, st, Flag<false>{});
        else use(kb, st, Flag<true>{});
    }

#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int64_t ci = m0 + wi + 16 * i + n16;
        if (ci >= p.M) continue;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int64_t cj = n0 + wj + 16 * j + 4 * g;
            if (cj >= p.N) continue;
            if (p.splits > 1) store_ws(p, split, ci, cj, acc[i][j]);
            else store_c(p, ci, cj, acc[i][j]);
        }
    }
}

// C = alpha * (slice 0 + slice 1 + ...) + beta * C, slices in ascending order.
__global__ void __launch_bounds__(256) fp8_finish_kernel(Fp8Params p) {
    const int64_t per_row = ((int64_t)p.N + 3) / 4, units = per_row * p.M;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * 256) {
        const int64_t i = u / per_row, j = (u - i * per_row) * 4;
        f4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.splits; ++s) {
            const float* w = p.ws + ((int64_t)s * p.M + i) * p.N + j;
            if ((p.N & 3) == 0) {
                sum = sum + *reinterpret_cast<const f4*>(w);
            } else {
                for (int e = 0; e < 4; ++e)
                    if (j + e < p.N) sum[e] += w[e];
            }
        }
        store_c(p, i, j, sum);
    }
}

template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(bool b_tile, const Fp8Params& p, hipStream_t stream) {
    constexpr int threads = 64 * (BM / WM) * (BN / WN);
    const dim3 grid((unsigned)(((p.M + BM - 1) / BM) * (int64_t)((p.N + BN - 1) / BN)),
                    (unsigned)p.splits);
    const bool fp8 = p.c_bf16;
#define FG_LAUNCH(BT, F)                                                                       \
    hipLaunchKernelGGL((fp8_tile_kernel<BM, BN, WM, WN, BT, F>), grid, dim3(threads), 0, stream, p)
    if (b_tile && fp8) FG_LAUNCH(true, true);
    else if (b_tile) FG_LAUNCH(true, false);
    else if (fp8) FG_LAUNCH(false, true);
    else FG_LAUNCH(false, false);
#undef FG_LAUNCH
    return hipGetLastError();
}

constexpr Fp8Shape kShapes[] = {
    {64, 64, 256},
    {128, 128, 256},
};

}  // namespace

int fp8_num_shapes() { return (int)(sizeof kShapes / sizeof kShapes[0]); }
Fp8Shape fp8_shape(int shape) { return kShapes[shape]; }

hipError_t launch_gemm_fp8(int shape, bool b_tile, const Fp8Params& p, hipStream_t stream) {
    switch (shape) {
        case 0: return launch_tile<64, 64, 32, 32>(b_tile, p, stream);
        case 1: return launch_tile<128, 128, 64, 64>(b_tile, p, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_fp8_finish(const Fp8Params& p, hipStream_t stream) {
    const int64_t units = ((int64_t)p.N + 3) / 4 * p.M, wgs = (units + 255) / 256;
    hipLaunchKernelGGL(fp8_finish_kernel, dim3((unsigned)(wgs < 16384 ? wgs : 16384)), dim3(256),
                       0, stream, p);
    return hipGetLastError();
}

}  // namespace fg
