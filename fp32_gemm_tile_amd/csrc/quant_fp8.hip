// Quantisation to e4m3 codes with one binary32 scale per block of 128 (or
// 128 x 128) elements, in the matrix's own order and/or transposed.
//
//   s = max(fl32(max|x| / 448), 2^-126),  code = e4m3 nearest to x / s
//
// Bound by HBM: 4 or 2 bytes read and 1 written per element and order, so X is
// read once for both orders; next by the vector ALU, hence the few instructions
// per element. Measured: 8192 x 8192 binary32 in both orders 76 us, 5.3 TB/s, the
// vector ALU 61 % busy (148 us with an exact division per element); a row of 4096
// bfloat16 3.6 us, a launch's own time; 3001 x 2047 bfloat16 in 128 x 128 blocks both
// ways 13 us, a single round of tiles, whose chain of load, fold, division and LDS
// exchange nothing covers. The code is the one nearest to the exact quotient: with s = 2^e
// s', s' in [1, 2), and r = fl(1 / s'), q = fl(x (2^-e r)) is within two units in
// the last place of x / s. The middle of two codes ends in 19 zero bits, so q
// rounds to the code that x / s does unless it is within two units of such a
// number m; only there it is settled: the sign of the remainder 2^-e x - m s',
// one fma and so exact in its sign, says on which side of m the quotient is.
#include "fg_device.h"
#include "fg_e4m3.h"
#include "fg_lowp_kernels.h"

namespace fg {
namespace {

// Bytes of a 4 x 4 block, rows to columns.
__device__ __forceinline__ void transpose4(const uint32_t (&r)[4], uint32_t (&c)[4]) {
    const uint32_t lo01 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u);
    const uint32_t hi01 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
    const uint32_t lo23 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
    const uint32_t hi23 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
    c[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
    c[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
    c[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
    c[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
}

// Elements (row, col .. col + 3); past the matrix they read as 0. Rows may begin
// at any element: the loads are wide but ask for no more than its alignment.
template <bool BF16>
__device__ __forceinline__ f4 load4(const QuantParams& p, int64_t row, int col) {
    f4 v = {0.f, 0.f, 0.f, 0.f};
    if (row >= p.M || col >= p.N) return v;
    if constexpr (BF16) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx + col;
        if (col + 4 <= p.N) {
            uint2 u;
            __builtin_memcpy(&u, x, sizeof(u));
            v[0] = __builtin_bit_cast(float, u.x << 16);
            v[1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
            v[2] = __builtin_bit_cast(float, u.y << 16);
            v[3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (col + i < p.N) v[i] = __builtin_bit_cast(float, (uint32_t)x[i] << 16);
        }
    } else {
        const float* x = static_cast<const float*>(p.x) + row * p.ldx + col;
        if (col + 4 <= p.N) {
            __builtin_memcpy(&v, x, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
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
// 32 rows by 128 columns per workgroup.
template <bool BF16>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantParams p, int64_t first) {
    const int l = threadIdx.x & 31, hw = threadIdx.x >> 5;
    const int nb = (p.N + kScaleBlock - 1) / kScaleBlock;
    const int64_t t = first + blockIdx.x;
    const int64_t row0 = t / nb * 32 + hw;
    const int b = (int)(t % nb);
    const int col = b * kScaleBlock + 4 * l;
    f4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load4<BF16>(p, row0 + 8 * i, col);
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = max(max(magnitude(v[i][0]), magnitude(v[i][1])),
                   max(magnitude(v[i][2]), magnitude(v[i][3])));
        if (m[i] >= kInf)
            m[i] = max(max(finite_magnitude(v[i][0]), finite_magnitude(v[i][1])),
                       max(finite_magnitude(v[i][2]), finite_magnitude(v[i][3])));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], o, 64));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + 8 * i;
        const float s = scale_of(m[i]);
        const Divisor d = divisor_of(s);
        const uint32_t c = codes4(v[i], [&](int) { return d[0]; }, [&](int) { return d; });
        if (row < p.M) {
            if (col < p.N) store_codes4(p.q + row * p.ldq + col, c, p.N - col);
            if (l == 0) p.s[b * p.lds + row] = s;
        }
    }
}

// A 128 x 128 tile per workgroup of 16 waves: half wave hw holds rows 4 hw ..
// 4 hw + 3, lane l columns 4 l .. 4 l + 3, so that a lane owns a dword of four
// rows of the codes and of four rows of the transposed codes; the latter go
// through LDS and leave as whole 128-byte rows. (128 x 128 blocks have the same
// codes both ways, which are transposed in registers.) (With 4 waves and 64 elements
// per lane the unrolled code was 20 KB, and fetching it took most of the time:
// 3001 x 2047 28 us.) No loop over tiles: what it kept in registers cost a second
// workgroup on the CU (104 us at 8192 x 8192).
constexpr int kTileThreads = 1024;
template <bool BF16, bool TILE>
__global__ void __launch_bounds__(kTileThreads) quant_tile_kernel(QuantParams p, int64_t first) {
    // Transposed codes: row c (a column of the tile) at c * kPitch, its 16-byte
    // chunk k at position k ^ ((c >> 4) & 7), which spreads the lanes' dwords
    // over the banks.
    constexpr int kPitch = 128 + 16;
    __shared__ __attribute__((aligned(16))) uint8_t codes_t[128 * kPitch];
    __shared__ __attribute__((aligned(16))) uint32_t row_part[128];
    __shared__ __attribute__((aligned(16))) uint32_t col_part[16][128];
    __shared__ Divisor row_d[128], col_d[128];
    __shared__ __attribute__((aligned(16))) float row_r[128], col_r[128];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l = tid & 31, hw = tid >> 5;
    const int nb = (p.N + 127) / 128;
    const int64_t t = first + blockIdx.x;
    const int bm = (int)(t / nb), bn = (int)(t % nb);
    const int64_t row0 = (int64_t)bm * 128 + 4 * hw;
    const int col0 = bn * 128, col = col0 + 4 * l;
    f4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load4<BF16>(p, row0 + i, col);
    uint32_t rm[4], cm[4];
    auto maxima = [&](auto of) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rm[i] = max(max(of(v[i][0]), of(v[i][1])), max(of(v[i][2]), of(v[i][3])));
            cm[i] = max(max(of(v[0][i]), of(v[1][i])), max(of(v[2][i]), of(v[3][i])));
        }
    };
    maxima([](float x) { return magnitude(x); });
    if (max(max(rm[0], rm[1]), max(rm[2], rm[3])) >= kInf)
        maxima([](float x) { return finite_magnitude(x); });
    if constexpr (TILE) {
        uint32_t m = max(max(rm[0], rm[1]), max(rm[2], rm[3]));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        if (lane == 0) row_part[wave] = m;
    } else {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rm[i] = max(rm[i], (uint32_t)__shfl_xor((int)rm[i], o, 64));
        if (l == 0) *reinterpret_cast<uint4*>(&row_part[4 * hw]) = make_uint4(rm[0], rm[1], rm[2], rm[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32, 64));
        if (lane < 32)
            *reinterpret_cast<uint4*>(&col_part[wave][4 * l]) =
                make_uint4(cm[0], cm[1], cm[2], cm[3]);
    }
    __syncthreads();
    Divisor tile_d;
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 16; w += 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(&row_part[w]);
            m = max(max(m, max(u.x, u.y)), max(u.z, u.w));
        }
        const float s = scale_of(m);
        tile_d = divisor_of(s);
        if (tid == 0) {
            if (p.q) p.s[bn * p.lds + bm] = s;
            if (p.qt) p.st[bm * p.ldst + bn] = s;
        }
    } else if (tid < 256) {
        // waves 0 and 1: the rows' scales, 2 and 3: the columns'
        const bool rows = tid < 128;
        const int c = tid & 127;
        uint32_t m = rows ? row_part[c] : 0u;
        if (!rows) {
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, col_part[i][c]);
        }
        const float s = scale_of(m);
        const Divisor d = divisor_of(s);
        (rows ? row_d : col_d)[c] = d;
        (rows ? row_r : col_r)[c] = d[0];
        const int64_t row = (int64_t)bm * 128 + c;
        if (rows && p.q && row < p.M) p.s[bn * p.lds + row] = s;
        if (!rows && p.qt && col0 + c < p.N) p.st[bm * p.ldst + col0 + c] = s;
    }
    if constexpr (!TILE) __syncthreads();
    uint32_t cq[4];  // codes of row i
    if (TILE || p.q) {
        f4 r;
        if constexpr (!TILE) r = *reinterpret_cast<const f4*>(&row_r[4 * hw]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cq[i] = codes4(v[i], [&](int) { return TILE ? tile_d[0] : r[i]; },
                           [&](int) { return TILE ? tile_d : row_d[4 * hw + i]; });
            if (p.q && row0 + i < p.M && col < p.N)
                store_codes4(p.q + (row0 + i) * p.ldq + col, cq[i], p.N - col);
        }
    }
    if (p.qt) {
        uint32_t ct[4];  // codes of column j
        if constexpr (TILE) {
            transpose4(cq, ct);  // (the same scale, the same codes)
        } else {
            const f4 r = *reinterpret_cast<const f4*>(&col_r[4 * l]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 x = {v[0][j], v[1][j], v[2][j], v[3][j]};
                ct[j] = codes4(x, [&](int) { return r[j]; }, [&](int) { return col_d[4 * l + j]; });
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (4 * l + j) * kPitch + (((hw >> 2) ^ ((l >> 2) & 7)) << 4) + 4 * (hw & 3);
            *reinterpret_cast<uint32_t*>(&codes_t[at]) = ct[j];
        }
        __syncthreads();
        const int rows_left = p.M - bm * 128;  // codes of a transposed row that exist
        const int c = tid >> 3, k = (tid & 7) * 16;
        const uint4 w = *reinterpret_cast<const uint4*>(
            &codes_t[c * kPitch + (((tid & 7) ^ ((c >> 4) & 7)) << 4)]);
        if (col0 + c < p.N && k < rows_left) {
            uint8_t* q = p.qt + (int64_t)(col0 + c) * p.ldqt + (int64_t)bm * 128 + k;
            if (k + 16 <= rows_left) {
                *reinterpret_cast<uint4*>(q) = w;
            } else {
                const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    const uint32_t b = e == 0 ? d[0] : (e == 1 ? d[1] : (e == 2 ? d[2] : d[3]));
                    store_codes4(q + 4 * e, b, rows_left - k - 4 * e);
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantParams& p, hipStream_t stream) {
    const int64_t nb = ((int64_t)p.N + 127) / 128;
    constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of one launch
    const bool rows = !p.qt && !p.tile;
    const int rows_per_wg = rows ? 32 : 128, threads = rows ? 256 : kTileThreads;
    auto kernel = p.bf16 ? quant_rows_kernel<true> : quant_rows_kernel<false>;
    if (!rows && p.tile) kernel = p.bf16 ? quant_tile_kernel<true, true> : quant_tile_kernel<false, true>;
    else if (!rows) kernel = p.bf16 ? quant_tile_kernel<true, false> : quant_tile_kernel<false, false>;
    const int64_t tiles = ((int64_t)p.M + rows_per_wg - 1) / rows_per_wg * nb;
    for (int64_t first = 0; first < tiles; first += kMaxGrid) {
        const int64_t n = tiles - first < kMaxGrid ? tiles - first : kMaxGrid;
        hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(threads), 0, stream, p, first);
    }
    return hipGetLastError();
}

}  // namespace fg
