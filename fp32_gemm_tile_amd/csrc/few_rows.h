// At most 16 rows of x beside gate and up, which are streamed once:
//
//   G = x Wg^T, U = x Wu^T, H = act(G) * U
//
// for binary32 and bfloat16.
//
// Bound by HBM: every weight is used T times only, so the weights come straight from
// memory into the registers of the wave that uses them, 16 bytes per lane, 64 bytes of
// each of 16 rows per load, the next three or seven units in flight while one is used. A workgroup
// owns 8 or 16 rows of both matrices, its waves share the columns (each takes a contiguous part
// of every row) and their sums are joined through LDS in wave order. The products run on
// the matrix cores with x's rows as the instruction's rows and W's as its columns: a lane
// holds one column of H and rows 4 e + g of it (rows of x are given to the instruction in
// that order, so that up to four rows of x leave one value per lane to be joined). x,
// which every workgroup reads, comes from the L2s. Sums are binary32; binary32 products
// are those of v_mfma_f32_16x16x4_f32.
//
// One token, 4096 x 8192 in bfloat16: 26 us, 5.1 TB/s of weights; four 27 and 16 33; in
// binary32 49 us, 5.5 TB/s. 2048 x 1408 in bfloat16 6 us, most of it the launch and two
// trips to memory.
#pragma once

#include "fg_device.h"
#include "fg_gated_kernels.h"
#include "fg_mfma16.h"

namespace fg {
namespace {

// XB: x, weights and results are bfloat16. NE rows of x per lane (rows 4 e + g, e < NE).
// FOLD: 8 rows of gate and 8 of up make one tile, for twice the workgroups.
template <bool XB, int NE, bool FOLD>
__global__ void __launch_bounds__(512) rows_kernel(RowsParams p) {
    constexpr int XS = XB ? 2 : 4, U = 64 / XS;   // columns of a unit: 64 bytes of a row
    constexpr int NT = FOLD ? 1 : 2, R = FOLD ? 8 : 16;   // tiles, rows of a matrix
    constexpr int UN = FOLD ? 8 : 4;              // units in flight
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * R;
    const int units = (p.K + U - 1) / U;
    const int per = (units + waves - 1) / waves;
    const int first = wave * per, end = first + per < units ? first + per : units;
    const int whole_end = p.K % U ? (end < units ? end : units - 1) : end;   // units without an edge

    // Buffers over the workgroup's rows of W and over x: rows past the matrix read as
    // zeros, a unit's place is a scalar offset. (Extents below 2^32: 16 rows of
    // FG_MAX_LD elements.)
    const int rows = p.N - n0 < R ? p.N - n0 : R;
    const int64_t row_bytes = ((int64_t)p.K * XS + 15) & ~15ll;
    __amdgpu_buffer_rsrc_t wbuf[2];
    uint32_t woff[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        wbuf[m] = make_rsrc_bytes(p.w[m].w + (int64_t)n0 * p.w[m].ld, (rows - 1) * p.w[m].ld + row_bytes);
        woff[m] = (uint32_t)(n16 * p.w[m].ld) + 16u * g;
    }
    // (FOLD: the lane's own row, or the last one in the place of a row past it)
    const uint8_t* own_row = nullptr;
    if constexpr (FOLD) {
        const int row = n0 + ((n16 & 7) < rows ? (n16 & 7) : rows - 1);
        own_row = n16 < 8 ? p.w[0].w + row * p.w[0].ld : p.w[1].w + row * p.w[1].ld;
    }
    const __amdgpu_buffer_rsrc_t xbuf = make_rsrc_bytes(p.x, (p.T - 1) * p.ldx * XS + row_bytes);
    const uint32_t xoff = (uint32_t)((4 * (n16 & 3) + (n16 >> 2)) * p.ldx * XS) + 16u * g;

    struct Unit {
        i4v w[NT], x;
    };
    auto load = [&](Unit& b, int u) __attribute__((always_inline)) {
        if constexpr (FOLD) {
            b.w[0] = __builtin_nontemporal_load(reinterpret_cast<const i4v*>(own_row + (int64_t)u * 64 + 16 * g));
        } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                b.w[m] = __builtin_amdgcn_raw_buffer_load_b128(wbuf[m], woff[m], u * 64, 2);
        }
        b.x = __builtin_amdgcn_raw_buffer_load_b128(xbuf, xoff, u * 64, 0);
    };
    f4 acc[NT] = {};
    auto use = [&](const Unit& b) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
            acc[m] = mfma16<XB>(b.x, b.w[m], acc[m]);
    };

    // No branch around a load, so that the wait before a unit's use counts the loads
    // after it and leaves them in flight: past the end the last unit comes again.
    if (first < whole_end) {
        Unit ring[UN];
        auto next = [&](int u) { return u < whole_end ? u : whole_end - 1; };
#pragma unroll
        for (int i = 0; i < UN; ++i) load(ring[i], next(first + i));
        int u = first;
        for (; u + UN < whole_end; u += UN) {
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                use(ring[i]);
                load(ring[i], next(u + i + UN));
                __builtin_amdgcn_sched_barrier(0);   // (else all units are waited for at once)
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (u + i < whole_end) use(ring[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The unit with K in it: elements past K are cleared. (A scalar offset is no part of
    // the bounds check.)
    if (first < end && whole_end < end) {
        const uint32_t at = (uint32_t)whole_end * 64;
        const int left = p.K - whole_end * U - 16 / XS * g;
        Unit b;
        if constexpr (FOLD) {
            // (a chunk past K may be past the matrix)
            b.w[0] = keep<XB>(*reinterpret_cast<const i4v*>(own_row + (left > 0 ? at + 16 * g : 0)), left);
        } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                b.w[m] = keep<XB>(__builtin_amdgcn_raw_buffer_load_b128(wbuf[m], woff[m] + at, 0, 2), left);
        }
        b.x = keep<XB>(__builtin_amdgcn_raw_buffer_load_b128(xbuf, xoff + at, 0, 0), left);
        use(b);
    }

    // The waves' sums, joined in wave order.
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int e = 0; e < NE; ++e) red[((wave * NT + m) * NE + e) * 64 + lane] = acc[m][e];
    __syncthreads();
    for (int e = wave; e < NE; e += waves) {
        float sum[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float* const from = red + (FOLD ? e : m * NE + e) * 64 + (FOLD ? (lane & ~8) + 8 * m : lane);
            sum[m] = from[0];
            for (int v = 1; v < waves; ++v) sum[m] += from[v * (NT * NE * 64)];
        }
        if (FOLD && n16 >= 8) continue;
        const int t = 4 * e + g, n = n0 + n16;
        if (t >= p.T || n >= p.N) continue;
        auto put = [&](void* to, int64_t ld, float v) {
            if constexpr (XB) static_cast<uint16_t*>(to)[t * ld + n] = (uint16_t)bf16_code(v);
            else static_cast<float*>(to)[t * ld + n] = v;
        };
        put(p.out, p.ldo, activate(sum[0], p.act) * sum[1]);
        if (p.save[0]) {
            put(p.save[0], p.ld_save[0], sum[0]);
            put(p.save[1], p.ld_save[1], sum[1]);
        }
    }
}

template <bool XB, int NE, bool FOLD>
hipError_t launch_rows_kernel(const RowsParams& p, hipStream_t stream) {
    constexpr int U = XB ? 32 : 16;
    const int units = (p.K + U - 1) / U;
    int waves = 8;   // two units each at least
    while (waves > 1 && waves * 2 > units) waves >>= 1;
    const dim3 grid((unsigned)(FOLD ? (p.N + 7) / 8 : (p.N + 15) / 16));
    hipLaunchKernelGGL((rows_kernel<XB, NE, FOLD>), grid, dim3((unsigned)(64 * waves)),
                       (unsigned)(waves * (FOLD ? 1 : 2) * NE * 64 * 4), stream, p);
    return hipGetLastError();
}

// Eight rows of both matrices to a workgroup, or 16. Up to four tokens eight: 2048 x 1408
// in bfloat16 6.1 us and 8.0, 2048 x 5632 11.9 and 14.8, 4096 x 8192 the same. More tokens
// are a seventh more work with eight, and as many where that leaves fewer rows to the
// busiest of the 256 CUs: 16 tokens, 2048 x 1408 7.2 us and 9.6, 2048 x 5632 15.5 and 17.6,
// 4096 x 4096 20.0 and 17.5, 4096 x 8192 37.8 and 33.0.
template <bool XB>
hipError_t launch(const RowsParams& p, hipStream_t stream) {
    if (p.T <= 4) return launch_rows_kernel<XB, 1, true>(p, stream);
    const int64_t of8 = ((int64_t)p.N + 8 * 256 - 1) / (8 * 256), of16 = ((int64_t)p.N + 16 * 256 - 1) / (16 * 256);
    return 8 * of8 < 14 * of16 ? launch_rows_kernel<XB, 4, true>(p, stream)
                               : launch_rows_kernel<XB, 4, false>(p, stream);
}

}  // namespace
}  // namespace fg
