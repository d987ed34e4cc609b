// At most 64 rows of x beside 4-bit weights w = s (q - z), which are streamed once:
//
//   out = x W^T          or          out = act(x W0^T) * (x W1^T)
//
// A byte 0x0q is the e4m3 number q 2^-9 for every q from 0 to 15, so the hardware's
// conversion of e4m3 with a scale of 2^9 makes two codes values at a time, exactly.
// Sums are binary32; a binary32 x is three bfloat16 terms that hold its 24 bits (down to
// 2^-133, bfloat16's smallest number). The instruction's rows are x's, its columns W's, as
// in few_rows.h.
//
// bfloat16 x: with t = sum q x over a group of columns and X = sum x, the group's part of
// the result is s (t - z X), where X is one more matrix instruction, shared by all rows of
// W, and codes need no arithmetic. Where q is near z the two cancel, and what their roundings
// leave is relative to (q + z) |x|: less than the result's own rounding as long as no x is
// some 10^5 times the others at its zero point. Not so for binary32 x (a column 3000 times
// the others: results off by 2 10^-5), where codes become q - z first, 12 more
// instructions for eight of them (results off by 5 10^-8; one row, 8192 x 8192 in groups of
// 64: 15.4 us, and 14.1 with the sums apart; 16 rows 20.0 and 19.4, 64 rows 55 both. bfloat16:
// 11.2 and 9.9, 13.3 and 12.9, 23.5 and 24.2).
//
// A workgroup owns 16 or 32 rows of W, its waves share the columns. Everything a wave
// reads goes straight to its own part of the LDS, up to four units (128 columns) ahead: 64
// bytes of each of 16 rows of W, their scales and zero points, one value per lane, and the
// rows of x. Loads into registers in the instruction's own order give neighbouring lanes
// different rows, and the L1 answers such a load at 16 bytes a cycle instead of 64: with
// 16 binary32 rows of x it was busy three quarters of the time. The LDS also exchanges the
// dwords of W between lanes on the way (a 32-column piece of the sum has to stay within
// one group): lane (n, g) reads dword g of chunk i of row n, chunk c of row r at place c ^
// (r / 4), so that 64 lanes cover all banks evenly.
//
// Up to four rows of x: a unit of them is 8 columns per lane, which are made terms once
// and go back to the LDS; more rows have as many terms as the instructions take.
//
// Bound by memory for one row of x (8192 x 8192, 4-bit gate and up in groups of 32 with
// binary32 scales and zero points, 89 MB past the caches: 22.7 us, 3.9 TB/s; one such matrix in groups
// of 128 10.0 us, 3.4 TB/s, of which 3 us are the launch and the first trip to memory), by the
// vector unit for many: a binary32 x costs 6 instructions per element to be made terms, in
// every workgroup anew (16 rows, 8192 x 8192 in groups of 64: 19 us, 12 of them these; 64
// rows 55 us, and 24 in bfloat16).
#pragma once

#include "few_rows.h"

namespace fg {
namespace {

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
// The codes minus the row's zero point, exactly (whole numbers of at most 255), in that order.
__device__ __forceinline__ i4v codes_minus(int w, float z) {
    i4v v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const int lo = w & 0x0F0F0F0F, hi = (int)(((unsigned)w >> 4) & 0x0F0F0F0Fu);
    auto two = [&](f2 q) {
        return upper_halves(__builtin_bit_cast(uint32_t, q[0] - z), __builtin_bit_cast(uint32_t, q[1] - z));
    };
    v[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, false));
    v[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, true));
    v[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, false));
    v[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, true));
#else
    (void)w, (void)z;
#endif
    return v;
}

__device__ __forceinline__ float bf16_value(uint32_t code) {
    return __builtin_bit_cast(float, code << 16);
}

// x of 32 columns as bfloat16 terms in the order of the codes. WIDE: times 2^-20,
// for sums that are not finite otherwise.
template <bool XB, bool WIDE>
__device__ __forceinline__ void terms(const i4v* x, i4v* t) {
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
}

// Workgroup id -> place along the rows of W: consecutive ids go to the 8 XCDs in turn, and
// each gets a contiguous part, so that neighbours share an L2. A line of scales holds two
// workgroups' and one of zero points eight, and each L2 would fetch it anew.
__device__ __forceinline__ int neighbours_of(int bid, int n) {
    const int x = bid & 7, q = n >> 3, r = n & 7;
    return x * q + (x < r ? x : r) + (bid >> 3);
}

// GP 32-column pieces in a group of codes; SB: its scales are bfloat16.
template <int GP_, bool SB_>
struct Kind {
    static constexpr int GP = GP_;
    static constexpr bool SB = SB_;
};

// What a wave keeps in the LDS: UN units, the terms of one.
template <typename KIND, bool XB, int NM, int RT, int CT, int NE, int UN>
struct Stages {
    static constexpr int NG = 4 / KIND::GP;                 // groups of a unit
    static constexpr int XS = XB ? 2 : 4, SS = KIND::SB ? 2 : 4, kTerms = XB ? 1 : 3;
    static constexpr int kXRow = 128 * XS;                  // bytes of a row of x
    static constexpr int kXLoads = (NE == 1 ? 4 : 16 * CT) * kXRow / 1024;
    static constexpr int kGLoads = (NG * RT + 3) / 4;       // of scales, and of zero points, of a matrix
    static constexpr int kS = NM * RT * 1024, kZ = kS + NM * kGLoads * 256, kX = kZ + NM * kGLoads * 256;
    static constexpr int kSlot = kX + kXLoads * 1024, kLoads = NM * (RT + 2 * kGLoads) + kXLoads;
    static constexpr int kTermsAt = UN * kSlot, kWave = kTermsAt + (NE == 1 ? kTerms * 1024 : 0);
    // waves of a SIMD that the LDS has room for, and that are worth their few registers
    static constexpr int waves(int w) {
        const int room = 163840 / (w * kWave) * w / 4, want = NE == 1 && NM == 2 ? 4 : 2;
        return room < 1 ? 1 : (room < want ? room : want);
    }
};

// XB: x and out are bfloat16. NM matrices, RT tiles of 16 rows of each, NE rows of x per
// lane (rows 4 e + g, e < NE), UN units ahead, at most W waves.
template <typename KIND, bool XB, int NM, int RT, int CT, int NE, int UN, int W>
__global__ void __launch_bounds__(64 * W)
    __attribute__((amdgpu_waves_per_eu(Stages<KIND, XB, NM, RT, CT, NE, UN>::waves(W)))) int4_kernel(RowsParams p) {
    using L = Stages<KIND, XB, NM, RT, CT, NE, UN>;
    constexpr int GP = KIND::GP, NG = L::NG, XS = L::XS, SS = L::SS, kTerms = L::kTerms, kPieces = XB ? 1 : 2;
    constexpr int kXRow = L::kXRow, kXLoads = L::kXLoads, kGLoads = L::kGLoads;
    constexpr int kS = L::kS, kZ = L::kZ, kX = L::kX, kSlot = L::kSlot, kLoads = L::kLoads;
    constexpr int kTermsAt = L::kTermsAt, kWave = L::kWave;
    constexpr int kXLanes = kXRow / 16;         // lanes of a row
    constexpr bool kApart = XB;                 // sum q x and sum x, not sum (q - z) x
    static_assert((UN - 1) * kLoads < 64, "loads left in flight must fit the vmcnt field");
    static_assert(NM * RT * CT * NE * 256 <= kTermsAt, "the wave's sums take the place of its units");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kWave];

    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = neighbours_of(blockIdx.x, gridDim.x) * (16 * RT);
    const int units = (p.K + 127) / 128, per = (units + waves - 1) / waves;
    const int first = wave * per, end = first + per < units ? first + per : units;
    const int groups = (p.K + 32 * GP - 1) / (32 * GP);
    const int rows = p.N - n0 < 16 * RT ? p.N - n0 : 16 * RT;
    uint8_t* const own = lds + wave * kWave;
    const uint32_t own0 = lds_address(own);

    // Buffers over the workgroup's rows of W, their scales and zero points (none: a buffer
    // without a byte) and x: rows past the matrix read as zeros. Extents below 2^32: at
    // most 32 rows of FG_MAX_LD elements; scales' and zero points' below 2^31.
    i4v wbuf[NM], sbuf[NM], zbuf[NM];
    const uint8_t* sbase[NM];
    uint32_t wsrc[NM][RT], ssrc[NM][kGLoads], smost[NM][kGLoads], zsrc[NM][kGLoads], zmost[NM][kGLoads];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        wbuf[m] = buffer_words(p.w[m].w + (int64_t)n0 * p.w[m].ld,
                               (rows - 1) * p.w[m].ld + (((int64_t)(p.K + 1) / 2 + 15) & ~15ll));
        sbase[m] = static_cast<const uint8_t*>(p.w[m].s) + (int64_t)n0 * SS;
        sbuf[m] = buffer_words(sbase[m], ((groups - 1) * p.w[m].lds + rows) * SS);
        zbuf[m] = buffer_words(p.w[m].z + n0, p.w[m].z ? (groups - 1) * p.w[m].ldz + rows : 0);
#pragma unroll
        for (int r = 0; r < RT; ++r)
            wsrc[m][r] = (uint32_t)((16 * r + lane / 4) * p.w[m].ld) + 16u * ((lane & 3) ^ ((lane >> 4) & 3));
#pragma unroll
        for (int j = 0; j < kGLoads; ++j) {
            // value k = 4 j + g of 16 rows: group k % NG of row tile k / NG
            const int k = 4 * j + g < NG * RT ? 4 * j + g : NG * RT - 1;
            const int in = 16 * (k / NG) + n16, row = in < rows ? in : rows - 1;
            ssrc[m][j] = (uint32_t)(k % NG * p.w[m].lds + row) * SS;
            smost[m][j] = (uint32_t)((groups - 1) * p.w[m].lds + row) * SS;
            zsrc[m][j] = (uint32_t)(k % NG * p.w[m].ldz + row);
            zmost[m][j] = (uint32_t)((groups - 1) * p.w[m].ldz + row);
        }
    }
    const int64_t x_bytes = (p.T - 1) * p.ldx * XS + (((int64_t)p.K * XS + 15) & ~15ll);
    const i4v xbuf = buffer_words(p.x, x_bytes);
    uint32_t xsrc[kXLoads];
#pragma unroll
    for (int q = 0; q < kXLoads; ++q) {
        const int row = q * (64 / kXLanes) + lane / kXLanes, c = lane % kXLanes;
        xsrc[q] = (uint32_t)(row * p.ldx * XS) + 16u * (NE == 1 ? c : c ^ (row & 15));
    }

    // Unit u into a stage. (Groups past the last, where x is zero, read the last one.)
    auto fetch = [&](int u, int stage) __attribute__((always_inline)) {
        const uint32_t to = own0 + stage * kSlot;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
#pragma unroll
            for (int r = 0; r < RT; ++r) dma16(wbuf[m], to + (m * RT + r) * 1024, wsrc[m][r] + (uint32_t)u * 64);
            const uint32_t so = (uint32_t)(u * NG) * (uint32_t)(p.w[m].lds * SS);
            const uint32_t zo = (uint32_t)(u * NG) * (uint32_t)p.w[m].ldz;
#pragma unroll
            for (int j = 0; j < kGLoads; ++j) {
                const uint32_t s = ssrc[m][j] + so, z = zsrc[m][j] + zo;
                dma_element<SS>(sbuf[m], to + kS + (m * kGLoads + j) * 256, s < smost[m][j] ? s : smost[m][j]);
                dma_element<1>(zbuf[m], to + kZ + (m * kGLoads + j) * 256, z < zmost[m][j] ? z : zmost[m][j]);
            }
        }
#pragma unroll
        for (int q = 0; q < kXLoads; ++q) dma16(xbuf, to + kX + q * 1024, xsrc[q] + (uint32_t)u * kXRow);
    };

    float acc[NM][RT][CT][NE];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int e = 0; e < NE; ++e) acc[m][r][c][e] = 0.f;
    };
    clear();
    // the row of x that lane (n, g) gives to the instruction, and where it finds it
    const int t0 = NE == 1 ? n16 >> 2 : 4 * (n16 & 3) + (n16 >> 2);

    struct Unit {
        int w[NM][RT][4];
        uint32_t s[NM][RT][NG], z[NM][RT][NG];
        i4v x[CT][NE == 1 ? 1 : 4][kPieces];
    };
    const uint8_t* wat[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wat[i] = own + n16 * 64 + ((i ^ (n16 >> 2)) << 4) + 4 * g;
    auto read = [&](Unit& b, int stage) __attribute__((always_inline)) {
        const uint8_t* const at = own + stage * kSlot;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b.w[m][r][i] = *reinterpret_cast<const int*>(wat[i] + stage * kSlot + (m * RT + r) * 1024);
#pragma unroll
                for (int k = 0; k < NG; ++k) {
                    const int v = (r * NG + k) / 4 * 256 + (r * NG + k) % 4 * 64 + 4 * n16;
                    b.s[m][r][k] = *reinterpret_cast<const uint32_t*>(at + kS + m * kGLoads * 256 + v);
                    b.z[m][r][k] = *reinterpret_cast<const uint32_t*>(at + kZ + m * kGLoads * 256 + v);
                }
            }
        if constexpr (NE == 1) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
                b.x[0][0][j] = *reinterpret_cast<const i4v*>(at + kX + lane * 16 * kPieces + 16 * j);
        } else {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < kPieces; ++j)
                        b.x[c][i][j] = *reinterpret_cast<const i4v*>(
                            at + kX + (16 * c + t0) * kXRow + ((((4 * i + g) * kPieces + j) ^ t0) << 4));
        }
    };
    // What a piece adds: codes a times terms xt, whose sum is at the end of its group
    // scaled into the wave's sums.
    auto use = [&](Unit& b, int u, auto edge) __attribute__((always_inline)) {
        constexpr int kOne = 0x3F803F80;   // two bfloat16 ones
        const i4v ones = {kOne, kOne, kOne, kOne};
        const f4 zero = {0.f, 0.f, 0.f, 0.f};
        i4v* const term_at = reinterpret_cast<i4v*>(own + kTermsAt);
        if constexpr (NE == 1) {
            i4v xt[kTerms];
            if constexpr (decltype(edge)::value) {
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    b.x[0][0][j] = keep<XB>(b.x[0][0][j], p.K - u * 128 - 8 * n16 - 4 * j);
            }
            terms<XB, false>(b.x[0][0], xt);
#pragma unroll
            for (int k = 0; k < kTerms; ++k) term_at[k * 64 + g * 16 + (n16 ^ (4 * g))] = xt[k];
            asm volatile("" ::: "memory");   // (other lanes read them)
        }
        f4 t[NM][RT][CT], sum[CT];   // (sum: kApart)
        auto zero_point = [&](int m, int r, int k) { return p.w[m].z ? (float)b.z[m][r][k] : 8.f; };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool begins = i % GP == 0, ends = i % GP == GP - 1;
            i4v a[NM][RT];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    a[m][r] = kApart ? codes_to_bf16(b.w[m][r][i]) : codes_minus(b.w[m][r][i], zero_point(m, r, i / GP));
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                i4v xt[kTerms];
                if constexpr (NE == 1) {
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) xt[k] = term_at[k * 64 + t0 * 16 + ((4 * i + g) ^ (4 * t0))];
                } else {
                    if constexpr (decltype(edge)::value) {
#pragma unroll
                        for (int j = 0; j < kPieces; ++j)
                            b.x[c][i][j] = keep<XB>(b.x[c][i][j], p.K - u * 128 - 32 * i - 8 * g - 4 * j);
                    }
                    terms<XB, false>(b.x[c][i], xt);
                }
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
                    const bool fresh = begins && k == 0;
#pragma unroll
                    for (int m = 0; m < NM; ++m)
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            t[m][r][c] = mfma16<true>(xt[k], a[m][r], fresh ? zero : t[m][r][c]);
                    if constexpr (kApart) sum[c] = mfma16<true>(xt[k], ones, fresh ? zero : sum[c]);
                }
            }
            if (ends) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const uint32_t code = b.s[m][r][i / GP];
                        const float s = __builtin_bit_cast(float, KIND::SB ? code << 16 : code);
                        const float z = kApart ? zero_point(m, r, i / GP) : 0.f;
#pragma unroll
                        for (int c = 0; c < CT; ++c)
#pragma unroll
                            for (int e = 0; e < NE; ++e) {
                                float v = t[m][r][c][e];
                                if constexpr (kApart) v = fmaf(-z, sum[c][e], v);
                                acc[m][r][c][e] = fmaf(s, v, acc[m][r][c][e]);
                            }
                    }
                if constexpr (CT > 1) __builtin_amdgcn_sched_barrier(0);   // (few registers)
            }
        }
    };

    if (first < end) {
        // no branch around a load, so that each wait can count those after its own: past
        // the end the last unit comes again
        auto next = [&](int u) { return u < end ? u : end - 1; };
        const int whole_end = p.K % 128 && end == units ? end - 1 : end;
#pragma unroll
        for (int i = 0; i < UN; ++i) fetch(next(first + i), i);
        int u = first;
        Unit b;
        auto take = [&](int stage) __attribute__((always_inline)) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((UN - 1) * kLoads) : "memory");
            read(b, stage);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            fetch(next(u + UN), stage);
        };
        for (; u + UN <= whole_end;) {
#pragma unroll
            for (int i = 0; i < UN; ++i, ++u) {
                take(i);
                use(b, u, Flag<false>{});
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i, ++u) {
            if (u >= end) break;
            take(i);
            use(b, u, Flag<true>{});
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }

    // The waves' sums, joined in wave order, each in the place of the wave's units.
    float* const red = reinterpret_cast<float*>(own) + lane;
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
                    red[slot(m, r, c, e)] = acc[m][r][c][e];
                    all = fmaf(acc[m][r][c][e], 0.f, all);
                }
    // z X may be infinite or NaN where the result is not (an infinity beside other
    // columns, sums past the largest binary32): such sums are taken again with the codes
    // minus their zero points and x times 2^-20.
    if (__builtin_expect(__ballot(all != 0.f) != 0, false)) {
        const __amdgpu_buffer_rsrc_t xagain = make_rsrc_bytes(p.x, x_bytes);
        const uint32_t xoff = (uint32_t)(8 * g * XS);
        clear();
#pragma unroll 1
        for (int i = 4 * first; i < 4 * end; ++i) {   // 32-column pieces
            const int grp = i / GP < groups ? i / GP : groups - 1;
            i4v a[NM][RT];
            float s[NM][RT];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int row = 16 * r + n16 < rows ? 16 * r + n16 : rows - 1;
                    // (a row's last 16 bytes are there, no matter how many it fills)
                    int code = 0;
                    if (32 * i + 8 * g < p.K)
                        __builtin_memcpy(&code, p.w[m].w + (n0 + row) * p.w[m].ld + 16 * (int64_t)i + 4 * g, 4);
                    a[m][r] = codes_minus(code, p.w[m].z ? (float)p.w[m].z[n0 + row + grp * p.w[m].ldz] : 8.f);
                    uint32_t bits = 0;
                    __builtin_memcpy(&bits, sbase[m] + (grp * p.w[m].lds + row) * SS, SS);
                    s[m][r] = __builtin_bit_cast(float, KIND::SB ? bits << 16 : bits);
                }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                i4v x[kPieces], xt[kTerms];
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    x[j] = keep<XB>(__builtin_amdgcn_raw_buffer_load_b128(
                                        xagain, (uint32_t)((16 * c + t0) * p.ldx * XS) + xoff +
                                                    (uint32_t)i * (32 * XS) + 16 * j, 0, 0),
                                    p.K - 32 * i - 8 * g - 4 * j);
                terms<XB, true>(x, xt);
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < kTerms; ++k) v = mfma16<true>(xt[k], a[m][r], v);
#pragma unroll
                        for (int e = 0; e < NE; ++e) acc[m][r][c][e] = fmaf(s[m][r], v[e], acc[m][r][c][e]);
                    }
            }
        }
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        const float o = red[slot(m, r, c, e)];
                        if (o - o != 0.f) red[slot(m, r, c, e)] = acc[m][r][c][e] * 0x1p20f;
                    }
    }
    __syncthreads();
    const float* const sums = reinterpret_cast<const float*>(lds) + lane;
    constexpr int kEach = RT * CT * NE;
    for (int i = wave; i < kEach; i += waves) {
        float sum[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sum[m] = sums[(m * kEach + i) * 64];
            for (int v = 1; v < waves; ++v) sum[m] += sums[v * (kWave / 4) + (m * kEach + i) * 64];
        }
        const int t = 16 * (i / NE % CT) + 4 * (i % NE) + g, n = n0 + 16 * (i / (NE * CT)) + n16;
        if (t >= p.T || n >= p.N) continue;
        const float v = NM == 2 ? activate(sum[0], p.act) * sum[NM - 1] : sum[0];
        if constexpr (XB) static_cast<uint16_t*>(p.out)[t * p.ldo + n] = (uint16_t)bf16_code(v);
        else static_cast<float*>(p.out)[t * p.ldo + n] = v;
    }
}

template <typename KIND, bool XB, int NM, int RT, int CT, int NE, int UN, int W>
hipError_t launch_staged(const RowsParams& p, hipStream_t stream) {
    const int units = (p.K + 127) / 128;
    const int waves = units / 2 < 1 ? 1 : (units / 2 < W ? units / 2 : W);   // two units each at least
    const dim3 grid((unsigned)((p.N + 16 * RT - 1) / (16 * RT)));
    hipLaunchKernelGGL((int4_kernel<KIND, XB, NM, RT, CT, NE, UN, W>), grid, dim3((unsigned)(64 * waves)), 0,
                       stream, p);
    return hipGetLastError();
}

// 16 rows of each matrix to a workgroup, or 32, which share their rows of x: by the rows
// that the busiest of the 256 CUs gets. A row costs a ninth more with 16 for up to four rows of
// x, two fifths more for many. One matrix, K 4096 (8192 for N 8192), groups of 64, 16 and 32
// rows: one row of x, bfloat16, N 4096 5.2 and 6.2 us, 6144 7.3 and 6.6, 8192 11.6 and 10.4, 12288 10.3 and
// 11.1, 16384 13.9 and 12.0 (binary32 7.2 and 9.0, 10.0 and 9.3, 16.5 and 15.2, 14.5 and 16.8, 18.0 and
// 17.7); 16 rows N 1024 5.0 and 6.3, 4096 6.3 and 7.6, 6144 10.0 and 8.0, 8192 16.8 and 13.4,
// 12288 14.0 and 13.3; 64 rows in binary32 N 1024 22 and 29, 4096 26 and 31, 6144 47 and 32, 12288 71 and
// 60. Two matrices, 16 rows: N 4096 9.2 and 11.7, 8192 25 and 22 (binary32 12.6 and 15.6, 37 and
// 29); of them with up to four rows of x 32 gain nothing (N 8192 19.5 and 19.3, 12288 16.5 and 18.7), and
// with more than 32 bfloat16 rows they have no room.
template <typename KIND, bool XB, int NM>
hipError_t launch_few(const RowsParams& p, hipStream_t stream) {
    const int of16 = (p.N + 16 * 256 - 1) / (16 * 256), of32 = (p.N + 32 * 256 - 1) / (32 * 256);
    if (p.T <= 4) {
        if constexpr (NM == 1)
            if (2 * of32 * 8 <= of16 * 9) return launch_staged<KIND, XB, NM, 2, 1, 1, 4, 4>(p, stream);
        return launch_staged<KIND, XB, NM, 1, 1, 1, NM == 2 ? 2 : 4, 4>(p, stream);
    }
    const bool wide = 2 * of32 * 5 <= of16 * 7;
    if (p.T <= 16)
        return wide ? launch_staged<KIND, XB, NM, 2, 1, 4, XB ? 2 : 1, XB ? 4 : 8>(p, stream)
                    : launch_staged<KIND, XB, NM, 1, 1, 4, XB ? 2 : 1, XB ? 4 : 8>(p, stream);
    if (p.T <= 32)
        return wide ? launch_staged<KIND, XB, NM, 2, 2, 4, 1, XB ? 8 : 6>(p, stream)
                    : launch_staged<KIND, XB, NM, 1, 2, 4, 1, XB ? 8 : 6>(p, stream);
    if constexpr (!(XB && NM == 2))
        if (wide) return launch_staged<KIND, XB, NM, 2, 4, 4, 1, XB ? 8 : 4>(p, stream);
    return launch_staged<KIND, XB, NM, 1, 4, 4, 1, XB ? 8 : 4>(p, stream);
}

template <bool XB, int NM>
hipError_t launch_int4(const RowsParams& p, hipStream_t stream) {
    if (p.s_bf16) {
        if (p.group == 32) return launch_few<Kind<1, true>, XB, NM>(p, stream);
        if (p.group == 64) return launch_few<Kind<2, true>, XB, NM>(p, stream);
        return launch_few<Kind<4, true>, XB, NM>(p, stream);
    }
    if (p.group == 32) return launch_few<Kind<1, false>, XB, NM>(p, stream);
    if (p.group == 64) return launch_few<Kind<2, false>, XB, NM>(p, stream);
    return launch_few<Kind<4, false>, XB, NM>(p, stream);
}

}  // namespace
}  // namespace fg
