// Product of two block-scaled e4m3 matrices on the matrix cores:
//
//   C(i,j) = alpha * sum_b SA(b,i) SB(b,j) sum_{k in b} A(i,k) B(j,k) + beta C(i,j)
//
// Every block of 128 starts from zero and is added to the running binary32
// sum with one v_fma per element, scaled by SA * SB. B's rows are the
// instruction's rows and A's its columns, so a lane holds one row of A (one SA
// per block) and four consecutive columns of C, stored with one access.
//
// The codes are converted to bfloat16, which holds them exactly, and summed by
// v_mfma_f32_16x16x32_bf16: products are exact and sums binary32. (The fp8 matrix
// instructions have twice the rate, but align the products of a group to the
// largest and drop what lies 2^-14 below it: 448^2 + x keeps x = 8 and loses
// x = 4, and where large products cancel the rest of a block's sum is lost, which
// no rounding of C hides.)
//
// Tiles of both operands go from memory straight to LDS (two or three stages, the
// next blocks in flight while this one is used). A 128-byte row of a tile is eight
// 16-byte chunks, chunk c of row r at position c ^ (r & 7), so the 16 rows
// that a wave's 128-bit LDS reads touch together fall on different banks.
// Rows past the matrix read as zero through the buffer's bound; the bytes of
// the last block past K are cleared when they are read from LDS.
//
// Bound by the matrix cores for large results, by HBM for few rows, by the
// latency of a block (load, LDS, one instruction after the other) in between.
// Measured on one MI355X: 4096^3, bfloat16 C 125 us (1100 TFLOP/s; 65 us with the fp8
// instruction); 8192^3, binary32 C, beta = 0.5 1086 us
// (1010 TFLOP/s; the library's bfloat16 product reaches 1207, and the sums of
// blocks take a v_fma per element and block beside it); 32 x 8192 x 8192 14.0 us
// (4.9 TB/s); 517 x 2047 x 3001, binary32 C 15.8 us. (Factors that always fit and
// the vote on sums that are not finite are 1.5 to 2.5 % of these.)
#include "fg_device.h"
#include "fg_lowp_kernels.h"

namespace fg {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));

// Eight codes times kDown as bfloat16, exactly. The products' 2^-64 goes into
// their factor SA * SB as kUp, which so keeps all its bits however small it is (a
// factor below 2^-190 adds less than 2^-165); one that is infinite with it, from
// 2^64 on, leaves infinities or NaN, for which the sums are taken again.
[[maybe_unused]] constexpr float kDown = 0x1p-32f, kUp = 0x1p64f;
__device__ __forceinline__ bf8 codes_to_bf16(int lo, int hi) {
    bf8 v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kDown, false);
    const bf2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kDown, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kDown, false);
    const bf2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kDown, true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
#else
    (void)lo, (void)hi;
#endif
    return v;
}

__device__ __forceinline__ f4 mfma_bf16(bf8 a, bf8 b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    (void)a, (void)b;
    return c;
#endif
}

// A lane's 32 codes as the operand of a block's sum.
struct Operand {
    bf8 v[4];
    Operand() = default;
    __device__ __forceinline__ explicit Operand(i8v c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = codes_to_bf16(c[2 * j], c[2 * j + 1]);
    }
    __device__ __forceinline__ f4 times(const Operand& o) const {
        f4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) t = mfma_bf16(v[j], o.v[j], t);
        return t;
    }
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
__device__ __forceinline__ i8v read_frag(const uint8_t* tile, int r, int g) {
    const uint8_t* row = tile + r * 128;
    const i4v lo = *reinterpret_cast<const i4v*>(row + ((g ^ (r & 7)) << 4));
    const i4v hi = *reinterpret_cast<const i4v*>(row + (((g + 4) ^ (r & 7)) << 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Those of them that are inside K (k_left: columns of the block that are).
__device__ __forceinline__ i8v keep_codes(i8v c, int g, int k_left) {
    const i4v lo = keep_bytes(__builtin_shufflevector(c, c, 0, 1, 2, 3), k_left - 16 * g);
    const i4v hi = keep_bytes(__builtin_shufflevector(c, c, 4, 5, 6, 7), k_left - 64 - 16 * g);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Loads straight to LDS: lane l's bytes go to lds + 16 l (or 4 l). Written as
// instructions, because the compiler makes every LDS read wait for all such
// loads it knows of, also those into the stage that is not being read; the loop
// below waits for them itself. They have no result registers, and offsets past
// the buffer's end read zeros. M0 holds the LDS address (one wait state); the
// compiler warns that it does not preserve M0 over the statement, and need not: it
// writes M0 before each use of its own.
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ i4v buffer_words(const void* base, int64_t bytes) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    return i4v{(int)(uint32_t)b, (int)(uint32_t)(b >> 32) & 0xFFFF, (int)(uint32_t)bytes,
               kBufferWord3};
}
__device__ __forceinline__ void dma16(i4v r, uint32_t lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(r)
                 : "m0");
#else
    (void)r, (void)lds, (void)off;
#endif
}
__device__ __forceinline__ void dma4(i4v r, uint32_t lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(r)
                 : "m0");
#else
    (void)r, (void)lds, (void)off;
#endif
}

// Four consecutive elements of C as they are in memory; rows may begin at any
// element, so the accesses are wide but ask for no more than its alignment.
template <bool BF16>
struct Quad {
    uint32_t u[BF16 ? 2 : 4];

    static __device__ __forceinline__ uint8_t* at(const Fp8Params& p, int64_t i, int64_t j) {
        return static_cast<uint8_t*>(p.C) + (i * p.ldc + j) * (BF16 ? 2 : 4);
    }
    __device__ __forceinline__ void load(const uint8_t* c) { __builtin_memcpy(u, c, sizeof u); }
    // alpha * sum + beta * this, stored
    __device__ __forceinline__ void store(uint8_t* c, f4 sum, float alpha, float beta) {
        f4 o = sum * alpha;
        if (beta != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] += beta * __builtin_bit_cast(
                                   float, !BF16 ? u[e % (BF16 ? 2 : 4)]
                                                : (e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16));
        }
        if constexpr (BF16) {
            const b4 r = __builtin_convertvector(o, b4);
            __builtin_memcpy(c, &r, sizeof r);
        } else {
            __builtin_memcpy(c, &o, sizeof o);
        }
    }
};

template <bool BF16>
__device__ __forceinline__ void store_c(const Fp8Params& p, int64_t i, int64_t j, f4 sum) {
    uint8_t* const at = Quad<BF16>::at(p, i, j);
    Quad<BF16> q{};
    if (j + 4 <= p.N) {
        if (p.beta != 0.f) q.load(at);
        q.store(at, sum, p.alpha, p.beta);
        return;
    }
    for (int e = 0; e < 3 && j + e < p.N; ++e) {
        if constexpr (BF16) {
            uint16_t* const c = reinterpret_cast<uint16_t*>(at) + e;
            float o = sum[e] * p.alpha;
            if (p.beta != 0.f) o += p.beta * __builtin_bit_cast(float, (uint32_t)*c << 16);
            *c = (uint16_t)bf16_code(o);
        } else {
            float* const c = reinterpret_cast<float*>(at) + e;
            *c = p.beta != 0.f ? sum[e] * p.alpha + p.beta * *c : sum[e] * p.alpha;
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

// A uniform scale, through the scalar cache.
__device__ __forceinline__ float scale_at(const float* s, int64_t i) {
    return *reinterpret_cast<const __attribute__((address_space(4))) float*>(
        reinterpret_cast<uintptr_t>(s + i));
}

// Workgroup id -> output tile. Consecutive ids go to the 8 XCDs in turn; XCD x
// gets the x-th contiguous part of the tiles, numbered in bands of kBand tile
// rows, column by column inside a band, so the tiles that run together on one
// XCD share rows of A and of B in its L2.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of(int bid, int n, int tiles_m, int tiles_n, int& tm,
                                        int& tn) {
    const int x = bid & 7, q = n >> 3, r = n & 7;
    const int id = x * q + (x < r ? x : r) + (bid >> 3);
    const int per_band = kBand * tiles_n;
    const int band = id / per_band, first = band * kBand;
    const int rows = tiles_m - first < kBand ? tiles_m - first : kBand;
    const int in = id - band * per_band;
    tm = first + in % rows;
    tn = in / rows;
}

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

// KG groups of waves take the blocks of K in turn, each with its own ring of NS
// stages and its own sums, which are added in group order at the end: small
// results get enough waves per SIMD to hide one block's chain of latencies.
template <int BM, int BN, int WM, int WN, int NS, int KG, bool B_TILE, bool BF16>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN) * KG) fp8_tile_kernel(Fp8Params p) {
    constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN;  // waves of one group
    constexpr int TI = WM / 16, TJ = WN / 16;
    constexpr int kStage = (BM + BN) * 128;
    // (scales come 64 at a time)
    constexpr int kScalesA = (BM + 63) / 64 * 64, kScalesB = (BN + 63) / 64 * 64;
    constexpr int kScales = kScalesA + (B_TILE ? 0 : kScalesB);
    __shared__ __attribute__((aligned(128))) uint8_t all_lds[KG * NS * kStage];
    __shared__ __attribute__((aligned(16))) float all_scales[KG * NS * kScales];

    const int lane = threadIdx.x & 63;
    const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave_id / NW, wave = wave_id % NW;
    uint8_t* const lds = all_lds + group * NS * kStage;
    float* const scales = all_scales + group * NS * kScales;
    const int n16 = lane & 15, g = lane >> 4;
    const int wi = (wave % NWM) * WM, wj = (wave / NWM) * WN;
    int tm, tn;
    tile_of(blockIdx.x, gridDim.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
    const int split = blockIdx.y;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows_a = p.M - m0 < BM ? (int)(p.M - m0) : BM;
    const int rows_b = p.N - n0 < BN ? (int)(p.N - n0) : BN;
    const int kb0 = split * p.kb_per_split;
    const int kb1 = kb0 + p.kb_per_split < p.kb ? kb0 + p.kb_per_split : p.kb;

    const int64_t k16 = ((int64_t)p.K + 15) & ~15ll;
    // (extents below 2^32: at most 256 rows of FG_MAX_LD bytes)
    const i4v a_words = buffer_words(p.A + m0 * p.lda, (int64_t)(rows_a - 1) * p.lda + k16);
    const i4v b_words = buffer_words(p.B + n0 * p.ldb, (int64_t)(rows_b - 1) * p.ldb + k16);
    // one wave's load: 8 rows, lane l row l / 8, chunk (l % 8) ^ (l / 8)
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t va = (uint32_t)((lane >> 3) * p.lda) + chunk;
    const uint32_t vb = (uint32_t)((lane >> 3) * p.ldb) + chunk;

    static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "whole loads per wave");
    constexpr int kPartsA = BM / 8 / NW, kParts = kPartsA + BN / 8 / NW;
    constexpr int kLoads = kParts + (B_TILE ? 1 : 2);  // of one wave for one block
    static_assert((NS - 2) * kLoads < 64, "loads left in flight must fit the vmcnt field");
    const uint32_t lds0 = lds_address(lds), scales0 = lds_address(scales);
    // Block kb into a stage. Past the last block: buffers without a byte, zeros.
    // Every wave loads 64 scales of each operand, some of them twice, so that
    // all have the same number of loads in flight.
    auto fetch = [&](int kb, int stage) __attribute__((always_inline)) {
        const bool more = kb < kb1;
        const uint32_t s = lds0 + stage * kStage, sc = scales0 + stage * kScales * 4;
        const int ca = wave % (kScalesA / 64), cb = wave % (kScalesB / 64);
        dma4(buffer_words(p.SA + kb * p.ldsa + m0, more ? (int64_t)rows_a * 4 : 0), sc + ca * 256,
             (uint32_t)(ca * 64 + lane) * 4u);
        if constexpr (!B_TILE)
            dma4(buffer_words(p.SB + kb * p.ldsb + n0, more ? (int64_t)rows_b * 4 : 0),
                 sc + (kScalesA + cb * 64) * 4, (uint32_t)(cb * 64 + lane) * 4u);
        i4v ra = a_words, rb = b_words;
        if (!more) ra[2] = rb[2] = 0;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            if (q < kPartsA) {
                const int c = wave + NW * q;
                dma16(ra, s + c * 1024, va + (uint32_t)(c * 8 * p.lda + (int64_t)kb * 128));
            } else {
                const int c = wave + NW * (q - kPartsA);
                dma16(rb, s + BM * 128 + c * 1024,
                      vb + (uint32_t)(c * 8 * p.ldb + (int64_t)kb * 128));
            }
        }
    };

    f4 acc[TI][TJ];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    // B_TILE: the scale of the wave's columns (0 past the last block)
    static_assert(128 % WN == 0, "the wave's columns are in one block");
    auto tile_scale = [&](int kb) {
        if constexpr (!B_TILE) return 1.f;
        const int64_t jb = (n0 + wj) >> 7;
        const float s = scale_at(p.SB, (kb < kb1 ? kb : kb1 - 1) * p.ldsb +
                                           (jb < (p.N + 127) >> 7 ? jb : 0));
        return kb < kb1 ? s : 0.f;
    };

    // The block in stage `stage` with factors in binary64.
    auto use_wide = [&](int kb, int stage) __attribute__((always_inline)) {
        const uint8_t* const sa = lds + stage * kStage + wi * 128;
        const uint8_t* const sb = lds + stage * kStage + (BM + wj) * 128;
        const float* const sc = scales + stage * kScales;
        auto codes = [&](const uint8_t* tile, int r) {
            return Operand(keep_codes(read_frag(tile, r + n16, g), g, p.K - kb * 128));
        };
        fetch(kb + KG * (NS - 1), stage == 0 ? NS - 1 : stage - 1);
        const float tile_s = tile_scale(kb);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const Operand b = codes(sb, 16 * j);
            f4 sj = {tile_s, tile_s, tile_s, tile_s};
            if constexpr (!B_TILE)
                sj = *reinterpret_cast<const f4*>(sc + kScalesA + wj + 16 * j + 4 * g);
#pragma unroll
            for (int i = 0; i < TI; ++i) {
                asm volatile("" ::: "memory");  // (read again for each: few registers)
                __builtin_amdgcn_sched_barrier(0);
                const f4 t = b.times(codes(sa, 16 * i));
                const double si = (double)sc[wi + 16 * i + n16] * kUp;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = (float)fma(si * (double)sj[e], (double)t[e], (double)acc[i][j][e]);
            }
        }
    };

    // The block in stage `stage`: one matrix instruction after the other, column
    // tile by column tile; the sum of the one kAhead before is taken over while
    // it runs, and the codes of the next column tile are read. (The scheduler is
    // kept to this order: left to itself it lines up all reads first and runs
    // out of registers.) The group's block NS - 1 further on is fetched into the
    // stage of the block before.
    auto use = [&](int kb, int stage, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        const int k_left = p.K - kb * 128;
        const uint8_t* const sa = lds + stage * kStage + wi * 128;
        const uint8_t* const sb = lds + stage * kStage + (BM + wj) * 128;
        const float* const sc = scales + stage * kScales;
        auto codes = [&](const uint8_t* tile, int r) {
            const i8v c = read_frag(tile, r + n16, g);
            return Operand(TAIL ? keep_codes(c, g, k_left) : c);
        };
        const float tile_s = tile_scale(kb);
        float s[TI];
        Operand a[TI], b[2];
        b[0] = codes(sb, 0);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            a[i] = codes(sa, 16 * i);
            const float si = sc[wi + 16 * i + n16];
            s[i] = B_TILE ? si * kUp * tile_s : si * kUp;
        }
        constexpr int kAhead = 2, kRing = kAhead + 1, kAll = TI * TJ;
        f4 t[kRing], sj[2];
        auto add = [&](int n) {
            const int i = n % TI, j = n / TI;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = B_TILE ? s[i] : s[i] * sj[j & 1][e];
                acc[i][j][e] = fmaf(f, t[n % kRing][e], acc[i][j][e]);
            }
        };
#pragma unroll
        for (int n = 0; n < kAll; ++n) {
            const int i = n % TI, j = n / TI;
            t[n % kRing] = b[j & 1].times(a[i]);
            __builtin_amdgcn_sched_barrier(0);
            if (n >= kAhead) add(n - kAhead);
            if (i == (TI > kAhead ? kAhead : TI - 1) && j + 1 < TJ)
                b[(j + 1) & 1] = codes(sb, 16 * (j + 1));
            if (i == 0) {
                if constexpr (!B_TILE)
                    sj[j & 1] = *reinterpret_cast<const f4*>(sc + kScalesA + wj + 16 * j + 4 * g);
                if (j == 0) fetch(kb + KG * (NS - 1), stage == 0 ? NS - 1 : stage - 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int n = kAll - kAhead; n < kAll; ++n) add(n);
    };

    // The next block is in LDS for everyone (later ones may still be on their
    // way), and everyone has read the block before.
    // (A wave that is a group by itself has nobody to meet.)
    auto meet = [] {
        if constexpr (NW == 1)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 2) * kLoads) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * kLoads)
                         : "memory");
    };
    // Only the last block of K can be partial: the last round of the groups takes
    // it, outside the loop (the other groups' masks keep everything).
    const int rounds = (kb1 - kb0 + KG - 1) / KG;
    const int whole = kb1 * 128 > p.K ? rounds - 1 : rounds;
    int kb = kb0 + group, stage = 0;
#pragma unroll
    for (int d = 0; d < NS - 1; ++d) fetch(kb + KG * d, d);
    for (int r = 0; r < whole; ++r) {
        meet();
        use(kb, stage, Flag<false>{});
        stage = stage + 1 == NS ? 0 : stage + 1;
        kb += KG;
    }
    if (whole < rounds) {
        meet();
        use(kb, stage, Flag<true>{});
    }
    // Sums that are not finite are taken again with factors in binary64: by all of
    // the workgroup's waves, which load for each other.
    __shared__ int votes[NW * KG];
    f4 zero = {0.f, 0.f, 0.f, 0.f};  // (NaN where a sum is not finite)
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) zero[e] = fmaf(acc[i][j][e], 0.f, zero[e]);
    const float all = zero[0] + zero[1] + zero[2] + zero[3];
    const int again = __ballot(all != 0.f) != 0;
    auto done = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    if (lane == 0) votes[wave_id] = again;
    done();
    int any = 0;
#pragma unroll
    for (int w = 0; w < NW * KG; ++w) any |= votes[w];
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(any) != 0, false)) {
        clear();
#pragma unroll
        for (int d = 0; d < NS - 1; ++d) fetch(kb0 + group + KG * d, d);
        stage = 0;
#pragma unroll 1
        for (int r = 0; r < rounds; ++r) {
            meet();
            use_wide(kb0 + group + KG * r, stage);
            stage = stage + 1 == NS ? 0 : stage + 1;
        }
        done();
    }

    // 16 rows at a time through the waves' own parts of the LDS: the groups' sums
    // are added in order, each group taking some of the rows, and a store covers
    // consecutive elements of a row (a lane holds four of each of 16 rows).
    constexpr int kPitch = WN + 4, kLanes = WN / 4, kRows = 64 / kLanes;
    constexpr int kPart = NW * 16 * kPitch;  // floats of one group
    static_assert(KG * kPart * 4 <= KG * NS * kStage, "the stages hold the waves' rows");
    static_assert(16 % KG == 0, "rows per group");
    float* const own = reinterpret_cast<float*>(all_lds) + wave * 16 * kPitch;
    const bool plain = p.splits == 1 && n0 + wj + WN <= p.N;
    auto sync = [] {
        if constexpr (KG > 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        constexpr int kMine = 16 / KG, kTurns = (kMine + kRows - 1) / kRows;
        const int r0 = group * kMine + lane / kLanes;
        const int64_t cj = n0 + wj + (lane % kLanes) * 4;
        const bool busy = kRows <= kMine || lane / kLanes < kMine;
        const bool whole_rows = plain && m0 + wi + 16 * i + 16 <= p.M;
        // (C's old elements on their way during the exchange)
        Quad<BF16> old[kTurns] = {};
        uint8_t* const at = Quad<BF16>::at(p, m0 + wi + 16 * i + r0, cj);
        constexpr int64_t kTurn = kRows * (BF16 ? 2 : 4);
        if (whole_rows && busy && p.beta != 0.f) {
#pragma unroll
            for (int r = 0; r < kTurns; ++r) old[r].load(at + r * kTurn * p.ldc);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            *reinterpret_cast<f4*>(own + group * kPart + n16 * kPitch + 16 * j + 4 * g) = acc[i][j];
        sync();
        const float* const from = own + r0 * kPitch + (lane % kLanes) * 4;
        auto sum_at = [&](int r) {
            f4 v = *reinterpret_cast<const f4*>(from + r * kPitch);
#pragma unroll
            for (int k = 1; k < KG; ++k)
                v = v + *reinterpret_cast<const f4*>(from + k * kPart + r * kPitch);
            return v;
        };
        if (whole_rows) {
            f4 v[kTurns];
#pragma unroll
            for (int r = 0; r < kTurns; ++r) v[r] = sum_at(r * kRows);
            if (busy) {
#pragma unroll
                for (int r = 0; r < kTurns; ++r)
                    old[r].store(at + r * kTurn * p.ldc, v[r], p.alpha, p.beta);
            }
        } else {
#pragma unroll 1
            for (int r = 0; r < kTurns * kRows; r += kRows) {
                const int64_t ci = m0 + wi + 16 * i + r + r0;
                const f4 v = sum_at(r);
                if (!busy || ci >= p.M || cj >= p.N) continue;
                if (p.splits > 1) store_ws(p, split, ci, cj, v);
                else store_c<BF16>(p, ci, cj, v);
            }
        }
        sync();
    }
}

// C = alpha * (slice 0 + slice 1 + ...) + beta * C, slices in ascending order.
template <bool BF16>
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
        store_c<BF16>(p, i, j, sum);
    }
}

template <int BM, int BN, int WM, int WN, int NS, int KG>
hipError_t launch_tile(bool b_tile, const Fp8Params& p, hipStream_t stream) {
    constexpr int threads = 64 * (BM / WM) * (BN / WN) * KG;
    static_assert(threads <= 512, "the host bounds the number of tiles by it");
    const dim3 grid((unsigned)(((p.M + BM - 1) / BM) * (int64_t)((p.N + BN - 1) / BN)),
                    (unsigned)p.splits);
#define FG_LAUNCH(BT, BF)                                                                      \
    hipLaunchKernelGGL((fp8_tile_kernel<BM, BN, WM, WN, NS, KG, BT, BF>), grid, dim3(threads), 0, stream, p)
    if (b_tile && p.c_bf16) FG_LAUNCH(true, true);
    else if (p.c_bf16) FG_LAUNCH(false, true);
    else if (b_tile) FG_LAUNCH(true, false);
    else FG_LAUNCH(false, false);
#undef FG_LAUNCH
    return hipGetLastError();
}

// The tile shapes, with what one costs by estimate: microseconds for the start and
// end of a round of 256 workgroups, and for a block of K in it, and for a block
// that comes from beyond the L2s where that is more (the latency over the loads in
// flight, with one workgroup on a CU). The estimates rank, and are no more than
// that: at 25 sizes of 1 to 8192 rows, both types of C, operands from HBM, the tile
// chosen took at most 13 % more than the best one, but 6 to 45 % more than its
// estimate, which has no term for C's bytes, and 78 % more where those are most of
// the work (7984 x 6830 x 80, binary32 C).
//   The tiles of up to 64 x 32 are for few rows: many groups of K, so that the
// whole of a CU's LDS is in flight (1 x 8192 x 8192 15.5 us; 32 rows 18.0,
// 64 rows 23.7; with the 64 x 64 tile 21.2, 22.5 and 24.4).
//   The tiles between 64 x 64 and 128 x 128 save results that a smaller tile
// takes in two rounds and a larger one in less than one (binary32 C):
// 517 x 2047 x 3001 80 x 64 16.2 us, 64 x 64 20.8, 128 x 128 29.6;
// 600 x 4096 x 4096 160 x 64 29.6 us, 64 x 64 38.3, 128 x 128 37.4;
// 944 x 1675 x 5460 128 x 64 36.1 us, 80 x 64 44.8, 128 x 128 39.9.
//   A third stage at 64 x 64 costs the second workgroup on the CU (256 x 8192 x 8192
// 49 -> 65 us, 4800 x 112 x 7125 28.5, where 80 x 64 takes 24.8).
constexpr Fp8Shape kShapes[] = {
    {16, 32, 1.5f, 0.074f, 0.f},
    {32, 32, 2.5f, 0.086f, 0.f},
    {64, 32, 3.0f, 0.185f, 0.f},
    {64, 64, 1.5f, 0.31f, 0.45f},
    {80, 64, 3.4f, 0.33f, 0.f},
    {128, 64, 2.0f, 0.62f, 0.f},
    {160, 64, 3.5f, 0.65f, 0.f},
    {128, 128, 3.0f, 0.94f, 0.f},
    {256, 128, 4.0f, 1.87f, 0.f},
};

}  // namespace

int fp8_num_shapes() { return (int)(sizeof kShapes / sizeof kShapes[0]); }
Fp8Shape fp8_shape(int shape) { return kShapes[shape]; }

hipError_t launch_gemm_fp8(int shape, bool b_tile, const Fp8Params& p, hipStream_t stream) {
    switch (shape) {
        case 0: return launch_tile<16, 32, 16, 32, 3, 8>(b_tile, p, stream);
        case 1: return launch_tile<32, 32, 32, 32, 2, 8>(b_tile, p, stream);
        case 2: return launch_tile<64, 32, 64, 32, 3, 4>(b_tile, p, stream);
        case 3: return launch_tile<64, 64, 32, 32, 2, 2>(b_tile, p, stream);
        case 4: return launch_tile<80, 64, 80, 32, 2, 4>(b_tile, p, stream);
        case 5: return launch_tile<128, 64, 64, 32, 3, 2>(b_tile, p, stream);
        case 6: return launch_tile<160, 64, 80, 32, 2, 2>(b_tile, p, stream);
        case 7: return launch_tile<128, 128, 64, 64, 2, 2>(b_tile, p, stream);
        case 8: return launch_tile<256, 128, 64, 64, 3, 1>(b_tile, p, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_fp8_finish(const Fp8Params& p, hipStream_t stream) {
    const int64_t units = ((int64_t)p.N + 3) / 4 * p.M, wgs = (units + 255) / 256;
    const dim3 grid((unsigned)(wgs < 16384 ? wgs : 16384));
    if (p.c_bf16) hipLaunchKernelGGL(fp8_finish_kernel<true>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(fp8_finish_kernel<false>, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace fg
