// The products of a gated feed-forward block on the matrix cores, for many rows:
//
//   FORWARD  G = x Wg^T, U = x Wu^T, h = act(G) * U; G and U kept in h's type, as
//            e4m3 codes with a scale per 1 x 128 block, or not at all
//   DX       dx = dG Wg + dU Wu
//   DW       dWg = dG^T x, dWu = dU^T x (+ beta times what was there)
//
// One kernel for all: B's rows are the instruction's rows and A's its columns, so that a
// lane holds one row of C and four consecutive columns of it. FORWARD's tile of B
// is half gate and half up, divided so that a wave has both products of the same columns and
// the activation needs no exchange. DX runs through gate's steps and then up's, in bfloat16
// into the same sums. bfloat16 products are exact and their sums binary32
// (v_mfma_f32_16x16x32_bf16); binary32 uses v_mfma_f32_16x16x4_f32.
//
// Tiles go from memory straight to LDS, NS stages, the next ones in flight while
// one is used. An operand stored along k (x and the weights in FORWARD, dG and dU in
// DX) has rows of KB bytes of k whose 16-byte chunks are exchanged so that the 16
// rows a wave reads together fall on different banks. One stored along m or n (the
// weights in DX, all of DW) keeps its order in memory, a row of LDS per k, and is
// transposed by the read (ds_read_b64_tr_b16: 4 k of 16 columns per 16 lanes), so no
// transposed copy is ever made. A binary32 one is read element by element.
//
// Large products are bound by the matrix cores: 4096 tokens, 4096 x 8192 in bfloat16, 256
// x 256 of B's and A's rows to a workgroup of eight waves (64 x 128 each, as large as the
// registers hold), one set of inputs again and again: forward 400 us (1370 TFLOP/s), 460 with
// G and U kept (475 on inputs that change), dx, and dgate and dup, 400 to 405 each; the cores
// are busy 58 % with G and U kept, 68 in dx, dgate and dup, the clock is down to 1.65 GHz, and
// with the 32 x 32 x 16 instruction both products give the same time. Short ones are bound by
// latency, a step of a small tile taking as long as its barrier, its loads' issue and the next
// reads: there a step is 128 or 256 bytes of k (32 tokens, 4096 x 8192: steps of 64 bytes 46
// us in tiles of 64 x 64 and 33 of 32 x 32, of 128 bytes 30, 4.5 TB/s of weights). Binary32
// reaches the instruction's rate where every CU has two workgroups (1024 tokens, 4096 x 4096:
// 473 us, 145 TFLOP/s).
#include "fg_device.h"
#include "fg_e4m3.h"
#include "fg_gated_kernels.h"
#include "fg_mfma16.h"

namespace fg {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));

// 4 k of 16 columns per 16 lanes: lane l gives the address of row l / 4, columns
// 4 (l % 4), and gets column l of the four rows.
__device__ __forceinline__ uint2 read_transposed(const uint8_t* p) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                   (__attribute__((address_space(3))) s4*)(uint32_t)(uintptr_t)(
                       __attribute__((address_space(3))) const uint8_t*)p));
#else
    (void)p;
    return uint2{0, 0};
#endif
}

// A tile of R rows (of m or n) and KB bytes of k, and how it gets to LDS and back.
// ALONG_K: stored with k along its rows.
template <bool BF16, bool ALONG_K, int R, int KB, int NW>
struct Tile {
    static constexpr int kSize = BF16 ? 2 : 4;
    static constexpr int kBytes = R * KB;
    static constexpr int kParts = kBytes / 1024 / NW;         // loads of one wave
    static_assert(kBytes % (1024 * NW) == 0, "whole loads per wave");
    static constexpr int kSteps = KB / kSize;                 // k of a step
    static constexpr int kRowBytes = ALONG_K ? KB : R * kSize;  // of a row in LDS
    static constexpr int kLanesPerRow = kRowBytes / 16;
    static constexpr int kRowsPerLoad = 64 / kLanesPerRow;
    static_assert(ALONG_K || R >= 64, "a row's chunks have 8 places or 16 to exchange");

    // Exchange of the 16-byte chunks of LDS row r: chunk c is at position c ^ turn(r).
    // ALONG_K: a 128-bit read of 16 rows (the 16 lanes that are served together are not
    // neighbours) covers all banks evenly; found by trying, 4 cycles a read, and 8 with
    // (r >> 2) & 3 for 64-byte rows.
    // Else the eight rows that 32 lanes read together do, or the four of 64 lanes.
    static __device__ __forceinline__ int turn(int r) {
        if constexpr (ALONG_K && KB == 256) return r & 15;
        else if constexpr (ALONG_K && KB == 128) return (r >> 1) & 7;
        else if constexpr (ALONG_K) return (r >> 2) & 2;
        else if constexpr (!BF16) return 4 * ((r >> 2) & 3);
        else if constexpr (R >= 128) return 2 * ((r & 3) + 4 * ((r >> 3) & 1));
        else return 2 * (((r >> 1) & 1) + 2 * ((r >> 3) & 1));
    }
    // Byte offset, from the tile's first element, of what lane `lane` loads in load i
    // of the tile.
    static __device__ __forceinline__ uint32_t source(int i, int lane, int64_t ld) {
        const int r = i * kRowsPerLoad + lane / kLanesPerRow;
        const int c = (lane % kLanesPerRow) ^ turn(r);
        return (uint32_t)(r * ld * kSize) + (uint32_t)(c * 16);
    }
    // What lane (n, g) = (lane % 16, lane / 16) gives to the instruction in sub-step
    // `sub`: the 16 bytes of k from 16 (4 sub + g) of row r0 + n (r0 a multiple of 16),
    // the same k from a tile of either kind.
    static __device__ __forceinline__ i4v read(const uint8_t* tile, int r0, int sub, int lane) {
        const int n = lane & 15, g = lane >> 4;
        if constexpr (ALONG_K) {
            return *reinterpret_cast<const i4v*>(tile + (r0 + n) * KB +
                                                 (((4 * sub + g) ^ turn(n)) << 4));
        } else if constexpr (!BF16) {
            i4v v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 4 * g + e;
                v[e] = *reinterpret_cast<const int*>(tile + (16 * sub + k) * kRowBytes +
                                                     (((r0 / 4 + (n >> 2)) ^ turn(k)) << 4) + 4 * (n & 3));
            }
            return v;
        } else {
            const int i = lane & 15, k = 8 * g + (i >> 2);
            const int c = r0 / 8 + ((i >> 1) & 1);
            const uint8_t* at = tile + (32 * sub + k) * kRowBytes + (i & 1) * 8 +
                                ((c ^ turn(k)) << 4);
            const uint2 lo = read_transposed(at), hi = read_transposed(at + 4 * kRowBytes);
            return i4v{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
        }
    }
};

// Four values of C's type at an element of any alignment.
template <bool BF16>
struct Quad {
    uint32_t u[BF16 ? 2 : 4];
    __device__ __forceinline__ void load(const uint8_t* c) { __builtin_memcpy(u, c, sizeof u); }
    // the first n of them, zeros after them
    __device__ __forceinline__ void load(const uint8_t* c, int n) {
        if (n >= 4) {
            load(c);
            return;
        }
#pragma unroll
        for (int d = 0; d < (BF16 ? 2 : 4); ++d) u[d] = 0;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (e >= n) continue;
            if constexpr (BF16) u[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(c)[e] << (16 * (e & 1));
            else u[e] = reinterpret_cast<const uint32_t*>(c)[e];
        }
    }
    __device__ __forceinline__ f4 values() const {
        f4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = __builtin_bit_cast(float, !BF16 ? u[e % (BF16 ? 2 : 4)]
                                                   : (e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16));
        return v;
    }
    __device__ __forceinline__ explicit Quad(f4 v) {
        if constexpr (BF16) {
            typedef __bf16 b4 __attribute__((ext_vector_type(4)));
            const b4 r = __builtin_convertvector(v, b4);
            __builtin_memcpy(u, &r, sizeof u);
        } else {
            __builtin_memcpy(u, &v, sizeof u);
        }
    }
    Quad() = default;
    // the first n of them
    __device__ __forceinline__ void store(uint8_t* c, int n) const {
        if (n >= 4) {
            __builtin_memcpy(c, u, sizeof u);
            return;
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (e >= n) continue;
            if constexpr (BF16) reinterpret_cast<uint16_t*>(c)[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
            else reinterpret_cast<uint32_t*>(c)[e] = u[e];
        }
    }
};

// codes4 for binary32 sums, whose quotients are seldom near a middle between codes: the
// codes of x r with r off by 2^-21 to either side, which is more than r and the product are
// off by (2^-23), agree unless one is in between. 15 instructions per four elements for 26
// (8192 tokens, 2048 x 8192, one set of inputs: 533 us, and 541 with codes4 alone).
__device__ __forceinline__ uint32_t codes_of(const f4& x, const Divisor& d) {
    const float lo = fmaf(d[0], -0x1p-21f, d[0]), hi = fmaf(d[0], 0x1p-21f, d[0]);
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * lo, x[1] * lo, 0, false);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * hi, x[1] * hi, 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * lo, x[3] * lo, a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * hi, x[3] * hi, b, true);
    if (a == b) return (uint32_t)a;
    return codes4(x, [&](int) { return d[0]; }, [&](int) { return d; });
}

// A workgroup's LDS: the stages, or the results' way out (16 rows of every wave, of both
// products, and what the codes of their rows are found with).
template <int OP, bool BF16, int BM, int BN, int WM, int WN, int KB, int NS>
constexpr int kLdsBytes = [] {
    constexpr int NW = BM / WM * (BN / WN), kColumns = OP == GATED_FORWARD ? WN / 2 : WN;
    constexpr int kStages = NS * (BM + BN) * KB, kRows = NW * 16 * (kColumns + 4) * 4;
    constexpr int kOut = OP != GATED_FORWARD
        ? kRows : 2 * kRows + 2 * (BN / WN) * BM * 4 + 2 * (BN / 2 / 128) * BM * 16;
    return kStages > kOut ? kStages : kOut;
}();

// The operands of a step are in registers before it begins, those of the next are read
// during it, and so a stage is free for its next load a step earlier. id: of n workgroups,
// which take slice `split` of the sums.
template <int OP, bool BF16, int BM, int BN, int WM, int WN, int KB, int NS>
__device__ __forceinline__ void tile_body(const GatedTileParams& p, uint8_t* lds, int id, int n,
                                          int split) {
    constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN;
    constexpr int TI = WM / 16, TJ = WN / 16;
    constexpr int SIZE = BF16 ? 2 : 4;
    constexpr bool kDual = OP == GATED_FORWARD;
    // (FORWARD: BN rows of B are BN / 2 of gate and BN / 2 of up)
    constexpr int kCols = kDual ? BN / 2 : BN;       // columns of C per workgroup
    constexpr int kWaveCols = kDual ? WN / 2 : WN;
    constexpr int PJ = kDual ? TJ / 2 : TJ;          // column tiles of one matrix
    using TA = Tile<BF16, OP != GATED_DW, BM, KB, NW>;
    using TB = Tile<BF16, OP == GATED_FORWARD, BN, KB, NW>;
    constexpr int kStage = TA::kBytes + TB::kBytes;
    constexpr int K1 = TA::kSteps;                   // k of a step
    constexpr int kPitch = kWaveCols + 4;

    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    constexpr int kSubs = KB / 64;   // instructions along k in a step
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = (wave % NWM) * WM, wj = (wave / NWM) * kWaveCols;
    const int tiles_m = (p.M + BM - 1) / BM;
    int tm, tn;
    tile_of(id, n, OP == GATED_DW ? 2 * tiles_m : tiles_m,
            (p.N + kCols - 1) / kCols, tm, tn);
    const int which = OP == GATED_DW && tm >= tiles_m ? 1 : 0;
    if (OP == GATED_DW && which) tm -= tiles_m;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * kCols;
    const int rows = p.M - m0 < BM ? (int)(p.M - m0) : BM;
    const int cols = p.N - n0 < kCols ? (int)(p.N - n0) : kCols;
    const int s0 = split * p.per_split;
    const int s1 = s0 + p.per_split < p.steps ? s0 + p.per_split : p.steps;
    const int half = OP == GATED_DX ? p.steps / 2 : p.steps;   // steps of one matrix

    // 16-byte pieces that exist in a row of n elements, in bytes
    auto whole = [](int64_t n) { return (n * SIZE + 15) & ~15ll; };
    auto at = [](const void* base, int64_t element) {
        return static_cast<const uint8_t*>(base) + element * SIZE;
    };
    const uint32_t lds0 = lds_address(lds);

    // Where the next step's loads come from. Steps are fetched one after the other, so
    // little is left to do for each: an operand stored along k moves its lanes' offsets
    // (rows past the matrix and the row's end stay past the buffer's), another its base,
    // by the rows of a step, of which the last step has fewer.
    const int first_m = OP == GATED_DX && s0 >= half ? 1 : 0;
    const int64_t first_k = (int64_t)(s0 - first_m * half) * K1;
    const int k_last = p.K % K1 ? p.K % K1 : K1;
    auto bytes_of = [&](int64_t n, int64_t ld, int64_t row) { return (uint32_t)((n - 1) * ld * SIZE + row); };
    // A
    constexpr bool kAlongA = OP != GATED_DW;
    const int64_t row_a = whole(kAlongA ? p.K : p.M) - (kAlongA ? 0 : m0 * SIZE);
    const uint8_t* base_a = kAlongA ? at(p.A[first_m], m0 * p.lda) : at(p.A[which], first_k * p.lda + m0);
    const uint32_t full_a = bytes_of(kAlongA ? rows : K1, p.lda, row_a);
    const uint32_t last_a = kAlongA ? full_a : bytes_of(k_last, p.lda, row_a);
    uint32_t cur_a[TA::kParts];
#pragma unroll
    for (int q = 0; q < TA::kParts; ++q)
        cur_a[q] = TA::source(wave + NW * q, lane, p.lda) + (kAlongA ? (uint32_t)first_k * SIZE : 0u);
    // B (FORWARD: the second half of its rows are up's first ones; DX: up's steps follow
    // gate's, with another leading dimension)
    constexpr int kHalfLoads = TB::kBytes / 1024 / 2;
    static_assert(!kDual || kHalfLoads % NW == 0, "a load of every wave is of one matrix");
    constexpr int kGateParts = kDual ? kHalfLoads / NW : TB::kParts;
    const int64_t row_b = whole(kDual ? p.K : p.N) - (kDual ? 0 : n0 * SIZE);
    const uint8_t* base_b[2];
    uint32_t full_b[2], last_b[2], cur_b[TB::kParts];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int u = OP == GATED_DW ? 0 : m;
        base_b[m] = kDual ? at(p.B[u], n0 * p.ldb[u])
                          : at(p.B[u], (OP == GATED_DX && m != first_m ? 0 : first_k) * p.ldb[u] + n0);
        full_b[m] = bytes_of(kDual ? cols : K1, p.ldb[u], row_b);
        last_b[m] = kDual ? full_b[m] : bytes_of(k_last, p.ldb[u], row_b);
    }
    if (OP == GATED_DX && first_m) base_b[0] = base_b[1];   // (the one that is read)
#pragma unroll
    for (int q = 0; q < TB::kParts; ++q) {
        const int i = wave + NW * q;
        if constexpr (kDual) {
            const int u = q >= kGateParts;
            cur_b[q] = TB::source(i - u * kHalfLoads, lane, p.ldb[u]) + (uint32_t)first_k * SIZE;
        } else {
            cur_b[q] = TB::source(i, lane, first_m ? +p.ldb[1] : +p.ldb[0]);
        }
    }
    // (A unary plus makes a value of an operand of ?:, which else chooses between two
    // places, and they then live in memory.)
    // Step s, the one after the last fetched, into a stage; past the last one buffers
    // without a byte, which read as zero.
    auto fetch = [&](int s, int stage) __attribute__((always_inline)) {
        const uint32_t to = lds0 + stage * kStage;
        const bool more = s < s1;
        const bool up = OP == GATED_DX && s >= half;
        const bool last = s == half - 1 || (OP == GATED_DX && s == 2 * half - 1);
        if constexpr (OP == GATED_DX) {
            if (s == half && s != s0) {   // from gate to up
                base_a = at(p.A[1], m0 * p.lda);
                base_b[0] = base_b[1];
#pragma unroll
                for (int q = 0; q < TA::kParts; ++q) cur_a[q] = TA::source(wave + NW * q, lane, p.lda);
#pragma unroll
                for (int q = 0; q < TB::kParts; ++q) cur_b[q] = TB::source(wave + NW * q, lane, p.ldb[1]);
            }
        }
        const i4v ra = buffer_words(base_a, more ? (last ? +last_a : +full_a) : 0u);
#pragma unroll
        for (int q = 0; q < TA::kParts; ++q) {
            dma16(ra, to + (wave + NW * q) * 1024, cur_a[q]);
            if constexpr (kAlongA) cur_a[q] += KB;
        }
        const uint32_t size0 = up ? (last ? +last_b[1] : +full_b[1]) : (last ? +last_b[0] : +full_b[0]);
        const i4v rb0 = buffer_words(base_b[0], more ? size0 : 0u);
        const i4v rb1 = buffer_words(base_b[1], more ? full_b[1] : 0u);
#pragma unroll
        for (int q = 0; q < TB::kParts; ++q) {
            dma16(kDual && q >= kGateParts ? +rb1 : +rb0, to + TA::kBytes + (wave + NW * q) * 1024, cur_b[q]);
            if constexpr (kDual) cur_b[q] += KB;
        }
        if constexpr (!kAlongA) base_a += K1 * p.lda * SIZE;
        if constexpr (!kDual) base_b[0] += K1 * (up ? +p.ldb[1] : +p.ldb[0]) * SIZE;
    };

    f4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

    // DX in binary32: gate's sum, while up's is taken. (One sum of both is 2 I roundings long
    // where two products and an addition have I: 1025 tokens, 1536 x 2047, errors 1.15 10^-6
    // and 8.1 10^-7, 248 us both. bfloat16 results round far above either.)
    constexpr bool kApart = OP == GATED_DX && !BF16;
    f4 of_gate[kApart ? TI : 1][kApart ? TJ : 1] = {};

    // row of B's tile that column tile j of the wave starts at
    auto b_row = [&](int j) {
        return kDual ? (j < PJ ? 0 : BN / 2) + wj + 16 * (j % PJ) : wj + 16 * j;
    };
    constexpr int kLoads = TA::kParts + TB::kParts;
    static_assert((NS - 1) * kLoads < 64, "loads left in flight must fit the vmcnt field");
    static_assert(OP != GATED_DX || kGradRow % K1 == 0, "a step past K reads its own row's zeros");
    auto meet = [] {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * kLoads)
                     : "memory");
    };
    // (FORWARD: the last step may end inside a row; elsewhere k runs over rows, of
    // which those past the last are zeros)
    const bool partial = kDual && s1 == p.steps && p.K % K1 != 0;
    const int whole_end = partial ? s1 - 1 : s1;
    struct Operands {
        i4v a[kSubs][TI], b[kSubs][TJ];
    };
    auto read = [&](int stage, Operands& o) __attribute__((always_inline)) {
        const uint8_t* const ta = lds + stage * kStage;
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
#pragma unroll
            for (int j = 0; j < TJ; ++j) o.b[u][j] = TB::read(ta + TA::kBytes, b_row(j), u, lane);
#pragma unroll
            for (int i = 0; i < TI; ++i) o.a[u][i] = TA::read(ta, wi + 16 * i, u, lane);
        }
    };
    auto row = [&](const Operands& o, int u, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma16<BF16>(o.b[u][j], o.a[u][i], acc[i][j]);
    };
    // Step s, its operands in `now`: stage s + 1 is there for everyone and everyone
    // has read stage s, which is loaded again. The matrix instructions begin at
    // once, the loads go out after the first row of them, and the reads between
    // the others.
    int stage = 0;
    auto step = [&](int s, const Operands& now, Operands& next) __attribute__((always_inline)) {
        meet();
        __builtin_amdgcn_s_setprio(1);
        row(now, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        fetch(s + NS, stage);
        stage = stage + 1 == NS ? 0 : stage + 1;
        __builtin_amdgcn_sched_barrier(0);
        read(stage, next);
#pragma unroll
        for (int u = 0; u < kSubs; ++u)
#pragma unroll
            for (int i = u == 0 ? 1 : 0; i < TI; ++i) row(now, u, i);
        constexpr int kEach = BF16 ? 2 : 4;   // of an operand stored across k
        constexpr int kReads = kSubs * (TI * (OP == GATED_DW ? kEach : 1) + TJ * (kDual ? 1 : kEach));
        constexpr int kLeft = kSubs * TI * TJ - TJ;
        constexpr int kGroups = kReads < kLeft ? kReads : kLeft;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kGroups - 1) / kGroups, 0);   // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x008, kLeft / kGroups, 0);                    // matrix
        }
    };
    Operands o[2];
#pragma unroll
    for (int d = 0; d < NS; ++d) fetch(s0 + d, d);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NS - 1) * kLoads) : "memory");
    read(0, o[0]);
    int s = s0;
    auto steps_to = [&](int end) __attribute__((always_inline)) {
        for (; s + 2 <= end; s += 2) {
            step(s, o[0], o[1]);
            step(s + 1, o[1], o[0]);
        }
        if (s < end) {
            step(s++, o[0], o[1]);
            if constexpr (kDual || kApart) o[0] = o[1];
        }
    };
    if constexpr (kApart) {
#pragma unroll 1
        for (int k = s0 < half && half < s1 ? 0 : 1; k < 2; ++k) {
            steps_to(k == 0 ? half : s1);
            if (k == 1) break;
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) {
                    of_gate[i][j] = acc[i][j];
                    acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
                }
        }
    } else {
        steps_to(whole_end);
    }
    if constexpr (kDual) {
        if (partial) {
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
                const int left = p.K - (s1 - 1) * K1 - (4 * u + g) * (16 / SIZE);
#pragma unroll
                for (int j = 0; j < TJ; ++j) o[0].b[u][j] = keep<BF16>(o[0].b[u][j], left);
#pragma unroll
                for (int i = 0; i < TI; ++i) o[0].a[u][i] = keep<BF16>(o[0].a[u][i], left);
#pragma unroll
                for (int i = 0; i < TI; ++i) row(o[0], u, i);
            }
        }
    }
    if constexpr (kApart) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] += of_gate[i][j];
    }
    auto all_done = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    all_done();

    // The wave's 16 rows at a time through its own part of the LDS, so that a store
    // covers consecutive elements of a row.
    constexpr int kLanes = kWaveCols / 4, kRows = 64 / kLanes;
    float* const own = reinterpret_cast<float*>(lds) + wave * 16 * kPitch;
    const int er = lane / kLanes, ec = (lane % kLanes) * 4;
    auto settle = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
    // of(j): column tile j of row tile i; to(row, column, value) for each
    auto by_rows = [&](int i, auto of, auto to) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PJ; ++j)
            *reinterpret_cast<f4*>(own + n16 * kPitch + 16 * j + 4 * g) = of(j);
        settle();
        f4 v[16 / kRows];
#pragma unroll
        for (int r = 0; r < 16 / kRows; ++r)
            v[r] = *reinterpret_cast<const f4*>(own + (r * kRows + er) * kPitch + ec);
        settle();
#pragma unroll
        for (int r = 0; r < 16 / kRows; ++r) {
            const int64_t row = m0 + wi + 16 * i + r * kRows + er, col = n0 + wj + ec;
            if (row < p.M && col < p.N) to(row, col, v[r]);
        }
    };
    auto put = [&](void* base, int64_t ld, int64_t row, int64_t col, const f4& v) {
        const int n = p.N - col < 4 ? (int)(p.N - col) : 4;
        Quad<BF16>(v).store(static_cast<uint8_t*>(base) + (row * ld + col) * SIZE, n);
    };
    if (p.splits > 1) {
        const int64_t slice = (int64_t)p.M * p.N;
        constexpr int kEach = OP == GATED_DX ? 1 : 2;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int m = 0; m < (kDual ? 2 : 1); ++m)
                by_rows(i, [&](int j) { return acc[i][m * PJ + j]; },
                        [&](int64_t row, int64_t col, const f4& v) {
                            const int n = p.N - col < 4 ? (int)(p.N - col) : 4;
                            Quad<false>(v).store(
                                reinterpret_cast<uint8_t*>(p.ws + (split * kEach + which + m) * slice +
                                                           row * p.N + col), n);
                        });
        return;
    }
    if constexpr (kDual) {
        // What dividing by the scale of a row in its block of 128 columns needs, from the
        // row's largest finite magnitude in the block: of the wave's columns, then of its
        // neighbours' along the row.
        constexpr int kPerBlock = 128 / kWaveCols;   // waves
        constexpr int kBlocks = kCols / 128;
        uint32_t* const most = reinterpret_cast<uint32_t*>(lds + 2 * NW * 16 * kPitch * 4);
        Divisor* const by = reinterpret_cast<Divisor*>(most + 2 * NWN * BM);
        if constexpr (kBlocks > 0) {
            static_assert(kCols % 128 == 0, "whole blocks, or no codes");
            if (p.save == SAVE_E4M3) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < TI; ++i) {
                        // (of all magnitudes, and again of the finite ones if need be: 533 us, at once 538)
                        uint32_t v = 0;
#pragma unroll
                        for (int j = 0; j < PJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) v = max(v, magnitude(acc[i][m * PJ + j][e]));
                        if (v >= kInf) {
                            v = 0;
#pragma unroll
                            for (int j = 0; j < PJ; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    v = max(v, finite_magnitude(acc[i][m * PJ + j][e]));
                        }
#pragma unroll
                        for (int o = 16; o < 64; o *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
                        if (g == 0) most[(m * NWN + wave / NWM) * BM + wi + 16 * i + n16] = v;
                    }
                __syncthreads();
                for (int k = threadIdx.x; k < 2 * kBlocks * BM; k += 64 * NW) {
                    const int m = k / (kBlocks * BM), block = k / BM % kBlocks, r = k % BM;
                    uint32_t v = 0;
#pragma unroll
                    for (int w = 0; w < kPerBlock; ++w)
                        v = max(v, most[(m * NWN + block * kPerBlock + w) * BM + r]);
                    const float s = scale_of(v);
                    by[k] = divisor_of(s);
                    if (m0 + r < p.M && n0 + block * 128 < p.N)
                        (m ? +p.scales[1] : +p.scales[0])[(n0 / 128 + block) *
                            (m ? +p.ld_scales[1] : +p.ld_scales[0]) + m0 + r] = s;
                }
                __syncthreads();
            }
        }
        // Row tile by row tile in one loop, whose code is fetched once (unrolled it was 130
        // KB; 8192 tokens, 2048 x 8192 with codes, eight rounds of tiles: 597 us before, 547 then).
        float* const own_u = own + NW * 16 * kPitch;
        constexpr int kTurns = 16 / kRows;
        auto codes_out = [&](int m, const f4& v, const Divisor& d, int64_t row, int64_t col) __attribute__((always_inline)) {
            const uint32_t c = codes_of(v, d);
            uint8_t* const to = static_cast<uint8_t*>(p.saved[m]) + row * p.ld_saved[m] + col;
            if (col + 4 <= p.N) {
                *reinterpret_cast<uint32_t*>(to) = c;
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (col + e < p.N) to[e] = (uint8_t)(c >> (8 * e));
            }
        };
        auto out = [&](auto act) __attribute__((always_inline)) {
#pragma unroll 1
            for (int i = 0; i < TI; ++i) {
#pragma unroll
                for (int k = 0; k < TI; ++k) {
                    if (__builtin_amdgcn_readfirstlane(i) != k) continue;   // (k stays a constant)
#pragma unroll
                    for (int j = 0; j < PJ; ++j) {
                        const int to = n16 * kPitch + 16 * j + 4 * g;
                        *reinterpret_cast<f4*>(own + to) = acc[k][j];
                        *reinterpret_cast<f4*>(own_u + to) = acc[k][PJ + j % PJ];
                    }
                }
                settle();
                f4 vg[kTurns], vu[kTurns];
#pragma unroll
                for (int r = 0; r < kTurns; ++r) {
                    vg[r] = *reinterpret_cast<const f4*>(own + (r * kRows + er) * kPitch + ec);
                    vu[r] = *reinterpret_cast<const f4*>(own_u + (r * kRows + er) * kPitch + ec);
                }
                const int64_t col = n0 + wj + ec;
#pragma unroll
                for (int r = 0; r < kTurns; ++r) {
                    const int in = wi + 16 * i + r * kRows + er;
                    const int64_t row = m0 + in;
                    if (row >= p.M || col >= p.N) continue;
                    f4 h;
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = activate_t<decltype(act)::value>(vg[r][e]) * vu[r][e];
                    put(p.C[0], p.ldc[0], row, col, h);
                    if (p.save == SAVE_SAME) {
                        put(p.saved[0], p.ld_saved[0], row, col, vg[r]);
                        put(p.saved[1], p.ld_saved[1], row, col, vu[r]);
                    }
                    if constexpr (kBlocks > 0) {
                        if (p.save == SAVE_E4M3) {
                            const Divisor* const d = by + (wj + ec) / 128 * BM + in;
                            codes_out(0, vg[r], d[0], row, col);
                            codes_out(1, vu[r], d[kBlocks * BM], row, col);
                        }
                    }
                }
            }
        };
        if (p.act == ACT_SILU) out(ActTag<ACT_SILU>{});
        else if (p.act == ACT_GELU) out(ActTag<ACT_GELU>{});
        else if (p.act == ACT_RELU) out(ActTag<ACT_RELU>{});
        else out(ActTag<ACT_NONE>{});
    } else {
#pragma unroll
        for (int i = 0; i < TI; ++i)
            by_rows(i, [&](int j) { return acc[i][j]; },
                    [&](int64_t row, int64_t col, f4 v) {
                        if (OP == GATED_DW && p.beta != 0.f) {
                            const uint8_t* c = static_cast<const uint8_t*>(p.C[which]) +
                                               (row * p.ldc[which] + col) * SIZE;
                            Quad<BF16> old;
                            old.load(c, p.N - col < 4 ? (int)(p.N - col) : 4);
                            const f4 o = old.values();
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = fmaf(p.beta, o[e], v[e]);
                        }
                        put(p.C[which], p.ldc[which], row, col, v);
                    });
    }
}

template <int OP, bool BF16, int BM, int BN, int WM, int WN, int KB, int NS>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) gated_tile_kernel(GatedTileParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsBytes<OP, BF16, BM, BN, WM, WN, KB, NS>];
    tile_body<OP, BF16, BM, BN, WM, WN, KB, NS>(p, lds, blockIdx.x, gridDim.x, blockIdx.y);
}

template <int OP, bool BF16, int BM, int BN, int WM, int WN, int KB, int NS>
hipError_t launch_tile(const GatedTileParams& p, hipStream_t stream) {
    constexpr int threads = 64 * (BM / WM) * (BN / WN);
    constexpr int kCols = OP == GATED_FORWARD ? BN / 2 : BN;
    const int64_t tiles = ((p.M + BM - 1) / BM) * (int64_t)((p.N + kCols - 1) / kCols) *
                          (OP == GATED_DW ? 2 : 1);
    const dim3 grid((unsigned)tiles, (unsigned)p.splits);
    hipLaunchKernelGGL((gated_tile_kernel<OP, BF16, BM, BN, WM, WN, KB, NS>), grid, dim3(threads), 0,
                       stream, p);
    return hipGetLastError();
}

// dx, its slices one after the other, and dgate and dup in one launch, dx first, whose sums
// are longer. n: tiles of dx. (What it saves is in plan_pair's comment.)
template <typename DX, typename DW>
__global__ void __launch_bounds__(DX::kThreads, 2) gated_pair_kernel(GatedTileParams dx, GatedTileParams dw, int n) {
    static_assert(DX::kThreads == DW::kThreads, "threads of the launch");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[DX::kLds > DW::kLds ? DX::kLds : DW::kLds];
    const int id = blockIdx.x, all = n * dx.splits;
    if (id < all) DX::run(dx, lds, id % n, n, id / n);
    else DW::run(dw, lds, id - all, gridDim.x - all, 0);
}
template <int OP, bool BF16, int BM, int BN, int WM, int WN, int KB, int NS>
struct Part {
    static constexpr int kThreads = 64 * (BM / WM) * (BN / WN);
    static constexpr int kLds = kLdsBytes<OP, BF16, BM, BN, WM, WN, KB, NS>;
    static __device__ __forceinline__ void run(const GatedTileParams& p, uint8_t* lds, int id, int n, int split) {
        tile_body<OP, BF16, BM, BN, WM, WN, KB, NS>(p, lds, id, n, split);
    }
    static int64_t tiles(int64_t M, int64_t N) {
        return ((M + BM - 1) / BM) * ((N + BN - 1) / BN) * (OP == GATED_DW ? 2 : 1);
    }
};
using PairDx32 = Part<GATED_DX, true, 32, 64, 16, 32, 256, 3>;
using PairDx64 = Part<GATED_DX, true, 64, 64, 32, 32, 128, 4>;
using PairDw = Part<GATED_DW, true, 128, 128, 64, 64, 64, 4>;
using PairDxF32 = Part<GATED_DX, false, 64, 128, 32, 32, 128, 3>;
using PairDwF32 = Part<GATED_DW, false, 64, 128, 32, 32, 128, 3>;

template <typename DX, typename DW>
hipError_t launch_pair(const GatedTileParams& dx, const GatedTileParams& dw, hipStream_t stream) {
    const int64_t n = DX::tiles(dx.M, dx.N);
    hipLaunchKernelGGL((gated_pair_kernel<DX, DW>), dim3((unsigned)(n * dx.splits + DW::tiles(dw.M, dw.N))),
                       dim3(DX::kThreads), 0, stream, dx, dw, (int)n);
    return hipGetLastError();
}

// Sums of the slices in ascending order, and what a launch with one slice does to
// them: half a wave per 128 columns of a row, four columns per lane, four slices' loads
// at a time. Partial sums come from the caches; 200 tokens x 1408, two slices with codes: 4.4
// us, most of it the launch and two dependent trips.
template <int OP, bool BF16>
__global__ void __launch_bounds__(256) gated_finish_kernel(GatedTileParams p) {
    constexpr int SIZE = BF16 ? 2 : 4;
    const int nb = (p.N + 127) / 128;
    const int64_t all = (int64_t)p.M * (OP == GATED_DW ? 2 : 1);
    const int64_t slice = (int64_t)p.M * p.N;
    constexpr int kEach = OP == GATED_DX ? 1 : 2;
    const int l = threadIdx.x & 31, block = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (block >= nb) return;
    const int64_t col = (int64_t)block * 128 + 4 * l;
    const int n = p.N - col < 4 ? (int)(p.N - col) : 4;   // (may be below 1)
    for (int64_t v = blockIdx.y; v < all; v += gridDim.y) {
        const int which = OP == GATED_DW && v >= p.M ? 1 : 0;
        const int64_t row = v - (which ? p.M : 0);
        auto sum = [&](int m) {
            f4 s = {0.f, 0.f, 0.f, 0.f};
            const float* const w = p.ws + (which + m) * slice + row * p.N + col;
            for (int k = 0; k < p.splits; k += 4) {
                f4 a[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = f4{0.f, 0.f, 0.f, 0.f};
                    if (k + q >= p.splits) continue;
                    const float* const at = w + (int64_t)(k + q) * kEach * slice;
                    if (n >= 4) {
                        __builtin_memcpy(&a[q], at, sizeof a[q]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < n) a[q][e] = at[e];
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) s = s + a[q];
            }
            return s;
        };
        auto put = [&](void* base, int64_t ld, const f4& x) {
            if (n > 0) Quad<BF16>(x).store(static_cast<uint8_t*>(base) + (row * ld + col) * SIZE, n);
        };
        const f4 a = sum(0);
        if constexpr (OP == GATED_FORWARD) {
            const f4 b = sum(1);
            f4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = activate(a[e], p.act) * b[e];
            put(p.C[0], p.ldc[0], h);
            if (p.save == SAVE_SAME) {
                put(p.saved[0], p.ld_saved[0], a);
                put(p.saved[1], p.ld_saved[1], b);
            } else if (p.save == SAVE_E4M3) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f4 x = m ? b : a;
                    uint32_t most = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) most = max(most, finite_magnitude(x[e]));
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o, 64));
                    const float s = scale_of(most);
                    const Divisor d = divisor_of(s);
                    const uint32_t c = codes_of(x, d);
                    if (l == 0) p.scales[m][block * p.ld_scales[m] + row] = s;
                    uint8_t* q = static_cast<uint8_t*>(p.saved[m]) + row * p.ld_saved[m] + col;
                    if (n >= 4) {
                        *reinterpret_cast<uint32_t*>(q) = c;
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < n) q[e] = (uint8_t)(c >> (8 * e));
                    }
                }
            }
        } else {
            f4 v4 = a;
            if (OP == GATED_DW && p.beta != 0.f) {
                const uint8_t* c = static_cast<const uint8_t*>(p.C[which]) + (row * p.ldc[which] + col) * SIZE;
                Quad<BF16> old;
                old.load(c, n);
                const f4 o = old.values();
#pragma unroll
                for (int e = 0; e < 4; ++e) v4[e] = fmaf(p.beta, o[e], v4[e]);
            }
            put(p.C[which], p.ldc[which], v4);
        }
    }
}

// The tiles, with what one costs by estimate: the start and end of a round, and a step
// for a workgroup alone on its CU and for as many as fit, fitted to times of 8 to 1024
// workgroups of 16 and 64 steps of 64 bytes (32 and 128 for binary32).
constexpr GatedShape kForwardBf16[] = {
    {256, 128, 64, 1, 10.2f, 0.78f, 0.78f},
    {128, 128, 64, 2, 9.0f, 0.49f, 0.90f},
    {64, 64, 128, 2, 5.3f, 0.31f, 0.63f},
    {64, 32, 128, 2, 6.0f, 0.16f, 0.35f},
    {32, 32, 128, 2, 6.3f, 0.09f, 0.23f},
};
constexpr GatedShape kForwardF32[] = {
    {128, 128, 128, 1, 13.0f, 3.55f, 3.55f},
    {128, 64, 64, 2, 8.0f, 0.98f, 1.82f},
    {64, 64, 128, 2, 4.5f, 1.05f, 1.86f},
    {64, 32, 128, 2, 4.0f, 0.59f, 1.03f},
    {32, 32, 128, 2, 3.7f, 0.36f, 0.59f},
};
constexpr GatedShape kDxBf16[] = {
    {256, 256, 64, 1, 8.0f, 0.81f, 0.81f},
    {128, 128, 64, 2, 5.5f, 0.38f, 0.52f},
    {64, 128, 128, 2, 5.0f, 0.46f, 0.65f},
    {64, 64, 128, 2, 5.5f, 0.27f, 0.47f},
    {32, 64, 256, 1, 5.5f, 0.25f, 0.25f},
};
constexpr GatedShape kDwBf16[] = {
    {256, 256, 64, 1, 9.0f, 0.76f, 0.76f},
    {128, 128, 64, 2, 5.5f, 0.33f, 0.46f},
    {64, 128, 128, 2, 5.5f, 0.37f, 0.67f},
    {64, 64, 128, 2, 6.5f, 0.18f, 0.46f},
};
constexpr GatedShape kDxF32[] = {
    {128, 128, 64, 2, 8.0f, 1.13f, 1.90f},
    {64, 128, 128, 2, 5.5f, 1.21f, 2.00f},
    {64, 64, 128, 2, 4.5f, 0.74f, 1.16f},
    {32, 64, 128, 2, 4.0f, 0.50f, 0.66f},
};
constexpr GatedShape kDwF32[] = {
    {128, 256, 128, 1, 13.5f, 3.68f, 3.68f},
    {128, 128, 64, 2, 8.0f, 1.09f, 1.95f},
    {64, 128, 128, 2, 5.5f, 1.18f, 2.08f},
    {64, 64, 128, 2, 4.5f, 0.72f, 1.16f},
};

struct Shapes {
    const GatedShape* list;
    int n;
};
template <int N>
constexpr Shapes all_of(const GatedShape (&list)[N]) {
    return {list, N};
}
constexpr Shapes kShapes[3][2] = {{all_of(kForwardF32), all_of(kForwardBf16)},
                                  {all_of(kDxF32), all_of(kDxBf16)},
                                  {all_of(kDwF32), all_of(kDwBf16)}};

}  // namespace

int gated_num_shapes(int op, bool bf16) { return kShapes[op][bf16].n; }
GatedShape gated_shape(int op, bool bf16, int shape) { return kShapes[op][bf16].list[shape]; }

hipError_t launch_gated_tile(int op, bool bf16, int shape, const GatedTileParams& p,
                             hipStream_t stream) {
    if (op == GATED_FORWARD && bf16) {
        switch (shape) {
            case 0: return launch_tile<GATED_FORWARD, true, 256, 256, 64, 128, 64, 4>(p, stream);
            case 1: return launch_tile<GATED_FORWARD, true, 128, 256, 64, 128, 64, 3>(p, stream);
            case 2: return launch_tile<GATED_FORWARD, true, 64, 128, 32, 64, 128, 3>(p, stream);
            case 3: return launch_tile<GATED_FORWARD, true, 64, 64, 32, 32, 128, 4>(p, stream);
            case 4: return launch_tile<GATED_FORWARD, true, 32, 64, 16, 32, 128, 6>(p, stream);
        }
    } else if (op == GATED_FORWARD) {
        switch (shape) {
            case 0: return launch_tile<GATED_FORWARD, false, 128, 256, 64, 64, 128, 3>(p, stream);
            case 1: return launch_tile<GATED_FORWARD, false, 128, 128, 64, 64, 64, 4>(p, stream);
            case 2: return launch_tile<GATED_FORWARD, false, 64, 128, 32, 32, 128, 3>(p, stream);
            case 3: return launch_tile<GATED_FORWARD, false, 64, 64, 32, 32, 128, 4>(p, stream);
            case 4: return launch_tile<GATED_FORWARD, false, 32, 64, 16, 32, 128, 6>(p, stream);
        }
    } else if (op == GATED_DX && bf16) {
        switch (shape) {
            case 0: return launch_tile<GATED_DX, true, 256, 256, 64, 128, 64, 4>(p, stream);
            case 1: return launch_tile<GATED_DX, true, 128, 128, 64, 64, 64, 4>(p, stream);
            case 2: return launch_tile<GATED_DX, true, 64, 128, 32, 64, 128, 3>(p, stream);
            case 3: return launch_tile<GATED_DX, true, 64, 64, 32, 32, 128, 4>(p, stream);
            case 4: return launch_tile<GATED_DX, true, 32, 64, 16, 32, 256, 4>(p, stream);
        }
    } else if (op == GATED_DW && bf16) {
        switch (shape) {
            case 0: return launch_tile<GATED_DW, true, 256, 256, 64, 128, 64, 4>(p, stream);
            case 1: return launch_tile<GATED_DW, true, 128, 128, 64, 64, 64, 4>(p, stream);
            case 2: return launch_tile<GATED_DW, true, 64, 128, 32, 64, 128, 3>(p, stream);
            case 3: return launch_tile<GATED_DW, true, 64, 64, 32, 32, 128, 4>(p, stream);
        }
    } else if (op == GATED_DX) {
        switch (shape) {
            case 0: return launch_tile<GATED_DX, false, 128, 128, 64, 64, 64, 4>(p, stream);
            case 1: return launch_tile<GATED_DX, false, 64, 128, 32, 32, 128, 3>(p, stream);
            case 2: return launch_tile<GATED_DX, false, 64, 64, 32, 32, 128, 4>(p, stream);
            case 3: return launch_tile<GATED_DX, false, 32, 64, 16, 32, 128, 6>(p, stream);
        }
    } else if (op == GATED_DW) {
        switch (shape) {
            case 0: return launch_tile<GATED_DW, false, 128, 256, 64, 64, 128, 3>(p, stream);
            case 1: return launch_tile<GATED_DW, false, 128, 128, 64, 64, 64, 4>(p, stream);
            case 2: return launch_tile<GATED_DW, false, 64, 128, 32, 32, 128, 3>(p, stream);
            case 3: return launch_tile<GATED_DW, false, 64, 64, 32, 32, 128, 4>(p, stream);
        }
    }
    return hipErrorInvalidValue;
}

int gated_pair(int64_t T, int64_t H, int64_t I) {
    const int64_t dw = PairDw::tiles(I, H);
    if (PairDx32::tiles(T, H) + dw <= 512) return kPairDx32;
    if (PairDx64::tiles(T, H) + dw <= 512) return kPairDx64;
    return PairDx32::tiles(T, H) <= 512 ? kPairDx32 : -1;
}

hipError_t launch_gated_pair(bool bf16, int dx_shape, const GatedTileParams& dx, const GatedTileParams& dw,
                             hipStream_t stream) {
    if (!bf16) return launch_pair<PairDxF32, PairDwF32>(dx, dw, stream);
    return dx_shape == kPairDx32 ? launch_pair<PairDx32, PairDw>(dx, dw, stream)
                                 : launch_pair<PairDx64, PairDw>(dx, dw, stream);
}

hipError_t launch_gated_finish(int op, bool bf16, const GatedTileParams& p, hipStream_t stream) {
    const int64_t rows = (int64_t)p.M * (op == GATED_DW ? 2 : 1);
    const dim3 grid((unsigned)((((int64_t)p.N + 127) / 128 + 7) / 8), (unsigned)(rows < 65535 ? rows : 65535));
    auto kernel = op == GATED_FORWARD ? (bf16 ? gated_finish_kernel<GATED_FORWARD, true>
                                              : gated_finish_kernel<GATED_FORWARD, false>)
                : op == GATED_DX ? (bf16 ? gated_finish_kernel<GATED_DX, true>
                                         : gated_finish_kernel<GATED_DX, false>)
                                 : (bf16 ? gated_finish_kernel<GATED_DW, true>
                                         : gated_finish_kernel<GATED_DW, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

// ---- gradients of the pre-activations -----------------------------------------

namespace {

// act(x) and act'(x). Where sigma or Phi has run out (x far below 0) both are 0, and
// far above 0 the derivative is 1. At the infinities the derivative is 0 and 1, too; act is
// what the forward product has there, -inf times 0: NaN for silu and gelu of -inf.
template <int ACT>
__device__ __forceinline__ void activate_both(float x, float& a, float& d) {
    if constexpr (ACT == ACT_RELU) {
        a = x < 0.f ? 0.f : x;
        d = x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);   // (NaN stays)
    } else if constexpr (ACT == ACT_GELU) {
        const float e = erf_as7126(x * 0.70710678118654752f), phi = 0.5f * (1.f + e);
        const float bell = 0.39894228040143268f * __expf(-0.5f * x * x);
        a = x * phi;
        d = bell == 0.f ? phi : fmaf(x, bell, phi);
    } else if constexpr (ACT == ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.f + __expf(-x));
        const float t = __builtin_amdgcn_rcpf(1.f + __expf(x));   // sigma(-x)
        a = x * s;
        const float st = s * t;
        d = st == 0.f ? s : fmaf(x, st, s);
    } else {
        a = x;
        d = 1.f;
    }
}

// dG, dU and h in one pass, four columns per thread, so that a wave reads and writes whole
// lines. bfloat16: dG and dU are rounded before the products that read them, as a tensor of
// that type between two layers is; dx, dgate and dup are off by 0.0024 of their size where
// binary32 dG and dU would leave 0.0017, as two bfloat16 terms each and twice the matrix
// instructions. Bound by HBM: 4096 x 8192 in bfloat16, five matrices, 61 us, 5.5 TB/s.
template <bool BF16, bool CODES, int ACT>
__global__ void __launch_bounds__(256) gated_grad_kernel(GatedGradParams p) {
    constexpr int SIZE = BF16 ? 2 : 4;
    // a workgroup: 1024 columns of a row, or as many short rows as fit
    const int per_row = (int)(p.ld_d / 4), tid = threadIdx.x;
    const int rows = per_row < 256 ? 256 / per_row : 1;
    const int in = per_row < 256 ? tid / per_row : 0;
    const int col = 4 * (per_row < 256 ? tid - in * per_row : (int)blockIdx.x * 256 + tid);
    if (in >= rows || col >= p.ld_d) return;
    const int n = p.I - col < 4 ? p.I - col : 4;
    for (int64_t row = (int64_t)blockIdx.y * rows + in; row < p.T; row += (int64_t)gridDim.y * rows) {
        f4 dg = {0.f, 0.f, 0.f, 0.f}, du = dg, h = dg;
        auto gradients = [&](int n) __attribute__((always_inline)) {
            auto get = [&](const void* base, int64_t ld) {
                Quad<BF16> q;
                q.load(static_cast<const uint8_t*>(base) + (row * ld + col) * SIZE, n);
                return q;
            };
            const Quad<BF16> dhq = get(p.dh, p.lddh);
            f4 pre[2];
            if constexpr (CODES) {
                uint32_t c[2] = {0, 0};
                float s[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint8_t* at = static_cast<const uint8_t*>(p.saved[m]) + row * p.ld_saved[m] + col;
                    s[m] = p.scales[m][(col >> 7) * p.ld_scales[m] + row];
                    if (n >= 4) {
                        c[m] = *reinterpret_cast<const uint32_t*>(at);
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < n) c[m] |= (uint32_t)at[e] << (8 * e);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    pre[m][0] = s[m] * __builtin_amdgcn_cvt_f32_fp8(c[m], 0);
                    pre[m][1] = s[m] * __builtin_amdgcn_cvt_f32_fp8(c[m], 1);
                    pre[m][2] = s[m] * __builtin_amdgcn_cvt_f32_fp8(c[m], 2);
                    pre[m][3] = s[m] * __builtin_amdgcn_cvt_f32_fp8(c[m], 3);
                }
            } else {
                const Quad<BF16> g = get(p.saved[0], p.ld_saved[0]), u = get(p.saved[1], p.ld_saved[1]);
                pre[0] = g.values();
                pre[1] = u.values();
            }
            const f4 dh = dhq.values();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e >= n) continue;
                float a, d;
                activate_both<ACT>(pre[0][e], a, d);
                du[e] = dh[e] * a;
                dg[e] = dh[e] * pre[1][e] * d;
                h[e] = a * pre[1][e];
            }
        };
        if (n >= 4) gradients(4);   // (all loads on their way together)
        else if (n > 0) gradients(n);
        // (rows of dg and du end with zeros)
        const int64_t at = (row * p.ld_d + col) * SIZE;
        Quad<BF16>(dg).store(static_cast<uint8_t*>(p.dg) + at, 4);
        Quad<BF16>(du).store(static_cast<uint8_t*>(p.du) + at, 4);
        if (p.h && n > 0) Quad<BF16>(h).store(static_cast<uint8_t*>(p.h) + (row * p.ldh + col) * SIZE, n);
    }
}

template <bool BF16, bool CODES>
void launch_grad(const GatedGradParams& p, dim3 grid, hipStream_t stream) {
    auto kernel = p.act == ACT_SILU   ? gated_grad_kernel<BF16, CODES, ACT_SILU>
                  : p.act == ACT_GELU ? gated_grad_kernel<BF16, CODES, ACT_GELU>
                  : p.act == ACT_RELU ? gated_grad_kernel<BF16, CODES, ACT_RELU>
                                      : gated_grad_kernel<BF16, CODES, ACT_NONE>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
}

}  // namespace

hipError_t launch_gated_grad(bool bf16, const GatedGradParams& p, hipStream_t stream) {
    const int64_t per_row = p.ld_d / 4, rows = per_row < 256 ? 256 / per_row : 1;
    const int64_t groups = (p.T + rows - 1) / rows;
    const dim3 grid((unsigned)(per_row < 256 ? 1 : (per_row + 255) / 256),
                    (unsigned)(groups < 65535 ? groups : 65535));
    const bool codes = p.save == SAVE_E4M3;
    if (bf16 && codes) launch_grad<true, true>(p, grid, stream);
    else if (bf16) launch_grad<true, false>(p, grid, stream);
    else if (codes) launch_grad<false, true>(p, grid, stream);
    else launch_grad<false, false>(p, grid, stream);
    return hipGetLastError();
}

}  // namespace fg
