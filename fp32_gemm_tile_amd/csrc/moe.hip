// Mixture-of-experts layer for a few tokens. Bound by HBM: every weight of a
// chosen expert is read once and used for the few tokens that chose it.
//
//   route    logits = x R^T summed in binary64 (float products are exact
//            there), so that experts with near logits are not exchanged;
//   top-k    a wave per token; then the plan: the groups of tokens that share
//            an expert (a call without a router runs the plan alone);
//   gate/up  one workgroup per 16 or 32 inner rows of one group: waves take
//            the steps of K in turn, sums joined in wave order, h = act(g) * u;
//   down     16 or 32 output rows and all groups per workgroup: waves take the
//            (group, step) units in turn, each adds its weighted results to a
//            private tokens x rows piece in LDS, and the pieces are joined in
//            wave order, those of several workgroups by the last to finish. No
//            atomics on values: repeated calls are identical.
//
// Measured (one MI355X; the experts' types e4m3, bfloat16, e4m3 and binary32):
// 1 token, 2 of 8 experts of 1024 x 512: route 3.1 us, top-k 2.4, gate/up 6.6,
// down 5.4; 8 tokens, 6 of 64 of 2048 x 1408: 5.5, 6.9, 79, 40; 16 tokens, 8 of
// 128 of 4096 x 1536: 7.6, 8.0, 178 (5.8 TB/s of the weights), 96 (5.4 TB/s);
// 64 routed tokens, 2 of 16 of 2048 x 2000: plan 5, 98 (5.3 TB/s), 51 (5.1 TB/s).
// Route, top-k and plan are chains of latencies. A read of that many bytes
// alone runs at 5.8 to 6.3 TB/s.
//
// The products run on v_mfma_f32_16x16x32_bf16 with the 16 weight rows as the
// instruction's rows and the group's tokens as its columns. e4m3 and bfloat16
// weights are exact in bfloat16; a binary32 x and every h are split into bfloat16
// terms, x = hi + mid + lo, which hold its 24 bits, so the products lose
// nothing. binary32 weights use v_mfma_f32_16x16x4_f32. A lane owns 32 of the
// 128 k of a step; which ones does not matter to the sum as long as both
// operands agree, so each weight type takes the order in which 16 lanes'
// 16-byte loads cover whole sectors.
#include <algorithm>

#include "fg_device.h"
#include "fg_lowp_kernels.h"

namespace fg {
namespace {

typedef int i4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kMaxT = 64, kMaxK = 16, kMaxE = 512;

__device__ __forceinline__ f4 mfma_bf16(bf8 a, bf8 b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    (void)a, (void)b;
    return c;
#endif
}
__device__ __forceinline__ f4 mfma_f32(float a, float b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
#else
    (void)a, (void)b;
    return c;
#endif
}

// Eight e4m3 codes (two dwords) times a power of two as bfloat16, exactly.
__device__ __forceinline__ bf8 codes_to_bf16(int lo, int hi, float power = 1.f) {
    bf8 v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, false);
    const bf2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, false);
    const bf2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
#else
    (void)lo, (void)hi, (void)power;
#endif
    return v;
}

// Takes a bfloat16 term off `left`, exactly (a term holds 8 bits). All but the
// last are cut off towards zero, so that sums of the first terms of values up to
// the largest binary32 do not pass it; the last is the nearest. An infinity or
// NaN keeps its first term only (the remainder would be NaN).
__device__ __forceinline__ __bf16 next_term(float& left, bool last) {
    const bool finite = fabsf(left) < __builtin_inff();
    const float cut = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, left) & 0xFFFF0000u);
    const __bf16 h = (__bf16)(last || !finite ? left : cut);
    left = finite ? left - (float)h : 0.f;
    return h;
}

// x = sum of NS bfloat16 terms.
template <int NS>
__device__ __forceinline__ void split_bf16(const float (&x)[8], bf8 (&t)[NS]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float left = x[e];
#pragma unroll
        for (int s = 0; s < NS; ++s) t[s][e] = next_term(left, s == NS - 1);
    }
}

// What a later term's sum adds to the first one's. An infinite weight makes the
// first infinite (NaN beside 0), and NaN of the later ones, which may be 0 because
// the value has no more bits.
__device__ __forceinline__ float beside(float first, float later) {
    return __builtin_isfinite(first) ? later : 0.f;
}

// Per weight type: bytes per element, 16-byte pieces of a lane's 32 elements,
// and the first k (within the step of 128) of piece j of lane group g.
template <int WT>
struct Weight;
template <>
struct Weight<TYPE_E4M3> {
    static constexpr int kSize = 1, kPieces = 2;
    static __device__ __forceinline__ int first(int j, int g) { return j * 64 + g * 16; }
};
template <>
struct Weight<TYPE_BF16> {
    static constexpr int kSize = 2, kPieces = 4;
    static __device__ __forceinline__ int first(int j, int g) { return j * 32 + g * 8; }
};
template <>
struct Weight<TYPE_F32> {
    static constexpr int kSize = 4, kPieces = 8;
    static __device__ __forceinline__ int first(int j, int g) { return j * 16 + g * 4; }
};

constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer's end: reads as 0

__device__ __forceinline__ i4v load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(i4v, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// A lane's 32 weights of one row in step kb. Every load of the loops below is
// unconditional (past the row or the last step it reads nowhere), so that the
// number of loads in flight is known at every point and a wait for one step
// does not drain the next ones.
template <int WT>
struct WeightStep {
    i4v v[Weight<WT>::kPieces];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int kb, int K,
                                         int g) {
        using W = Weight<WT>;
#pragma unroll
        for (int j = 0; j < W::kPieces; ++j) {
            const int k = kb * 128 + W::first(j, g);
            v[j] = load16(r, k < K ? row + (uint32_t)(k * W::kSize) : kNowhere);
        }
    }
    // clears what the last step's pieces hold past K
    __device__ __forceinline__ void clear_tail(int kb, int K, int g) {
        using W = Weight<WT>;
        if (K - kb * 128 >= 128) return;
#pragma unroll
        for (int j = 0; j < W::kPieces; ++j) {
            const int left = (K - kb * 128 - W::first(j, g)) * W::kSize;  // bytes inside the row
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int n = left - 4 * d;
                const uint32_t m = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
                v[j][d] &= (int)m;
            }
        }
    }

    // bfloat16 operand j (of 4) of the step; codes times `power`
    __device__ __forceinline__ bf8 frag(int j, float power = 1.f) const {
        if constexpr (WT == TYPE_E4M3) {
            return codes_to_bf16(v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1], power);
        } else {
            return __builtin_bit_cast(bf8, v[j]);
        }
    }
};

// First k of bfloat16 operand j.
template <int WT>
__device__ __forceinline__ int frag_first(int j, int g) {
    return WT == TYPE_E4M3 ? Weight<TYPE_E4M3>::first(j >> 1, g) + 8 * (j & 1)
                           : Weight<TYPE_BF16>::first(j, g);
}

// The other operand of one step: a lane's part of one term of a row of x or h,
// bfloat16, or binary32 for binary32 weights. `cols` (a multiple of a piece)
// bounds the row; what lies past the matrix's own columns in it is 0.
template <int WT>
struct TokenStep {
    i4v t[4];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int kb, int cols,
                                         int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = kb * 128 + frag_first<WT>(j, g);
            t[j] = load16(r, row == kNowhere || k >= cols ? kNowhere : row + (uint32_t)k * 2u);
        }
    }
    __device__ __forceinline__ f4 times(const WeightStep<WT>& w, f4 c, float power = 1.f) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = mfma_bf16(w.frag(j, power), __builtin_bit_cast(bf8, t[j]), c);
        return c;
    }
};
template <>
struct TokenStep<TYPE_F32> {
    i4v x[8];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int kb, int cols,
                                         int g) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = kb * 128 + Weight<TYPE_F32>::first(j, g);
            x[j] = load16(r, row == kNowhere || k >= cols ? kNowhere : row + (uint32_t)k * 4u);
        }
    }
    __device__ __forceinline__ f4 times(const WeightStep<TYPE_F32>& w, f4 c) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f4 a = __builtin_bit_cast(f4, w.v[j]), b = __builtin_bit_cast(f4, x[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = mfma_f32(a[e], b[e], c);
        }
        return c;
    }
};

// acc[i] += f[i] * (step of w[i] times x), for N matrices: of codes with their
// block's scale f, else without.
template <int N, int WT>
__device__ __forceinline__ void add_step(f4 (&acc)[N], const WeightStep<WT> (&w)[N],
                                         const TokenStep<WT>& x, const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (WT == TYPE_E4M3) {
            const f4 b = x.times(w[i], f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(f[i], b[c], acc[i][c]);
        } else {
            acc[i] = x.times(w[i], acc[i]);
        }
    }
}

// A block's sum of codes is taken before its scale, and passes the largest
// binary32 (a code of 448 beside a value from 2^119 on) where the scaled sum need
// not. What follows is then infinite or NaN, so that it shows at the end and the
// loops need not look: where `passed`, they are gone through again with
// add_step_wide, which takes such a sum from codes times 2^-16, of which 128 add
// up to less than 1; 2^16 goes into the scale, or into the sum beside a scale that
// it would make infinite. (A look at every sum cost 4 % of the 16-token layer.)
template <int N>
__device__ __forceinline__ bool passed(const f4 (&acc)[N]) {
    bool over = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) over |= !__builtin_isfinite(acc[i][c]);
    return __builtin_expect(__ballot(over) != 0, false);
}
template <int N, int WT>
__device__ __forceinline__ void add_step_wide(f4 (&acc)[N], const WeightStep<WT> (&w)[N],
                                              const TokenStep<WT>& x, const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const f4 b = x.times(w[i], f4{0.f, 0.f, 0.f, 0.f});
        const f4 low = x.times(w[i], f4{0.f, 0.f, 0.f, 0.f}, 0x1p-16f);
        const bool large = fabsf(f[i]) >= 0x1p64f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool in = __builtin_isfinite(b[c]);
            const float v = in ? b[c] : (large ? low[c] * 0x1p16f : low[c]);
            acc[i][c] = fmaf(in || large ? f[i] : f[i] * 0x1p16f, v, acc[i][c]);
        }
    }
}

// Terms of one value of x and of h, and bytes of one of them. The terms of a
// token are columns of the matrix instruction next to each other, summed at
// the end: one load and one instruction serve 16 columns whatever they hold,
// and few tokens leave columns free (a load and an instruction per term cost
// the vector memory unit 12 loads instead of 4 per step of binary32 x, which
// bounded the kernels).
template <int WT, bool XBF16>
struct Terms {
    static constexpr int kX = WT == TYPE_F32 || XBF16 ? 1 : 3;
    static constexpr int kH = WT == TYPE_F32 ? 1 : 3;
    static constexpr int kSize = WT == TYPE_F32 ? 4 : 2;
};

// A uniform scale, through the scalar cache.
__device__ __forceinline__ float scale_at(const float* s, int64_t i) {
    return *reinterpret_cast<const __attribute__((address_space(4))) float*>(
        reinterpret_cast<uintptr_t>(s + i));
}

// N consecutive elements of a row of x (binary32 or bfloat16) as floats, 0
// past K or when the lane has no row.
template <int N, bool XBF16>
__device__ __forceinline__ void load_row(const void* row, bool have, int k, int K, bool vec,
                                         float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
    if (!have || k >= K) return;
    if constexpr (XBF16) {
        const uint16_t* r = static_cast<const uint16_t*>(row) + k;
        if (vec && k + N <= K) {
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                const uint2 u = *reinterpret_cast<const uint2*>(r + e);
                x[e] = __builtin_bit_cast(float, u.x << 16);
                x[e + 1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
                x[e + 2] = __builtin_bit_cast(float, u.y << 16);
                x[e + 3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (k + e < K) x[e] = __builtin_bit_cast(float, (uint32_t)r[e] << 16);
        }
    } else {
        const float* r = static_cast<const float*>(row) + k;
        if (vec && k + N <= K) {
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                const f4 u = *reinterpret_cast<const f4*>(r + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[e + i] = u[i];
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (k + e < K) x[e] = r[e];
        }
    }
}

__device__ __forceinline__ float act_exact(float x, int act) {
    // (a handful of values per workgroup: accurate library functions)
    if (act == ACT_SILU) return x / (1.f + expf(-x));
    if (act == ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    return activate(x, act);
}

// ---- route -----------------------------------------------------------------

// x as the experts' products read it: bfloat16 terms, or binary32 for binary32
// weights; eight elements per thread, of the grid's threads [first, first + all).
template <bool XBF16>
__device__ __forceinline__ void prepare_tokens(const MoeParams& p, int64_t first, int64_t all) {
    const int per_row = p.xs_ld / 8;
    for (int64_t u = first; u < (int64_t)p.T * per_row; u += all) {
        const int t = (int)(u / per_row), k = (int)(u - (int64_t)t * per_row) * 8;
        float x[8];
        load_row<8, XBF16>(static_cast<const uint8_t*>(p.x) + t * p.ldx * (XBF16 ? 2 : 4), true, k,
                           p.H, p.vec_x, x);
        const int64_t at = (int64_t)t * p.xs_ld + k;
        if (p.wtype == TYPE_F32) {
            float* const o = static_cast<float*>(p.xs) + at;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<f4*>(o + e) = f4{x[e], x[e + 1], x[e + 2], x[e + 3]};
        } else {
            constexpr int NS = XBF16 ? 1 : 3;
            bf8 s[NS];
            split_bf16<NS>(x, s);
#pragma unroll
            for (int i = 0; i < NS; ++i)
                *reinterpret_cast<bf8*>(static_cast<uint16_t*>(p.xs) + i * p.xs_plane + at) = s[i];
        }
    }
}

// NT tokens by 4 experts per workgroup; the waves take 256 k at a time, so that
// all of a row of up to 4096 is in flight at once (the kernel is a chain of
// latencies: one wave of loads, the sums' exchange, one LDS round). The last
// workgroups of the x dimension prepare x (other_wgs of them).
template <int NT, int NW, bool XBF16, bool RBF16>
__global__ void __launch_bounds__(64 * NW) route_kernel(MoeParams p, int other_wgs) {
    constexpr int NE = 4, NV = NT * NE;
    __shared__ double part[NW][NV];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int expert_wgs = gridDim.x - other_wgs;
    if ((int)blockIdx.x >= expert_wgs) {
        prepare_tokens<XBF16>(
            p, ((int64_t)(blockIdx.x - expert_wgs) * gridDim.y + blockIdx.y) * blockDim.x + threadIdx.x,
            (int64_t)other_wgs * gridDim.y * blockDim.x);
        return;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.plan->ticket = 0;
    const int e0 = blockIdx.x * NE, t0 = blockIdx.y * NT;
    double acc[NV] = {};
    for (int k = wave * 256 + lane * 4; k < p.H; k += NW * 256) {
        float x[NT][4], r[NE][4];
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int row = e0 + e < p.E ? e0 + e : p.E - 1;
            load_row<4, RBF16>(static_cast<const uint8_t*>(p.router) +
                                   row * p.ldr * (RBF16 ? 2 : 4), true, k, p.H, p.vec_r, r[e]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = t0 + t < p.T ? t0 + t : p.T - 1;
            load_row<4, XBF16>(static_cast<const uint8_t*>(p.x) + row * p.ldx * (XBF16 ? 2 : 4),
                               true, k, p.H, p.vec_x, x[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            double rd[NE];
#pragma unroll
            for (int e = 0; e < NE; ++e) rd[e] = (double)r[e][i];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const double xd = (double)x[t][i];
#pragma unroll
                for (int e = 0; e < NE; ++e) acc[t * NE + e] = fma(xd, rd[e], acc[t * NE + e]);
            }
        }
    }
    // Sum over the lanes: while there are several values left, half of the
    // lanes keep one half of them and the others the other half (lane bit 5
    // decides first); then plain exchanges. Lane l ends with value `mine`.
    int n = NV, o = 32, mine = 0;
#pragma unroll
    for (int h = NV / 2; h >= 1; h >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const double keep = upper ? acc[h + i] : acc[i], give = upper ? acc[i] : acc[h + i];
            acc[i] = keep + __shfl_xor(give, o, 64);
        }
        if (upper) mine += h;
        o >>= 1;
        n = h;
    }
    (void)n;
#pragma unroll
    for (int b = 64 / NV / 2; b >= 1; b >>= 1) acc[0] += __shfl_xor(acc[0], b, 64);
    if ((lane & (64 / NV - 1)) == 0) part[wave][mine] = acc[0];
    __syncthreads();
    if (threadIdx.x < NV) {
        const int t = t0 + threadIdx.x / NE, e = e0 + threadIdx.x % NE;
        double v = 0.0;
        for (int w = 0; w < NW; ++w) v += part[w][threadIdx.x];
        if (t < p.T && e < p.E) p.logits[t * p.E + e] = v;
    }
}

// ---- plan --------------------------------------------------------------------
//
// The unit of the experts' work is a group: tokens of one expert that fill the
// 16 columns of a matrix instruction, G = 16 / terms of them. Groups are
// numbered by expert, then by token; an expert with more tokens is read once
// per group, the later ones from the caches. x and h can have different
// numbers of terms, so there are two lists.

constexpr int kPlanThreads = 1024;

// Values that one workgroup leaves for another of the same launch. Agent-scope
// accesses go past the XCDs' own L2s, so once a workgroup's stores have been
// acknowledged they can be counted as done with a relaxed atomic; an agent-wide
// release and acquire (which write back and invalidate a whole L2) cost the
// 8-token layer 10 us in top-k and 60 us in the kernels that stream weights.
template <typename V>
__device__ __forceinline__ void leave(V* at, V v) {
    __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V fetch_left(const V* at) {
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether this workgroup is the last of `all` to arrive at the counter; all its
// threads call it after their stores. s_last: in LDS.
__device__ __forceinline__ bool last_to_arrive(int32_t* counter, int all, int* s_last) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores are acknowledged
    __syncthreads();
    if (threadIdx.x == 0)
        *s_last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT) == all - 1;
    __syncthreads();
    return *s_last;
}

static_assert(kPlanThreads == 2 * kMaxE, "a thread per expert and list");
struct PlanLds {
    int ids[kMaxT * kMaxK];
    float w[kMaxT * kMaxK];
    unsigned long long chose[kMaxE];   // the tokens that chose the expert
    int base[2][kMaxE];                // its first group, in the list for x and for h
    int wave_sum[kPlanThreads / 64];
};

// The plan, from l.ids and l.w (kPlanThreads threads, half of them for each list);
// the tickets of the down kernel are set to 0.
__device__ __forceinline__ void write_plan(const MoeParams& p, PlanLds& l) {
    const int tid = threadIdx.x, list = tid / kMaxE, e0 = tid % kMaxE;
    if (!list) l.chose[e0] = 0;
    for (int i = tid; i < (p.H + 15) / 16; i += kPlanThreads) p.tickets[i] = 0;
    __syncthreads();
    for (int i = tid; i < p.T * p.k; i += kPlanThreads) {
        const int e = l.ids[i];
        if (e >= 0 && e < p.E) atomicOr(&l.chose[e], 1ull << ((unsigned)i / (unsigned)p.k));
    }
    __syncthreads();
    const bool wanted = !list || p.groups_h != p.groups_x;
    const int G = list ? p.gh : p.gx;
    MoeGroup* const out = list ? p.groups_h : p.groups_x;
    const int own = (unsigned)(__popcll(l.chose[e0]) + G - 1) / (unsigned)G;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(sum, o, 64);
        if ((tid & 63) >= o) sum += v;
    }
    if ((tid & 63) == 63) l.wave_sum[tid >> 6] = sum;
    __syncthreads();
#pragma unroll 1
    for (int w = list * (kMaxE / 64); w < (tid >> 6); ++w) sum += l.wave_sum[w];
    l.base[list][e0] = sum - own;
    if (wanted) {
        if (e0 == kMaxE - 1) *(list ? &p.plan->total_h : &p.plan->total_x) = sum;
#pragma unroll 1
        for (int c = 0; c < own; ++c) {
            MoeGroup& m = out[sum - own + c];
            m.expert = e0;
            const int left = __popcll(l.chose[e0]) - c * G;
            m.count = left < G ? left : G;
        }
    }
    __syncthreads();
    if (!wanted) return;
#pragma unroll 1
    for (int i = e0; i < p.T * p.k; i += kMaxE) {
        const int e = l.ids[i], t = (unsigned)i / (unsigned)p.k;
        if (e < 0 || e >= p.E) continue;
        float w = 0.f;
        bool first = true;
#pragma unroll 1
        for (int s = 0; s < p.k; ++s)
            if (l.ids[t * p.k + s] == e) {
                first = first && t * p.k + s >= i;
                w += l.w[t * p.k + s];
            }
        if (!first) continue;
        const int rank = __popcll(l.chose[e] & ((1ull << t) - 1ull));
        const int c = (unsigned)rank / (unsigned)G;
        MoeGroup& m = out[l.base[list][e] + c];
        m.pair[rank - c * G] = (int16_t)i;
        m.weight[rank - c * G] = w;
    }
}

// Workgroup 0 writes the plan; the others prepare x.
template <bool XBF16>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(MoeParams p) {
    __shared__ PlanLds l;
    if (blockIdx.x > 0) {
        prepare_tokens<XBF16>(p, (int64_t)(blockIdx.x - 1) * kPlanThreads + threadIdx.x,
                              (int64_t)(gridDim.x - 1) * kPlanThreads);
        return;
    }
    for (int i = threadIdx.x; i < p.T * p.k; i += kPlanThreads) {
        l.ids[i] = p.ids[i];
        l.w[i] = p.weights[i];
    }
    __syncthreads();
    write_plan(p, l);
}

// The largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
#define FG_ROR(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 15, 15, true))
    FG_ROR(8);  // rotations within rows of 16
    FG_ROR(4);
    FG_ROR(2);
    FG_ROR(1);
#undef FG_ROR
#endif
    const uint32_t a = __builtin_amdgcn_readlane((int)v, 0), b = __builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = __builtin_amdgcn_readlane((int)v, 32), d = __builtin_amdgcn_readlane((int)v, 48);
    return max(max(a, b), max(c, d));
}

// Top-k, a wave per token, and the plan: one workgroup writes it from LDS, of
// several (of `per` tokens each) the last to finish does. A lane holds experts
// lane, lane + 64, ... as integers in the logits' order (NaN as -inf, -0 as 0); k
// times the largest is taken out: the larger upper half, of several the larger
// lower half, of several the lowest expert. A NaN logit's weight is NaN. (Counting
// every expert's rank against all others took 23 us for 64 tokens of 512 experts
// against 16, and 7.7 for 8 of 64 against 5.6.) The code is short for few experts,
// J = 1 and 2: it runs about once, and fetching it is most of the time (J = 8 for
// all: 9.6 us for 8 tokens of 64). A lone token's slots are the groups: LONE, one
// wave.
template <bool LONE, int J>
__global__ void __launch_bounds__(LONE ? 64 : kPlanThreads) topk_kernel(MoeParams p, int per) {
    __shared__ PlanLds l;
    __shared__ int s_last;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = blockIdx.x * per, t1 = t0 + per < p.T ? t0 + per : p.T;
    for (int t = t0 + wave; t < t1; t += (LONE ? 1 : kPlanThreads / 64)) {
        double raw[J];
        uint64_t key[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = 64 * j + lane;
            raw[j] = e < p.E ? p.logits[t * p.E + e] : 0.0;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const double v = raw[j] == raw[j] ? raw[j] + 0.0 : -__builtin_inf();
            const uint64_t b = __builtin_bit_cast(uint64_t, v);
            const uint64_t order = b >> 63 ? ~b : b | 1ull << 63;  // not 0
            key[j] = 64 * j + lane < p.E ? order : 0;
        }
        int chosen = 0;  // of slot `lane`
        double value = 0.0;
#pragma unroll 1
        for (int s = 0; s < p.k; ++s) {
            uint64_t best = key[0];
            int at = 0;
#pragma unroll
            for (int j = 1; j < J; ++j)
                if (64 * j < p.E && key[j] > best) best = key[j], at = j;
            const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
            // (wave_max is called by all lanes, never behind && or ?:, since it reads
            // the other lanes' registers)
            const uint32_t max_hi = wave_max(hi);
            bool in = hi == max_hi;
            uint64_t who = __ballot(in);
            if (who & (who - 1)) {
                const uint32_t max_lo = wave_max(in ? lo : 0u);
                in = in && lo == max_lo;
                who = __ballot(in);
                if (who & (who - 1)) {
                    const uint32_t low = in ? ~(uint32_t)(64 * at + lane) : 0u;
                    const uint32_t max_low = wave_max(low);
                    who = __ballot(low == max_low);
                }
            }
            const int winner = __builtin_amdgcn_readfirstlane(__builtin_ctzll(who));
            const int slot = __builtin_amdgcn_readlane(at, winner);
            double v = raw[0];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (slot != j) continue;
                v = raw[j];
                if (lane == winner) key[j] = 0;
            }
            const uint64_t bits = __builtin_bit_cast(uint64_t, v);
            const uint32_t v_lo = __builtin_amdgcn_readlane((int)(uint32_t)bits, winner);
            const uint32_t v_hi = __builtin_amdgcn_readlane((int)(uint32_t)(bits >> 32), winner);
            if (lane == s) {
                chosen = 64 * slot + winner;
                value = __builtin_bit_cast(double, (uint64_t)v_hi << 32 | v_lo);
            }
        }
        const double top = __shfl(value, 0, 64);
        const float mine = lane < p.k ? expf((float)(value - top)) : 0.f;
        float sum = mine;
        if (!p.renorm) {
            sum = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (64 * j + lane < p.E) sum += expf((float)(raw[j] - top));
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
        if (lane < p.k) {
            const float w = mine / sum;
            leave(p.ids + t * p.k + lane, (int32_t)chosen);
            leave(p.weights + t * p.k + lane, w);
            if constexpr (LONE) {
                MoeGroup& m = p.groups_x[lane];
                m.expert = chosen;
                m.count = 1;
                m.pair[0] = (int16_t)lane;
                m.weight[0] = w;
                if (lane == 0) p.plan->total_x = p.k;
            } else {
                l.ids[t * p.k + lane] = chosen;
                l.w[t * p.k + lane] = w;
            }
        }
    }
    if constexpr (LONE) {
        for (int i = lane; i < (p.H + 15) / 16; i += 64) p.tickets[i] = 0;
    } else {
        if (gridDim.x > 1) {
            // (the counter was set to 0 by the router kernel)
            if (!last_to_arrive(&p.plan->ticket, gridDim.x, &s_last)) return;
            for (int i = threadIdx.x; i < p.T * p.k; i += kPlanThreads) {
                l.ids[i] = fetch_left(p.ids + i);
                l.w[i] = fetch_left(p.weights + i);
            }
        }
        __syncthreads();
        write_plan(p, l);
    }
}

// ---- experts ---------------------------------------------------------------

// Rows [row0, row0 + rows) of an expert's matrix as a buffer.
template <int WT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t expert_rows(const ExpertMatrix& m, int e,
                                                              int row0, int rows, int cols) {
    constexpr int S = Weight<WT>::kSize;
    const int64_t bytes = ((int64_t)(rows - 1) * m.ld + cols) * S;
    return make_rsrc_bytes(static_cast<const uint8_t*>(m.w) + (e * m.stride + row0 * m.ld) * S,
                           (bytes + 15) & ~15ll);
}

// gate and up: RT x 16 inner rows of one group per workgroup, NW waves taking
// the steps of K in turn. A wave keeps the operands of its next D - 1 steps in
// flight while it uses the present ones.
template <int WT, bool XBF16, int RT, int NW, int D>
__global__ void __launch_bounds__(64 * NW, D == 1 ? 4 : 2) gate_up_kernel(MoeParams p) {
    static_assert(NW >= 4, "the joining of the waves' sums takes 256 threads");
    using W = Weight<WT>;
    using N = Terms<WT, XBF16>;
    constexpr int kStreams = 2 * RT;  // gate and up of each row tile
    __shared__ __attribute__((aligned(16))) f4 red[NW][2][64];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    // (past the last group the list holds nothing, but can be read)
    const MoeGroup* const group = p.groups_x + blockIdx.y;
    const int total = p.plan->total_x, e_read = group->expert, count = group->count;
    const int16_t column_pair = group->pair[n16 / N::kX], token_pair = group->pair[n16];
    if ((int)blockIdx.y >= total) return;
    const int e = __builtin_amdgcn_readfirstlane(e_read);

    const int row0 = blockIdx.x * 16 * RT;
    const int rows = p.I - row0 < 16 * RT ? p.I - row0 : 16 * RT;
    const __amdgpu_buffer_rsrc_t rg = expert_rows<WT>(p.gate, e, row0, rows, p.H);
    const __amdgpu_buffer_rsrc_t ru = expert_rows<WT>(p.up, e, row0, rows, p.H);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc_bytes(p.xs, p.xs_bytes);
    uint32_t at[kStreams];
    const float* s[kStreams];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        // (rows past the matrix read its last one; their h is 0 or not stored)
        const int row = 16 * r + n16 < rows ? 16 * r + n16 : rows - 1;
        at[2 * r] = (uint32_t)(row * p.gate.ld) * W::kSize;
        at[2 * r + 1] = (uint32_t)(row * p.up.ld) * W::kSize;
        if (WT == TYPE_E4M3) {
            const int b = (16 * r < rows ? row0 + 16 * r : row0) >> 7;
            s[2 * r] = p.gate.s + e * p.gate.s_stride + b;
            s[2 * r + 1] = p.up.s + e * p.up.s_stride + b;
        }
    }
    uint32_t token = kNowhere;  // this lane's column: a term of a token's row
    if (n16 / N::kX < count)
        token = ((uint32_t)column_pair / (uint32_t)p.k) * (uint32_t)(p.xs_ld * N::kSize) +
                (uint32_t)(n16 % N::kX) * (uint32_t)(p.xs_plane * N::kSize);

    struct Step {
        WeightStep<WT> w[kStreams];
        TokenStep<WT> x;
        float f[kStreams];
    };
    const int steps = (p.H + 127) / 128;
    f4 acc[kStreams];
#pragma unroll
    for (int i = 0; i < kStreams; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
    auto fetch = [&](Step& v, int kb) {
#pragma unroll
        for (int i = 0; i < kStreams; ++i) v.w[i].load(i & 1 ? ru : rg, at[i], kb, p.H, g);
        v.x.load(rx, token, kb, p.xs_cols, g);
        if constexpr (WT == TYPE_E4M3) {
            const int b = kb < steps ? kb : steps - 1;
#pragma unroll
            for (int i = 0; i < kStreams; ++i)
                v.f[i] = scale_at(s[i], b * (i & 1 ? p.up.lds : p.gate.lds));
        }
    };
    auto clear = [&](Step& v, int kb) {
        if (kb == steps - 1) {
#pragma unroll
            for (int i = 0; i < kStreams; ++i) v.w[i].clear_tail(kb, p.H, g);
        }
    };
    Step v[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(v[d], wave + d * NW);
    for (int kb = wave; kb < steps; kb += D * NW) {  // (past the last step: zeros)
#pragma unroll
        for (int d = 0; d < D; ++d) {
            fetch(v[(d + D - 1) % D], kb + (d + D - 1) * NW);
            clear(v[d], kb + d * NW);
            add_step<kStreams, WT>(acc, v[d].w, v[d].x, v[d].f);
        }
    }
    if constexpr (WT == TYPE_E4M3) {
        if (passed(acc)) {
#pragma unroll
            for (int i = 0; i < kStreams; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int kb = wave; kb < steps; kb += NW) {
                fetch(v[0], kb);
                clear(v[0], kb);
                add_step_wide<kStreams, WT>(acc, v[0].w, v[0].x, v[0].f);
            }
        }
    }

    // the sums over waves and terms, in order, 16 rows at a time; h in its terms
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        red[wave][0][lane] = acc[2 * r];
        red[wave][1][lane] = acc[2 * r + 1];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int i = row0 + 16 * r + 4 * g + wave;  // component `wave` of the four
            if (n16 < count && i < p.h_ld) {             // column n16: a token here
                float gs = 0.f, us = 0.f;
                for (int v = 0; v < NW; ++v) {
                    const f4* const gv = red[v][0] + 16 * g + n16 * N::kX;
                    const f4* const uv = red[v][1] + 16 * g + n16 * N::kX;
                    gs += gv[0][wave];
                    us += uv[0][wave];
#pragma unroll
                    for (int t = 1; t < N::kX; ++t) {
                        gs += beside(gv[0][wave], gv[t][wave]);
                        us += beside(uv[0][wave], uv[t][wave]);
                    }
                }
                const float h = i < p.I ? act_exact(gs, p.act) * us : 0.f;
                const int64_t to = (int64_t)token_pair * p.h_ld + i;
                if constexpr (WT == TYPE_F32) {
                    reinterpret_cast<float*>(p.h)[to] = h;
                } else {
                    float left = h;
#pragma unroll
                    for (int t = 0; t < N::kH; ++t) {
                        const __bf16 b = next_term(left, t == N::kH - 1);
                        p.h[t * p.h_plane + to] = __builtin_bit_cast(uint16_t, b);
                    }
                }
            }
        }
        __syncthreads();
    }
}

// down: RT x 16 output rows per workgroup. The (group, step of K) units of all
// groups go to the waves of the row's gridDim.y workgroups in turn; a wave
// keeps the weights and h of its next D units in flight, over the border of two
// groups too, and adds each group's weighted results to its own tokens x rows
// piece in LDS. (One CU draws about 25 GB/s whatever it keeps in flight, so
// fewer than 256 row tiles are split among several workgroups; one on a CU is
// best, since each has a start and a piece to join: 47, 64 and 97 us with two,
// 41, 53 and 92 with one for 34 experts of 2048 x 1408 bfloat16, 16 of 2048 x 2000
// binary32 and 82 of 4096 x 1536 e4m3.)
// Output rows of a workgroup: 32 share the reads of h (e4m3: 125 -> 102 us for
// 82 experts of 4096 x 1536), 16 for binary32 weights (61 -> 53 us).
constexpr int down_rows(int wtype) { return wtype == TYPE_F32 ? 16 : 32; }
// Its waves: 4, 8 for e4m3, whose units are small (111 -> 92 us).
constexpr int down_waves(int wtype) { return wtype == TYPE_E4M3 ? 8 : 4; }

template <int WT, bool XBF16, int RT, int D>
__global__ void __launch_bounds__(64 * down_waves(WT), 2) down_kernel(MoeParams p, int most) {
    constexpr int kDownWaves = down_waves(WT);
    constexpr int kRows = 16 * RT;
    using W = Weight<WT>;
    using N = Terms<WT, XBF16>;
    extern __shared__ __attribute__((aligned(16))) uint8_t down_lds[];
    MoeGroup* const groups = reinterpret_cast<MoeGroup*>(down_lds);            // [most]
    float* const sums = reinterpret_cast<float*>(down_lds + most * sizeof(MoeGroup));
    __shared__ int s_last;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * kRows;
    const int piece = p.T * kRows;
    float* const sum = sums + wave * piece;
    const int total = __builtin_amdgcn_readfirstlane(
        p.groups_h == p.groups_x ? p.plan->total_x : p.plan->total_h);
    {
        const i4v* const from = reinterpret_cast<const i4v*>(p.groups_h);
        i4v* const to = reinterpret_cast<i4v*>(groups);
        for (int i = threadIdx.x; i < most * (int)(sizeof(MoeGroup) / 16); i += blockDim.x)
            to[i] = from[i];
    }
    for (int i = lane; i < piece; i += 64) sum[i] = 0.f;
    __syncthreads();
    const int steps = (p.I + 127) / 128;
    const int rows = p.H - row0 < kRows ? p.H - row0 : kRows;
    uint32_t at[RT];
    int sb[RT];  // row block of the scales
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = 16 * r + n16 < rows ? 16 * r + n16 : rows - 1;
        at[r] = (uint32_t)(row * p.down.ld) * W::kSize;
        sb[r] = (16 * r < rows ? row0 + 16 * r : row0) >> 7;
    }
    const __amdgpu_buffer_rsrc_t rh = make_rsrc_bytes(p.h, p.h_bytes);

    struct Unit {
        WeightStep<WT> w[RT];
        TokenStep<WT> h;
        float f[RT];
    };
    // the unit to fetch next (its group's number, step, expert and this lane's
    // column, a term of a row of h) and the one to use next
    const int first = blockIdx.y * kDownWaves + wave, stride = kDownWaves * gridDim.y;
    const int stride_a = stride / steps, stride_k = stride - stride_a * steps;
    int fa = first / steps, fk = first - fa * steps, fe = 0, last = -1;
    int ua = fa, uk = fk;
    uint32_t frow = kNowhere;
    auto next = [&](int& a, int& k) {
        a += stride_a;
        k += stride_k;
        if (k >= steps) k -= steps, ++a;
    };
    auto expert_of = [&](int a) { return __builtin_amdgcn_readfirstlane(groups[a].expert); };
    auto row_of = [&](int a) {
        return n16 / N::kH < groups[a].count
                   ? (uint32_t)groups[a].pair[n16 / N::kH] * (uint32_t)(p.h_ld * N::kSize) +
                         (uint32_t)(n16 % N::kH) * (uint32_t)(p.h_plane * N::kSize)
                   : kNowhere;
    };
    // step k of expert e and the lane's row of h; in == false: reads nowhere
    auto load = [&](Unit& v, int e, uint32_t h_row, int step, bool in) {
        const int k = in ? step : steps;
        const __amdgpu_buffer_rsrc_t r = expert_rows<WT>(p.down, e, row0, rows, p.I);
#pragma unroll
        for (int i = 0; i < RT; ++i) v.w[i].load(r, at[i], k, p.I, g);
        v.h.load(rh, h_row, k, p.h_ld, g);
        if constexpr (WT == TYPE_E4M3) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
                v.f[i] = scale_at(p.down.s, e * p.down.s_stride + step * p.down.lds + sb[i]);
        }
    };
    auto fetch = [&](Unit& v) {
        const int a = fa < total ? fa : total - 1;
        if (a != last) {
            last = a;
            fe = expert_of(a);
            frow = row_of(a);
        }
        load(v, fe, frow, fk, fa < total);
        next(fa, fk);
    };
    auto clear = [&](Unit& v, int k) {
        if (k == steps - 1) {
#pragma unroll
            for (int r = 0; r < RT; ++r) v.w[r].clear_tail(k, p.I, g);
        }
    };
    f4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f4{0.f, 0.f, 0.f, 0.f};
    auto flush = [&](int a) {
        if constexpr (WT == TYPE_E4M3) {
            if (passed(acc)) {  // this wave's units of group a again
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r] = f4{0.f, 0.f, 0.f, 0.f};
                const int e = expert_of(a);
                const uint32_t row = row_of(a);
                int k = first - a * steps;
                if (k < 0) k += (stride - 1 - k) / stride * stride;
#pragma unroll 1
                for (; k < steps; k += stride) {
                    Unit v;
                    load(v, e, row, k, true);
                    clear(v, k);
                    add_step_wide<RT, WT>(acc, v.w, v.h, v.f);
                }
            }
        }
        // a token's terms are next to each other: their sum in the first
        const int c = n16 / N::kH;
        const bool have = n16 % N::kH == 0 && c < groups[a].count;
        const int to = have ? (int)((unsigned)groups[a].pair[c] / (unsigned)p.k) * kRows + 4 * g : 0;
        const float f = groups[a].weight[c];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            f4 s = acc[r];
#pragma unroll
            for (int t = 1; t < N::kH; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[i] += beside(acc[r][i], __shfl(acc[r][i], (lane + t) & 63, 64));
            if (have) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[to + 16 * r + i] += f * s[i];
            }
            acc[r] = f4{0.f, 0.f, 0.f, 0.f};
        }
    };
    auto use = [&](Unit& v) {
        clear(v, uk);
        add_step<RT, WT>(acc, v.w, v.h, v.f);
        const int a = ua;
        next(ua, uk);
        if (ua != a) flush(a);
    };
    if (ua < total) {
        Unit v[D];
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(v[d]);
        while (ua < total) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (ua < total) use(v[d]);
                fetch(v[d]);
            }
        }
    }
    __syncthreads();
    auto store = [&](int i, float s) {
        const int n = row0 + i % kRows;
        const int64_t to = (int64_t)(i / kRows) * p.ldo + n;
        if (n >= p.H) return;
        if (XBF16) static_cast<uint16_t*>(p.out)[to] = (uint16_t)bf16_code(s);
        else static_cast<float*>(p.out)[to] = s;
    };
    auto joined = [&](int i) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) s += sums[w * piece + i];
        return s;
    };
    if (gridDim.y == 1) {
        for (int i = threadIdx.x; i < piece; i += blockDim.x) store(i, joined(i));
        return;
    }
    // Several workgroups: each leaves its piece, the last one adds them in order.
    float* const pieces = p.pieces + (int64_t)blockIdx.x * gridDim.y * piece;
    for (int i = threadIdx.x; i < piece; i += blockDim.x)
        leave(pieces + blockIdx.y * piece + i, joined(i));
    if (!last_to_arrive(p.tickets + blockIdx.x, gridDim.y, &s_last)) return;
    for (int i = threadIdx.x; i < piece; i += blockDim.x) {
        float s = 0.f;
        for (int y = 0; y < (int)gridDim.y; y += 8) {  // (eight loads in flight)
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int from = y + q < (int)gridDim.y ? y + q : 0;
                v[q] = fetch_left(pieces + from * piece + i);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) s += y + q < (int)gridDim.y ? v[q] : 0.f;
        }
        store(i, s);
    }
}

template <int WT, bool XBF16>
hipError_t launch_experts(const MoeParams& p, hipStream_t stream) {
    // Workgroups of 4 waves, so that some stream while others start or join; 8
    // waves while that leaves CUs idle (e4m3, units of 32 rows: 468 of them 16.5 us
    // against 22, 384 22.6 against 20.6; binary32, units of 16: 352 25.8 against
    // 31.3). What covers the memory's latency is best
    // kept in other workgroups (four on a CU, one step per wave) for 8- and 16-bit
    // weights (82 experts of 4096 x 1536 e4m3 180 us against 189 with two
    // workgroups and two steps in flight, 34 of 2048 x 1408 bfloat16 81 against
    // 90); a step of binary32 weights takes too many registers for that (98 us for
    // 16 of 2048 x 2000, two workgroups, two steps; 100).
    constexpr int RT = WT == TYPE_E4M3 ? 2 : 1;
    constexpr int D = WT == TYPE_F32 ? 2 : 1;
    const int tiles = (p.I + 16 * RT - 1) / (16 * RT);
    if ((int64_t)tiles * p.most_x >= (RT == 2 ? 448 : 256))
        hipLaunchKernelGGL((gate_up_kernel<WT, XBF16, RT, 4, D>), dim3(tiles, p.most_x), dim3(256),
                           0, stream, p);
    else
        hipLaunchKernelGGL((gate_up_kernel<WT, XBF16, 1, 8, 2>), dim3((p.I + 15) / 16, p.most_x),
                           dim3(512), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int kRows = down_rows(WT), kWaves = down_waves(WT);
    const size_t lds = p.most_h * sizeof(MoeGroup) + (size_t)kWaves * p.T * kRows * 4;
    hipLaunchKernelGGL((down_kernel<WT, XBF16, kRows / 16, 2>),
                       dim3((p.H + kRows - 1) / kRows, p.down_wgs), dim3(64 * kWaves),
                       lds, stream, p, p.most_h);
    return hipGetLastError();
}

// Workgroups of `threads` that prepare x, 8 elements per thread.
int prepare_workgroups(const MoeParams& p, int threads) {
    if (!p.xs_made) return 0;
    return (int)(((int64_t)p.T * (p.xs_ld / 8) + threads - 1) / threads);
}

template <int NT, int NW>
void launch_logits(const MoeParams& p, hipStream_t stream) {
    const int rows = (p.T + NT - 1) / NT;
    const int other = (prepare_workgroups(p, 64 * NW) + rows - 1) / rows;
    const dim3 g((p.E + 3) / 4 + other, rows);
#define FG_LAUNCH(X, R)                                                                     \
    hipLaunchKernelGGL((route_kernel<NT, NW, X, R>), g, dim3(64 * NW), 0, stream, p, other)
    if (p.x_bf16 && p.router_bf16) FG_LAUNCH(true, true);
    else if (p.x_bf16) FG_LAUNCH(true, false);
    else if (p.router_bf16) FG_LAUNCH(false, true);
    else FG_LAUNCH(false, false);
#undef FG_LAUNCH
}

}  // namespace

hipError_t launch_moe_route(const MoeParams& p, hipStream_t stream) {
    // One token per workgroup while all of them run at once (16 tokens of 128
    // experts 7.6 us, four tokens per workgroup 8.2; 8 of 64 6.0 and 8.3).
    if (p.T == 1) launch_logits<1, 8>(p, stream);
    else if ((p.E + 3) / 4 * p.T <= 512) launch_logits<1, 16>(p, stream);
    else launch_logits<4, 16>(p, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto kernel = p.T == 1 ? topk_kernel<true, 8> : topk_kernel<false, 8>;
    if (p.E <= 64) kernel = p.T == 1 ? topk_kernel<true, 1> : topk_kernel<false, 1>;
    else if (p.E <= 128) kernel = p.T == 1 ? topk_kernel<true, 2> : topk_kernel<false, 2>;
    // One workgroup for few tokens, four tokens each for more (us, one against four
    // each: 16 of 64 experts 6.0, 7.1; 16 of 128 7.4, 8.1; 16 of 256 11.3, 9.3; 64 of
    // 64, sixteen against four each 9.6, 8.5; 64 of 512 21.6, 16.3).
    const int per = p.E <= 128 && p.T <= 16 ? 16 : 4;
    hipLaunchKernelGGL(kernel, dim3((p.T + per - 1) / per), dim3(p.T == 1 ? 64 : kPlanThreads), 0,
                       stream, p, per);
    return hipGetLastError();
}

hipError_t launch_moe_plan(const MoeParams& p, hipStream_t stream) {
    const dim3 g(1 + prepare_workgroups(p, kPlanThreads));
    if (p.x_bf16) hipLaunchKernelGGL(plan_kernel<true>, g, dim3(kPlanThreads), 0, stream, p);
    else hipLaunchKernelGGL(plan_kernel<false>, g, dim3(kPlanThreads), 0, stream, p);
    return hipGetLastError();
}

int moe_group_size(int terms) { return 16 / terms; }

int moe_down_workgroups(int wtype, int H, int I, int most_groups) {
    // As many as n workgroups on every CU take, for the n with the most even share,
    // with 2 % for every piece to join; each wave with at least two units.
    const int tiles = (H + down_rows(wtype) - 1) / down_rows(wtype);
    int best = 1;
    float best_cost = 0.f;
    for (int n = (tiles + 255) / 256, all = n + 4; n < all; ++n) {
        const int y = n * 256 / tiles;
        const float cost = (float)n / (float)y + 0.02f * (float)n;
        if (best_cost == 0.f || cost < best_cost) best = y, best_cost = cost;
    }
    const int units = most_groups * ((I + 127) / 128);
    return std::max(1, std::min(best, units / (2 * down_waves(wtype))));
}

hipError_t launch_moe_experts(const MoeParams& p, hipStream_t stream) {
    switch (p.wtype * 2 + (p.x_bf16 ? 1 : 0)) {
        case TYPE_F32 * 2: return launch_experts<TYPE_F32, false>(p, stream);
        case TYPE_F32 * 2 + 1: return launch_experts<TYPE_F32, true>(p, stream);
        case TYPE_BF16 * 2: return launch_experts<TYPE_BF16, false>(p, stream);
        case TYPE_BF16 * 2 + 1: return launch_experts<TYPE_BF16, true>(p, stream);
        case TYPE_E4M3 * 2: return launch_experts<TYPE_E4M3, false>(p, stream);
        case TYPE_E4M3 * 2 + 1: return launch_experts<TYPE_E4M3, true>(p, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace fg
