// Mixture-of-experts layer for a few tokens. Bound by HBM: every weight of a
// chosen expert is read once and used for the few tokens that chose it.
//
//   route    logits = x R^T summed in binary64 (float products are exact
//            there), so that experts with near logits are not exchanged;
//   top-k    one wave per token;
//   gate/up  one workgroup per 16 inner rows of one chosen expert: waves split
//            K, sums joined in LDS in wave order, h = act(g) * u;
//   down     one workgroup per 16 output rows and all chosen experts: waves
//            split the (expert, block of K) pairs, each adds its weighted
//            results to a private tokens x 16 piece in LDS, and the pieces are
//            joined in wave order. No atomics: repeated calls are identical.
//
// The products run on v_mfma_f32_16x16x32_bf16 with the 16 weight rows as the
// instruction's rows and the expert's tokens as its columns (padded to 16; the
// matrix cores have time to spare). e4m3 and bfloat16 weights are exact in
// bfloat16; a binary32 x or h is split into bfloat16 terms, x = hi + mid + lo,
// which hold its 24 bits, so the products lose nothing. binary32 weights use
// v_mfma_f32_16x16x4_f32. A lane owns 32 of the 128 k of a step; which ones
// does not matter to the sum as long as both operands agree, so each weight
// type takes the order in which 16 lanes' 16-byte loads cover whole sectors.
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

// Eight e4m3 codes (two dwords) as bfloat16, exactly.
__device__ __forceinline__ bf8 codes_to_bf16(int lo, int hi) {
    bf8 v{};
#if defined(__HIP_DEVICE_COMPILE__)
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
#else
    (void)lo, (void)hi;
#endif
    return v;
}

// x = sum of NS bfloat16 terms, each the nearest to what the others leave (a
// term holds 8 bits, and the remainders are exact). An infinity keeps its
// first term only (the remainder would be NaN).
template <int NS>
__device__ __forceinline__ void split_bf16(const float (&x)[8], bf8 (&t)[NS]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float left = x[e];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const __bf16 h = (__bf16)left;
            t[s][e] = h;
            left -= (float)h;
            if (s == 0 && !(fabsf(left) < __builtin_inff())) left = 0.f;
        }
    }
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

// A lane's 32 weights of one row in step [k0, k0 + 128); past K they are 0.
template <int WT>
struct WeightStep {
    i4v v[Weight<WT>::kPieces];

    __device__ __forceinline__ void load(const uint8_t* row, int k0, int K, int g) {
        using W = Weight<WT>;
        const uint8_t* const at = row + (int64_t)k0 * W::kSize;
        if (k0 + 128 <= K) {
#pragma unroll
            for (int j = 0; j < W::kPieces; ++j)
                v[j] = *reinterpret_cast<const i4v*>(at + W::first(j, g) * W::kSize);
        } else {
#pragma unroll
            for (int j = 0; j < W::kPieces; ++j) {
                const int left = (K - k0 - W::first(j, g)) * W::kSize;  // bytes inside the row
                v[j] = i4v{0, 0, 0, 0};
                if (left > 0) {
                    v[j] = *reinterpret_cast<const i4v*>(at + W::first(j, g) * W::kSize);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int n = left - 4 * d;
                        const uint32_t m =
                            n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
                        v[j][d] &= (int)m;
                    }
                }
            }
        }
    }

    // bfloat16 operand j (of 4) of the step
    __device__ __forceinline__ bf8 frag(int j) const {
        if constexpr (WT == TYPE_E4M3) {
            return codes_to_bf16(v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1]);
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

// One token row as the operands of one step, from x.
template <int WT, bool XBF16>
struct XStep {
    static constexpr int kTerms = XBF16 ? 1 : 3;
    bf8 t[4][kTerms];

    __device__ __forceinline__ void load(const void* row, bool have, int k0, int K, bool vec,
                                         int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + frag_first<WT>(j, g);
            if constexpr (XBF16) {
                if (vec && have && k + 8 <= K) {
                    t[j][0] = *reinterpret_cast<const bf8*>(static_cast<const uint16_t*>(row) + k);
                    continue;
                }
            }
            float x[8];
            load_row<8, XBF16>(row, have, k, K, vec, x);
            split_bf16<kTerms>(x, t[j]);
        }
    }
    __device__ __forceinline__ f4 times(const WeightStep<WT>& w, f4 c) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf8 a = w.frag(j);
#pragma unroll
            for (int s = 0; s < kTerms; ++s) c = mfma_bf16(a, t[j][s], c);
        }
        return c;
    }
};
template <bool XBF16>
struct XStep<TYPE_F32, XBF16> {
    float x[8][4];

    __device__ __forceinline__ void load(const void* row, bool have, int k0, int K, bool vec,
                                         int g) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            load_row<4, XBF16>(row, have, k0 + Weight<TYPE_F32>::first(j, g), K, vec, x[j]);
    }
    __device__ __forceinline__ f4 times(const WeightStep<TYPE_F32>& w, f4 c) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f4 a = __builtin_bit_cast(f4, w.v[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = mfma_f32(a[e], x[j][e], c);
        }
        return c;
    }
};

// One pair's h as the operands of one step: bfloat16 terms in planes (binary32
// for binary32 weights), rows of h_ld elements, valid up to a multiple of 16.
template <int WT, int NP>
struct HStep {
    bf8 t[4][NP];

    __device__ __forceinline__ void load(const MoeParams& p, int pair, bool have, int k0, int K16,
                                         int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + frag_first<WT>(j, g);
#pragma unroll
            for (int s = 0; s < NP; ++s) {
                t[j][s] = bf8{};
                if (have && k < K16)
                    t[j][s] = *reinterpret_cast<const bf8*>(p.h + s * p.h_plane +
                                                            (int64_t)pair * p.h_ld + k);
            }
        }
    }
    __device__ __forceinline__ f4 times(const WeightStep<WT>& w, f4 c) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf8 a = w.frag(j);
#pragma unroll
            for (int s = 0; s < NP; ++s) c = mfma_bf16(a, t[j][s], c);
        }
        return c;
    }
};
template <int NP>
struct HStep<TYPE_F32, NP> {
    f4 x[8];

    __device__ __forceinline__ void load(const MoeParams& p, int pair, bool have, int k0, int K16,
                                         int g) {
        const float* row = reinterpret_cast<const float*>(p.h) + (int64_t)pair * p.h_ld;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k0 + Weight<TYPE_F32>::first(j, g);
            x[j] = f4{0.f, 0.f, 0.f, 0.f};
            if (have && k < K16) x[j] = *reinterpret_cast<const f4*>(row + k);
        }
    }
    __device__ __forceinline__ f4 times(const WeightStep<TYPE_F32>& w, f4 c) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f4 a = __builtin_bit_cast(f4, w.v[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = mfma_f32(a[e], x[j][e], c);
        }
        return c;
    }
};

__device__ __forceinline__ float act_exact(float x, int act) {
    // (a handful of values per workgroup: accurate library functions)
    if (act == ACT_SILU) return x / (1.f + expf(-x));
    if (act == ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    return activate(x, act);
}

// ---- route -----------------------------------------------------------------

template <int N, bool BF16>
__device__ __forceinline__ void load_doubles(const void* row, int k, int K, bool vec,
                                             double (&x)[N]) {
    float f[N];
    load_row<N, BF16>(row, true, k, K, vec, f);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = (double)f[e];
}

// NT tokens by 4 experts per workgroup; 4 waves split K.
template <int NT, bool XBF16, bool RBF16>
__global__ void __launch_bounds__(256) route_kernel(MoeParams p) {
    constexpr int NE = 4;
    __shared__ double part[4][NT * NE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * NE, t0 = blockIdx.y * NT;
    double acc[NT][NE] = {};
    for (int k = wave * 256 + lane * 4; k < p.H; k += 1024) {
        double x[NT][4], r[NE][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = t0 + t < p.T ? t0 + t : p.T - 1;
            load_doubles<4, XBF16>(static_cast<const uint8_t*>(p.x) +
                                       row * p.ldx * (XBF16 ? 2 : 4), k, p.H, p.vec_x, x[t]);
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int row = e0 + e < p.E ? e0 + e : p.E - 1;
            load_doubles<4, RBF16>(static_cast<const uint8_t*>(p.router) +
                                       row * p.ldr * (RBF16 ? 2 : 4), k, p.H, p.vec_r, r[e]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][e] = fma(x[t][i], r[e][i], acc[t][e]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            double v = acc[t][e];
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
            if (lane == 0) part[wave][t * NE + e] = v;
        }
    __syncthreads();
    if (threadIdx.x < NT * NE) {
        const int t = t0 + threadIdx.x / NE, e = e0 + threadIdx.x % NE;
        double v = 0.0;
        for (int w = 0; w < 4; ++w) v += part[w][threadIdx.x];
        if (t < p.T && e < p.E) p.logits[t * p.E + e] = v;
    }
}

// One wave per token. A NaN logit ranks as -inf (and its weight is NaN).
__global__ void __launch_bounds__(64) topk_kernel(MoeParams p) {
    const int t = blockIdx.x, lane = threadIdx.x;
    double key[kMaxE / 64];
    const double ninf = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < kMaxE / 64; ++i) {
        const int e = lane + 64 * i;
        key[i] = ninf;
        if (e < p.E) key[i] = p.logits[t * p.E + e];
    }
    uint32_t taken = 0;
    double top = 0.0;
    double mine = 0.0;  // lane s: the s-th chosen logit
    int mine_id = 0;
    for (int s = 0; s < p.k; ++s) {
        double v = ninf;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kMaxE / 64; ++i) {
            const int e = lane + 64 * i;
            const double c = key[i] == key[i] ? key[i] : ninf;
            if (e < p.E && !(taken >> i & 1) && (c > v || (c == v && e < at))) v = c, at = e;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double ov = __shfl_xor(v, o, 64);
            const int oa = __shfl_xor(at, o, 64);
            if (ov > v || (ov == v && oa < at)) v = ov, at = oa;
        }
        // at < E: k <= E, so some expert is left
        if ((at & 63) == lane) taken |= 1u << (at >> 6);
        double raw = 0.0;
#pragma unroll
        for (int i = 0; i < kMaxE / 64; ++i)
            if ((at >> 6) == i) raw = key[i];
        raw = __shfl(raw, at & 63, 64);
        if (s == 0) top = raw;
        if (lane == s) mine = raw, mine_id = at;
    }
    float sum = 0.f;
    if (p.renorm) {
        if (lane < p.k) sum = expf((float)(mine - top));
    } else {
#pragma unroll
        for (int i = 0; i < kMaxE / 64; ++i)
            if (lane + 64 * i < p.E) sum += expf((float)(key[i] - top));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = mine_id;
        p.weights[t * p.k + lane] = expf((float)(mine - top)) / sum;
    }
}

// ---- experts ---------------------------------------------------------------

// The ids in LDS and the chosen experts as a bit set (two barriers).
__device__ __forceinline__ void mark_experts(const MoeParams& p, int* ids, uint32_t* bits) {
    const int n = p.T * p.k;
    const int first = (int)threadIdx.x < n ? p.ids[threadIdx.x] : -1;  // in flight over the barrier
    for (int i = threadIdx.x; i < kMaxE / 32; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = i < (int)blockDim.x ? first : p.ids[i];
        ids[i] = e;
        if (e >= 0 && e < p.E) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// Chosen experts before word `lane` of the bit set (lanes 0 .. 15), and how
// many there are, from the words' own counts.
__device__ __forceinline__ int experts_before(const uint32_t* bits, int lane, int& total) {
    int own = lane < kMaxE / 32 ? __popc(bits[lane]) : 0, sum = own;
#pragma unroll
    for (int o = 1; o < kMaxE / 32; o <<= 1) {
        const int v = __shfl_up(sum, o, 64);
        if (lane >= o) sum += v;
    }
    total = __shfl(sum, kMaxE / 32 - 1, 64);
    return sum - own;
}

// The y-th chosen expert in ascending order, or -1 (the whole wave takes part).
__device__ __forceinline__ int nth_expert(const uint32_t* bits, int lane, int y) {
    int total;
    const int before = experts_before(bits, lane, total);
    int found = -1;
    if (lane < kMaxE / 32) {
        uint32_t w = bits[lane];
        const int skip = y - before;
        if (skip >= 0 && skip < __popc(w)) {
            for (int i = 0; i < skip; ++i) w &= w - 1;
            found = lane * 32 + __ffs(w) - 1;
        }
    }
    const uint64_t m = __ballot(found >= 0);
    return m ? __builtin_amdgcn_readfirstlane(__shfl(found, __ffsll((unsigned long long)m) - 1, 64))
             : -1;
}

// The tokens that chose expert e: this lane's token (lane < T), whether it
// did, the first of its slots that did, and (weights) the sum of those slots'
// weights.
struct Chosen {
    bool have;
    int pair;
    float weight;
};
template <bool WEIGHTS>
__device__ __forceinline__ Chosen chosen_by(const MoeParams& p, const int* ids, int lane, int e) {
    Chosen c{false, 0, 0.f};
    if (lane < p.T)
        for (int s = p.k - 1; s >= 0; --s)
            if (ids[lane * p.k + s] == e) {
                c.have = true;
                c.pair = lane * p.k + s;
                if (WEIGHTS) c.weight += p.weights[lane * p.k + s];
            }
    return c;
}

// Orders one wave's LDS accesses across its lanes.
__device__ __forceinline__ void wave_lds_sync() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// gate and up: RT x 16 inner rows of one expert per workgroup, NW waves
// splitting K. Each wave keeps the weights of its next step in flight while it
// uses the present ones.
template <int WT, bool XBF16, int RT, int NW>
struct GateUp {
    static constexpr int kStreams = 2 * RT;  // gate and up of each row tile
    using W = Weight<WT>;
    const MoeParams& p;
    const int lane, wave, n16, g, row0, steps;
    const uint8_t* w[kStreams];
    const float* s[kStreams];

    __device__ __forceinline__ GateUp(const MoeParams& p, int e, int row0)
        : p(p), lane(threadIdx.x & 63),
          wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), n16(lane & 15), g(lane >> 4),
          row0(row0), steps((p.H + 127) / 128) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            // (rows past I read the last one; their h is 0 or not stored)
            const int first = row0 + 16 * r < p.I ? row0 + 16 * r : p.I - 1;
            const int row = first + n16 < p.I ? first + n16 : p.I - 1;
            w[2 * r] = static_cast<const uint8_t*>(p.gate.w) +
                       (e * p.gate.stride + row * p.gate.ld) * W::kSize;
            w[2 * r + 1] = static_cast<const uint8_t*>(p.up.w) +
                           (e * p.up.stride + row * p.up.ld) * W::kSize;
            if (WT == TYPE_E4M3) {
                s[2 * r] = p.gate.s + e * p.gate.s_stride + (first >> 7);
                s[2 * r + 1] = p.up.s + e * p.up.s_stride + (first >> 7);
            }
        }
    }

    __device__ __forceinline__ void fetch(WeightStep<WT> (&v)[kStreams], int kb) const {
        if (kb >= steps) return;
#pragma unroll
        for (int i = 0; i < kStreams; ++i) v[i].load(w[i], kb * 128, p.H, g);
    }

    // NT groups of 16 tokens (tok: their indices, `count` of them)
    template <int NT>
    __device__ __forceinline__ void sums(const int* tok, int count, f4 (&acc)[NT][kStreams]) const {
        const void* x[NT];
        bool have[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            have[t] = 16 * t + n16 < count;
            x[t] = static_cast<const uint8_t*>(p.x) +
                   (have[t] ? tok[16 * t + n16] : 0) * p.ldx * (XBF16 ? 2 : 4);
#pragma unroll
            for (int i = 0; i < kStreams; ++i) acc[t][i] = f4{0.f, 0.f, 0.f, 0.f};
        }
        auto use = [&](const WeightStep<WT>(&v)[kStreams], int kb) {
            float f[kStreams];
#pragma unroll
            for (int i = 0; i < kStreams; ++i)
                f[i] = WT == TYPE_E4M3 ? s[i][kb * (i & 1 ? p.up.lds : p.gate.lds)] : 1.f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                XStep<WT, XBF16> xs;
                xs.load(x[t], have[t], kb * 128, p.H, p.vec_x, g);
#pragma unroll
                for (int i = 0; i < kStreams; ++i) {
                    if constexpr (WT == TYPE_E4M3) {
                        const f4 b = xs.times(v[i], f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[t][i][e] = fmaf(f[i], b[e], acc[t][i][e]);
                    } else {
                        acc[t][i] = xs.times(v[i], acc[t][i]);
                    }
                }
            }
        };
        if constexpr (NT > 2) {  // (many tokens: no registers for a second step)
            for (int kb = wave; kb < steps; kb += NW) {
                WeightStep<WT> v[kStreams];
                fetch(v, kb);
                use(v, kb);
            }
            return;
        }
        WeightStep<WT> v0[kStreams], v1[kStreams];
        fetch(v0, wave);
        for (int kb = wave; kb < steps; kb += 2 * NW) {
            fetch(v1, kb + NW);
            use(v0, kb);
            if (kb + NW >= steps) break;
            fetch(v0, kb + 2 * NW);
            use(v1, kb + NW);
        }
    }

    // Joins the waves' sums in wave order and stores h of the groups.
    template <int NT>
    __device__ __forceinline__ void finish(const int* pair, int count, f4 (&acc)[NT][kStreams],
                                           f4 (*red)[2][64]) const {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                red[wave][0][lane] = acc[t][2 * r];
                red[wave][1][lane] = acc[t][2 * r + 1];
                __syncthreads();
                if (threadIdx.x < 256) {
                    float gs = 0.f, us = 0.f;  // component `wave` of the four
                    for (int v = 0; v < NW; ++v) {
                        gs += red[v][0][lane][wave];
                        us += red[v][1][lane][wave];
                    }
                    const int i = row0 + 16 * r + 4 * g + wave;
                    if (16 * t + n16 < count && i < p.h_ld)
                        store_h(pair[16 * t + n16], i, i < p.I ? act_exact(gs, p.act) * us : 0.f);
                }
                __syncthreads();
            }
    }

    __device__ __forceinline__ void store_h(int pair, int i, float h) const {
        const int64_t at = (int64_t)pair * p.h_ld + i;
        if constexpr (WT == TYPE_F32) {
            reinterpret_cast<float*>(p.h)[at] = h;
        } else {
            float left = h;
#pragma unroll
            for (int s = 0; s < (XBF16 ? 2 : 3); ++s) {
                const __bf16 b = (__bf16)left;
                p.h[s * p.h_plane + at] = __builtin_bit_cast(uint16_t, b);
                left -= (float)b;
                if (s == 0 && !(fabsf(left) < __builtin_inff())) left = 0.f;
            }
        }
    }

    template <int NT>
    __device__ __forceinline__ void run(const int* tok, const int* pair, int count,
                                        f4 (*red)[2][64]) const {
        f4 acc[NT][kStreams];
        sums<NT>(tok, count, acc);
        finish<NT>(pair, count, acc, red);
    }
};

template <int WT, bool XBF16, int RT, int NW>
__global__ void __launch_bounds__(64 * NW, 2) gate_up_kernel(MoeParams p) {
    static_assert(NW >= 4, "the joining of the waves' sums takes 256 threads");
    __shared__ int ids[kMaxT * kMaxK];
    __shared__ uint32_t bits[kMaxE / 32];
    __shared__ int tok[NW][kMaxT], pair[NW][kMaxT];
    __shared__ __attribute__((aligned(16))) f4 red[NW][2][64];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    mark_experts(p, ids, bits);
    const int e = nth_expert(bits, lane, blockIdx.y);
    if (e < 0) return;
    // every wave makes its own copy of the expert's list: no barrier
    const Chosen c = chosen_by<false>(p, ids, lane, e);
    const uint64_t m = __ballot(c.have);
    const int count = __popcll(m);
    if (c.have) {
        const int at = __popcll(m & ((1ull << lane) - 1ull));
        tok[wave][at] = lane;
        pair[wave][at] = c.pair;
    }
    wave_lds_sync();
    const GateUp<WT, XBF16, RT, NW> gu(p, e, blockIdx.x * 16 * RT);
    // (binary32 x by 32 rows: four groups of tokens do not fit the registers,
    // and the second pass over the weights mostly hits the L2)
    constexpr int kMost = !XBF16 && RT > 1 ? 2 : 4;
    if (count <= 16) {
        gu.template run<1>(tok[wave], pair[wave], count, red);
    } else if (count <= 32) {
        gu.template run<2>(tok[wave], pair[wave], count, red);
    } else {
        for (int c0 = 0; c0 < count; c0 += 16 * kMost)
            gu.template run<kMost>(tok[wave] + c0, pair[wave] + c0, count - c0, red);
    }
}

// down: 16 output rows per workgroup. The (expert, block of K) units of all
// chosen experts are dealt to the waves in contiguous runs; a wave keeps the
// weights of its next D units in flight, over the border of two experts too.
constexpr int kDownWaves = 8;

template <int WT, bool XBF16>
__global__ void __launch_bounds__(64 * kDownWaves) down_kernel(MoeParams p) {
    using W = Weight<WT>;
    constexpr int NP = XBF16 ? 2 : 3;
    constexpr int D = WT == TYPE_E4M3 ? 4 : 2;
    __shared__ int ids[kMaxT * kMaxK];
    __shared__ uint32_t bits[kMaxE / 32];
    __shared__ int active[kMaxE];
    __shared__ int tok[kDownWaves][kMaxT], pair[kDownWaves][kMaxT];
    __shared__ float wt[kDownWaves][kMaxT];
    __shared__ float sum[kDownWaves][kMaxT][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * 16;
    mark_experts(p, ids, bits);
    int chosen;
    {
        int before = experts_before(bits, lane, chosen);
        if (wave == 0 && lane < kMaxE / 32)
            for (uint32_t w = bits[lane]; w; w &= w - 1) active[before++] = lane * 32 + __ffs(w) - 1;
    }
    for (int i = lane; i < p.T * 16; i += 64) sum[wave][i >> 4][i & 15] = 0.f;
    __syncthreads();
    const int steps = (p.I + 127) / 128;
    const int64_t units = (int64_t)__builtin_amdgcn_readfirstlane(chosen) * steps;
    const int K16 = p.h_ld;
    const int64_t u0 = units * wave / kDownWaves, u1 = units * (wave + 1) / kDownWaves;
    const int row = row0 + n16 < p.H ? row0 + n16 : p.H - 1;
    const uint8_t* const w0 = static_cast<const uint8_t*>(p.down.w) + row * p.down.ld * W::kSize;

    // the unit to fetch next and the one to use next
    int fa = (int)(u0 / steps), fk = (int)(u0 - (int64_t)fa * steps);
    int ua = fa, uk = fk;
    auto fetch = [&](WeightStep<WT>& v) {
        const int e = __builtin_amdgcn_readfirstlane(active[fa]);
        v.load(w0 + e * p.down.stride * W::kSize, fk * 128, p.I, g);
        if (++fk == steps) fk = 0, ++fa;
    };
    f4 acc[4];
    int count = 0;
    const float* sw = nullptr;
    auto flush = [&] {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (16 * t + n16 < count) {
                const int at = tok[wave][16 * t + n16];
                const float f = wt[wave][16 * t + n16];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[wave][at][4 * g + i] += f * acc[t][i];
            }
    };
    auto use = [&](const WeightStep<WT>& v, bool first) {
        if (first || uk == 0) {
            flush();
            wave_lds_sync();
            const int e = __builtin_amdgcn_readfirstlane(active[ua]);
            const Chosen c = chosen_by<true>(p, ids, lane, e);
            const uint64_t m = __ballot(c.have);
            count = __popcll(m);
            if (c.have) {
                const int at = __popcll(m & ((1ull << lane) - 1ull));
                tok[wave][at] = lane;
                pair[wave][at] = c.pair;
                wt[wave][at] = c.weight;
            }
            wave_lds_sync();
            if (WT == TYPE_E4M3) sw = p.down.s + e * p.down.s_stride + (row0 >> 7);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};
        }
        const float f = WT == TYPE_E4M3 ? sw[uk * p.down.lds] : 1.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (16 * t >= count) break;
            const bool have = 16 * t + n16 < count;
            HStep<WT, NP> hs;
            hs.load(p, have ? pair[wave][16 * t + n16] : 0, have, uk * 128, K16, g);
            if constexpr (WT == TYPE_E4M3) {
                const f4 b = hs.times(v, f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(f, b[i], acc[t][i]);
            } else {
                acc[t] = hs.times(v, acc[t]);
            }
        }
        if (++uk == steps) uk = 0, ++ua;
    };
    WeightStep<WT> v[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (u0 + d < u1) fetch(v[d]);
    for (int64_t u = u0; u < u1; u += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + d < u1) use(v[d], u + d == u0);
            if (u + d + D < u1) fetch(v[d]);
        }
    }
    flush();
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * 16; i += blockDim.x) {
        const int t = i >> 4, n = i & 15;
        if (row0 + n >= p.H) continue;
        float s = 0.f;
        for (int w = 0; w < kDownWaves; ++w) s += sum[w][t][n];
        const int64_t at = (int64_t)t * p.ldo + row0 + n;
        if (XBF16) static_cast<uint16_t*>(p.out)[at] = (uint16_t)bf16_code(s);
        else static_cast<float*>(p.out)[at] = s;
    }
}

template <int WT, bool XBF16>
hipError_t launch_experts(const MoeParams& p, hipStream_t stream) {
    const int most = p.E < p.T * p.k ? p.E : p.T * p.k;
    // Two workgroups of 4 waves on a CU, so that one streams while the other
    // finds its expert; 8 waves while that leaves CUs idle. 32 inner rows per
    // workgroup where the weights of two steps fit the registers.
    constexpr int RT = WT == TYPE_F32 ? 1 : 2;
    const int tiles = (p.I + 16 * RT - 1) / (16 * RT);
    if ((int64_t)tiles * most >= 512)
        hipLaunchKernelGGL((gate_up_kernel<WT, XBF16, RT, 4>), dim3(tiles, most), dim3(256), 0,
                           stream, p);
    else
        hipLaunchKernelGGL((gate_up_kernel<WT, XBF16, 1, 8>), dim3((p.I + 15) / 16, most),
                           dim3(512), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((down_kernel<WT, XBF16>), dim3((p.H + 15) / 16), dim3(64 * kDownWaves), 0,
                       stream, p);
    return hipGetLastError();
}

template <int NT>
void launch_logits(const MoeParams& p, hipStream_t stream) {
    const dim3 g((p.E + 3) / 4, (p.T + NT - 1) / NT);
    if (p.x_bf16 && p.router_bf16)
        hipLaunchKernelGGL((route_kernel<NT, true, true>), g, dim3(256), 0, stream, p);
    else if (p.x_bf16)
        hipLaunchKernelGGL((route_kernel<NT, true, false>), g, dim3(256), 0, stream, p);
    else if (p.router_bf16)
        hipLaunchKernelGGL((route_kernel<NT, false, true>), g, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((route_kernel<NT, false, false>), g, dim3(256), 0, stream, p);
}

}  // namespace

int moe_planes(int x_bf16) { return x_bf16 ? 2 : 3; }

hipError_t launch_moe_route(const MoeParams& p, hipStream_t stream) {
    if (p.T == 1) launch_logits<1>(p, stream);
    else launch_logits<4>(p, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(topk_kernel, dim3(p.T), dim3(64), 0, stream, p);
    return hipGetLastError();
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
