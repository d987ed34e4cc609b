// Device-side e4m3 codes of binary32 values with a common scale: the scale, and the
// code nearest to the exact quotient (see quant_fp8.hip for why it is).
#pragma once

#include "fg_device.h"

namespace fg {

constexpr float kTop = 448.f;

__device__ __forceinline__ float scale_of(uint32_t amax) {
    return fmaxf(__builtin_bit_cast(float, amax) / kTop, 1.17549435e-38f);
}

// What dividing by a scale needs: 2^-e r, 2^-e, s'.
typedef f4 Divisor;
__device__ __forceinline__ Divisor divisor_of(float s) {
    const uint32_t u = __builtin_bit_cast(uint32_t, s);  // normal, positive, < 2^121
    const float f = __builtin_bit_cast(float, (254u << 23) - (u & 0x7F800000u));
    const float s1 = __builtin_bit_cast(float, (u & 0x007FFFFFu) | 0x3F800000u);
    return Divisor{f * (1.f / s1), f, s1, 0.f};
}

// q, which is within two units of a number m that ends in 19 zero bits, as m or
// the next number on the side of it that x / s is on.
__device__ __forceinline__ float settle(float x, float q, const Divisor& d) {
    const uint32_t u = __builtin_bit_cast(uint32_t, q);
    const uint32_t m = (u + 2u) & 0xFFF80000u;  // (the sign stays: q is far from 0)
    const float rem = fmaf(-__builtin_bit_cast(float, m), d[2], x * d[1]);
    const uint32_t away = m + 1u, back = m - 1u;
    const uint32_t side = (rem > 0.f) == (q > 0.f) ? away : back;
    return __builtin_bit_cast(float, rem == 0.f ? m : side);
}

// At most 4 when q is within two units in the last place of a number that ends
// in 19 zero bits. Below 2^-10 (zeros among them) and above 432 (the block's
// largest element among them, at 448) there is no middle: magnitudes are clamped
// to numbers of those ranges that do not end so.
__device__ __forceinline__ uint32_t near_middle(float q) {
    const uint32_t u = __builtin_bit_cast(uint32_t, q) & 0x7FFFFFFFu;
    constexpr uint32_t kLow = 0x3A040000u, kHigh = 0x43DC0000u;  // 1.03 * 2^-11, 440
    return (min(max(u, kLow), kHigh) + 2u) & 0x7FFFFu;
}

// Codes of four elements, in one dword; r(i) is the divisor's 2^-e r for x[i] and
// d(i) the whole of it, fetched only to settle.
template <typename R, typename D>
__device__ __forceinline__ uint32_t codes4(const f4& x, R r, D d) {
    float q[4];
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = x[i] * r(i);
        m[i] = near_middle(q[i]);
    }
    if (min(min(m[0], m[1]), min(m[2], m[3])) <= 4u) {
        // (not rare in bfloat16: elements and largest elements of few bits have
        // many quotients that are codes or middles)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = m[i] <= 4u ? settle(x[i], q[i], d(i)) : q[i];
    }
    const int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], c, true);
}

// Magnitudes as bits, whose order is that of the values (NaN and infinities at
// the top): an integer maximum needs no care for NaN.
constexpr uint32_t kInf = 0x7F800000u;
__device__ __forceinline__ uint32_t magnitude(float x) {
    return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
    const uint32_t m = magnitude(x);
    return m < kInf ? m : 0u;
}

}  // namespace fg
