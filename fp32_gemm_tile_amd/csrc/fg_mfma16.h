// The 16 x 16 matrix instructions on 16-byte pieces of k, and pieces at a row's end: shared by
// the kernels of the gated block and of 4-bit weights.
#pragma once

#include "fg_lds_tile.h"

namespace fg {

// Lane (n, g) = (lane % 16, lane / 16) gives 16 bytes of k of row n of both operands and gets
// rows 4 g to 4 g + 3 of a's, in column n of b's.
template <bool BF16>
__device__ __forceinline__ f4 mfma16(i4v a, i4v b, f4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (BF16) {
        typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                    __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    } else {
        const f4 fa = __builtin_bit_cast(f4, a), fb = __builtin_bit_cast(f4, b);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[e], fb[e], c, 0, 0, 0);
    }
#else
    (void)a, (void)b;
#endif
    return c;
}

// Elements [0, left) of a 16-byte piece, zeros after them.
template <bool BF16>
__device__ __forceinline__ i4v keep(i4v v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if constexpr (!BF16) {
            v[d] = d < left ? v[d] : 0;
        } else {
            const int n = left - 2 * d;
            v[d] &= n >= 2 ? -1 : (n == 1 ? 0xFFFF : 0);
        }
    }
    return v;
}

}  // namespace fg
