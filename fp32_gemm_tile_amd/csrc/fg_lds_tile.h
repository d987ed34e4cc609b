// Device-side helpers of the kernels whose tiles go from memory straight to LDS:
// the loads, and the workgroup-to-tile mapping.
#pragma once

#include "fg_device.h"

namespace fg {

typedef int i4v __attribute__((ext_vector_type(4)));

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

// One element of SIZE bytes per lane, with zeros above it, to lds + 4 l.
template <int SIZE>
__device__ __forceinline__ void dma_element(i4v r, uint32_t lds, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (SIZE == 4)
        dma4(r, lds, off);
    else if constexpr (SIZE == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, 0 offen lds"
                     :
                     : "s"(lds), "v"(off), "s"(r)
                     : "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds"
                     :
                     : "s"(lds), "v"(off), "s"(r)
                     : "m0");
#else
    (void)r, (void)lds, (void)off;
#endif
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

}  // namespace fg
