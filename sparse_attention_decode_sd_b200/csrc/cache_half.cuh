// cache_half.cuh -- 8-bit cache elements as half-precision tensor-core operands (mma.sync), which hold them exactly.
#pragma once

#include <cuda_fp16.h>

#include "cache_format.cuh"

namespace sd {

// The elements in the low (hi = 0) or high two bytes of w as a half-precision pair.  int8 as 1024 + (x + 128) less 1152.
template <int kFmt, int hi>
__device__ __forceinline__ uint32_t half_pair(uint32_t w) {
    uint32_t r;
    if (kFmt == kFmtFp8) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)(hi ? w >> 16 : w)));
    } else {
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w ^ 0x80808080u, 0x64646464u, hi ? 0x4342 : 0x4140)), "r"(0x64806480u));
    }
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with zeros in the lower eight rows of A: only the upper rows of the result are kept.
__device__ __forceinline__ void mma_f16_upper(float (&c)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    [[maybe_unused]] float x, y;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%8,%5,%8}, {%6,%7}, {%0,%1,%9,%9};\n"
        : "+f"(c[0]), "+f"(c[1]), "=f"(x), "=f"(y)
        : "r"(a0), "r"(a2), "r"(b0), "r"(b1), "r"(0u), "f"(0.f));
}

// What an element counts, times 2^(byte - 127) of its block.
template <int kFmt>
__device__ __forceinline__ constexpr float unit_of() {
    return kFmt == kFmtFp8 ? 1.f : 0.015625f;
}
// 2^(byte x of w - 127); byte 255 gives an infinity (NaN with the block's zeros), byte 0 zero (int8 blocks below 2^-126).
__device__ __forceinline__ float power_of(uint32_t w, int x) {
    return __uint_as_float((x == 0 ? w << 23 : x == 1 ? w << 15 : x == 2 ? w << 7 : w >> 1) & 0x7f800000u);
}

// `down`, the power of two that brings `big` (>= 0) into [1, 2) (as far as there is one), and its reciprocal.
__device__ __forceinline__ void power_of_two(float big, float& down, float& up) {
    const uint32_t bits = min(max(__float_as_uint(big) & 0x7f800000u, 0x00800000u), 0x7e800000u);
    down = __uint_as_float(0x7f000000u - bits);
    up = __uint_as_float(bits);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

}  // namespace sd
