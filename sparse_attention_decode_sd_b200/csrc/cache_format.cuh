// cache_format.cuh -- the 8-bit cache formats (OCP microscaling: blocks of 32 values along the head
// dimension that share one power-of-two scale, stored as a biased exponent byte).
//
//   MXFP8    value = e4m3 element * 2^(byte - 127); the byte is that of the least exponent e in [-124, 119] with
//            amax <= 448 * 2^e (elements saturate at 448 where none is left).
//   MXINT8   value = int8 element * 2^(byte - 133) (the format's 2^-6 unit times 2^(byte - 127)), elements
//            -127 .. 127; the byte is that of the least exponent e in [-133, 121] for which amax * 2^-e
//            rounds to at most 127 (elements saturate at 127 where none is left).
//   Byte 255 marks a block that held an infinity or a NaN: its elements are zero and it reads as NaN.
//
// A power-of-two scale makes every step but the rounding of the elements exact, and every stored value
// exact in bf16 (4 or 7 significant bits; the limits of e keep the smallest steps at 2^-133, bf16's own
// smallest, and the largest values finite): what reads the cache in bf16 loses nothing.
#pragma once

#include "common.cuh"

namespace sd {

constexpr int kFmtBf16 = SD_CACHE_BF16, kFmtFp8 = SD_CACHE_MXFP8, kFmtInt8 = SD_CACHE_MXINT8;
constexpr int kBlock = 32;                      // values that share a scale
constexpr int kScaleBytes = kHeadDim / kBlock;  // scale bytes of one K or V row: 4

// Scale byte of a block whose largest magnitude has the (non-negative) fp32 bits `amax`; the values are
// bf16, so the low 16 bits are zero and bits 16-22 are the whole mantissa.
template <int kFmt>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int ex = (int)(amax >> 23), m7 = (int)((amax >> 16) & 0x7f);
    if (ex == 255) return 255u;
    if (kFmt == kFmtFp8) {       // 448 = 1.75 * 2^8
        const int e = ex - 127 - 8 + (m7 > 0x60 ? 1 : 0);
        return (uint32_t)(min(max(e, -124), 119) + 127);
    }
    // 127.5 = (1 + 127/128) * 2^6; a subnormal amax (ex = 0) is below 127.5 * 2^-133
    const int e = ex == 0 ? -133 : ex - 127 - 6 + (m7 == 0x7f ? 1 : 0);
    return (uint32_t)(min(e, 121) + 133);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four values (two bf16 pairs) to elements, one byte each, the first in the low byte: the values times 2^-e for the
// block's byte (not 255), rounded to nearest, ties to even.  The product is exact in bf16 but for results below its
// range, which round to zero all the same.  (int8: 2^-e is beyond bf16 for the six smallest bytes, and the largest
// byte's elements may have to saturate: both rare, in a branch.)
template <int kFmt>
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, uint32_t byte) {
    if (kFmt == kFmtFp8) {
        const uint32_t f = (254u - byte) * 0x00800080u;   // 2^(127 - byte)
        a = mul_bf16x2(a, f);
        b = mul_bf16x2(b, f);
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(bf16_hi(a)), "f"(bf16_lo(a)));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(bf16_hi(b)), "f"(bf16_lo(b)));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    if (byte < 6u) {
        a = mul_bf16x2(a, 0x42804280u);   // 2^6, and 2^(127 - byte) below
        b = mul_bf16x2(b, 0x42804280u);
        byte += 6u;
    }
    const uint32_t f = (260u - byte) * 0x00800080u;   // 2^(133 - byte)
    a = mul_bf16x2(a, f);
    b = mul_bf16x2(b, f);
    float x[4] = {bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b)};
    if (byte == 254u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaxf(-127.f, fminf(127.f, x[i]));
    }
    uint32_t u[4];   // adding 1.5 * 2^23 rounds to an integer and leaves it in the low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(x[i] + 12582912.f);
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}

// The bf16 factors that turn expand4()'s values into the stored ones.  e4m3 elements come out of expand4
// 2^-120 too small (their exponent field sits in bf16's as it is), so the factor is 2^(e + 120): one bf16
// for e <= 7, else 2^120 and 2^e (`two`).  Byte 255 gives an infinity, which makes NaN of the block's zeros.
struct Factor {
    uint32_t f1, f2;   // the factor in both halves
    bool two;
};
template <int kFmt>
__device__ __forceinline__ Factor factor_of(uint32_t byte) {
    Factor f;
    f.f2 = 0x3f803f80u;
    f.two = false;
    uint32_t b;
    if (kFmt == kFmtFp8) {
        f.two = byte > 134u;
        b = f.two ? 0x7b80u : (byte + 120u) << 7;
        if (f.two) f.f2 = (byte << 7) * 0x10001u;
    } else {
        b = byte == 255u ? 0x7f80u : byte > 6u ? (byte - 6u) << 7 : 1u << byte;   // below 2^-126: subnormal
    }
    f.f1 = b * 0x10001u;
    return f;
}

// Bytes whose factor is one normal bf16 (nearly all: e from -124 to 7, or from -126 to 121), and that factor.
template <int kFmt>
__device__ __forceinline__ bool plain_factor(uint32_t byte) {
    return kFmt == kFmtFp8 ? byte <= 134u : byte - 7u <= 247u;
}
template <int kFmt>
__device__ __forceinline__ uint32_t factor_plain(uint32_t byte) {
    return (kFmt == kFmtFp8 ? byte + 120u : byte - 6u) * 0x00800080u;
}

// Four elements to two bf16 pairs, before the factor.
//   e4m3: sign to bit 15, exponent and mantissa to bits 4-10 of each half: the value times 2^-120, the
//         subnormals too.
//   int8: 0x4300 | (low 7 bits) is 128 + them, 0x4300 | (bit 7) is 128 or 256; the difference is exact.
template <int kFmt>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (kFmt == kFmtFp8) {
        const uint32_t a = __byte_perm(w, 0u, 0x4140), b = __byte_perm(w, 0u, 0x4342);   // the bytes in the low halves
        lo = a * 16u + (a & 0x00800080u) * 240u;   // up by 4, the sign by 8 (multiplications: the shifter is the busier pipe)
        hi = b * 16u + (b & 0x00800080u) * 240u;
    } else {
        const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140), b = __byte_perm(w, 0x43434343u, 0x4342);
        lo = sub_bf16x2(a & 0xff7fff7fu, a & 0xff80ff80u);
        hi = sub_bf16x2(b & 0xff7fff7fu, b & 0xff80ff80u);
    }
}

// Four elements of a block to two bf16 pairs, exactly the stored values.
template <int kFmt>
__device__ __forceinline__ void decode4(uint32_t w, const Factor& f, uint32_t& lo, uint32_t& hi) {
    expand4<kFmt>(w, lo, hi);
    lo = mul_bf16x2(lo, f.f1);
    hi = mul_bf16x2(hi, f.f1);
    if (kFmt == kFmtFp8 && f.two) {
        lo = mul_bf16x2(lo, f.f2);
        hi = mul_bf16x2(hi, f.f2);
    }
}

// Byte offset of the scales of (page, KV head, slot): K's four bytes, then V's.
__device__ __forceinline__ long scale_offset(long page, int kvh, int slot, int Hkv) {
    return ((page * Hkv + kvh) * kPageSize + slot) * (2 * kScaleBytes);
}

}  // namespace sd
