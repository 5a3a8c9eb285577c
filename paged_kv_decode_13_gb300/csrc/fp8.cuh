// The 8-bit K/V format (PKV_FP8) and its conversions (sm_103a).
//
// The 16 tokens of a page and kv head share one scale, a power of two 2^e; a
// value is 2^e * e4m3.  e4m3 is a floating-point number itself (4 significant
// bits from 2^-6 to 448, steps of 2^-9 below), so a power of two loses no
// precision against any other scale, and moving a page to a larger one only
// lowers the codes' exponents: exact but for values below 2^-6 2^e, 2^-14 of the
// page's largest.  That is what lets a page be filled token by token: a token
// that does not fit raises e, and the tokens before it follow.
//
// A block (one kv head of one page, D = head_dim) is 16 D bytes of codes, token
// after token, then 16 bytes: the biased exponent e + 127 (0: no scale yet, all
// values zero), a zero byte, a 16-bit mask of the tokens that hold a NaN (a NaN's
// code is 0; the whole token reads back as NaN), twelve bytes that are not used.  The
// 16-byte chunk c of a token's row is in place place8(): lane (g, t) = (lane /
// 4, lane % 4) reads chunks t + 4 i of tokens g and g + 8 (K) or chunks g + 8 i of
// tokens 2 t, 2 t + 1 and those 8 on (V), and the eight lanes that a 16-byte
// shared load serves at once meet no bank twice.  A row is contiguous, so an append
// writes whole sectors.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pkv {

constexpr unsigned kScaleMax8 = 246;  // 2^119: 448 * 2^119 is the largest such product in fp32

// Bytes of a page block of one kv head (K or V).
__host__ __device__ constexpr int block8_bytes(int head_dim) { return 16 * head_dim + 16; }
// Place of 16-byte chunk `c` of token `t`'s row.
__host__ __device__ constexpr int place8(int t, int c, int head_dim) { return c ^ (((t & 6) ^ ((t & 1) << 2)) & (head_dim / 16 - 1)); }

// Biased exponent of the smallest scale under which the largest magnitude, of float
// bits `amax` (no NaN; a bf16 number), fits 448 = 1.75 * 2^8; an infinity saturates.
__device__ __forceinline__ unsigned scale8_of(unsigned amax) {
    if (amax == 0) return 0;
    return (unsigned)min(max((int)((amax + 0x1fffffu) >> 23) - 8, 1), (int)kScaleMax8);
}
__device__ __forceinline__ float scale8_value(unsigned b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float scale8_inverse(unsigned b) { return __uint_as_float((254u - b) << 23); }  // b <= kScaleMax8

// Four floats to four e4m3 codes, a in the low byte (nearest, ties to even, saturating at 448).
__device__ __forceinline__ unsigned pack_e4m3x4(float a, float b, float c, float d) {
    unsigned r;
    asm("{\n .reg .b16 x, y;\n"
        " cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
        " mov.b32 %0, {x, y};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// The four bytes of a code word as two fp16 pairs, low byte first (exact).
__device__ __forceinline__ void unpack_e4m3x4(unsigned &lo, unsigned &hi, unsigned w) {
    asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 half2_floats(unsigned h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
// The codes of a word, their values times `by` (saturating).
__device__ __forceinline__ unsigned scale_e4m3x4(unsigned w, float by) {
    unsigned lo, hi;
    unpack_e4m3x4(lo, hi, w);
    const float2 a = half2_floats(lo), b = half2_floats(hi);
    return pack_e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
}

}  // namespace pkv
