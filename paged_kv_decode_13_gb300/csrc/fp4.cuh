// The 4-bit K/V format (PKV_FP4) and its conversions (sm_103a).
//
// Sixteen consecutive head_dim columns of one token and kv head share a
// scale s; a value is s * e2m1, the eight magnitudes {0, 0.5, 1, 1.5, 2, 3, 4,
// 6} with a sign.  The scale is an unsigned 8-bit float of 5 exponent and 3
// mantissa bits (e5m3): its byte shifted left by 7 is the fp16 number it
// stands for, so decoding is one shift, and its range (2^-17 .. 10240, where
// 6 s still fits fp16) needs no second scale for the tensor, which a scale
// with 4 exponent bits would.  s * e2m1 has at most 6 significant bits: exact in
// fp16, so the tensor-core products below see the stored values themselves.
//
// A page block holds one kv head of one page: 8 D bytes of codes, D bytes of
// scales (16 tokens, D = head_dim).
//   K: code of (token, column) in byte token * D / 2 + column / 2, even
//      columns in the low nibble; its scale at 8 D + token * D / 16 + column / 16.
//      Lane (g, t) = (lane / 4, lane % 4) of a warp reads tokens g and g + 8,
//      columns t * D / 4 ..: the A fragments of S^T = K Q^T, whose contraction
//      order is free as long as Q follows it.
//   V: token = 8 hi + 2 t + n, column = g * D / 8 + 8 p + i: byte
//      512 p + 16 (4 g + t) + 2 i + hi, nibble n; its scale at
//      8 D + 4 (4 (column / 16) + t) + 2 hi + n.  A byte is a token pair of one
//      column, which is what the A fragments of O^T = V^T P^T hold, and lane
//      (g, t) reads 16 contiguous bytes per plane p, one scale word per 16
//      columns.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pkv {

constexpr unsigned kScaleMax = 0xE2;  // 10240: 6 * 10240 is the largest such product below 65504
constexpr unsigned kScaleNan = 0xFF;  // an fp16 NaN: a group with a NaN reads back as NaN

// Bytes of a page block of one kv head (K or V).
__host__ __device__ constexpr int block4_bytes(int head_dim) { return 9 * head_dim; }

// Scale byte of a group whose largest magnitude has the float bits `amax`
// (NaN payloads compare above infinity; a bf16 number): nearest e5m3 to max / 6,
// ties to even.  max / 6 is on a border between two scales (a number of at most
// 5 significant bits) or at least 2^-10 of it away, and max * (1 / 6) is within
// 2^-23 of it: rounded to 16 significant bits it is on the same side, or on the
// border exactly.
__device__ __forceinline__ unsigned scale4_of(unsigned amax) {
    if (amax > 0x7f800000u) return kScaleNan;
    const unsigned u = (__float_as_uint(__uint_as_float(amax) * 0.16666667f) + 0x80u) & ~0xffu;
    if (u < 0x38800000u) return (unsigned)__float2int_rn(__uint_as_float(u) * 131072.f);  // steps of 2^-17 below 2^-14
    return min(((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3), kScaleMax);
}
// 1 / scale to within 2^-22 (0 for a zero scale, whose codes are all 0).
__device__ __forceinline__ float scale4_inverse(unsigned byte) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(__half2float(__ushort_as_half((unsigned short)(byte << 7)))));
    return byte ? r : 0.f;
}
// Eight floats to eight e2m1 codes, x[0] in the low nibble (nearest, ties to
// even, saturating at 6).
__device__ __forceinline__ unsigned pack_e2m1x8(const float (&x)[8]) {
    unsigned r;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// The four bytes of a code word as fp16 pairs (low nibble first).
__device__ __forceinline__ void unpack_e2m1x8(unsigned (&h)[4], unsigned w) {
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ unsigned hmul2(unsigned a, unsigned b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const unsigned *>(&r);
}
// A scale byte in both halves of an fp16 pair.
__device__ __forceinline__ unsigned scale4_both(unsigned byte) { return byte * 0x00800080u; }
// Scale bytes i and i + 1 of a word as an fp16 pair.
__device__ __forceinline__ unsigned scale4_pair(unsigned w, int i) {
    return __byte_perm(w, 0u, 0x4040u | (unsigned)(i | ((i + 1) << 8))) << 7;
}

}  // namespace pkv
