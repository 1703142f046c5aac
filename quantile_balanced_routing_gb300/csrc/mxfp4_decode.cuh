// Decoding MXFP4 (OCP MX: E2M1 elements, one E8M0 scale per 32).
#pragma once

#include "common.cuh"

namespace qb {

// ---- MXFP4 (OCP MX: E2M1 elements, E8M0 scale per 32) -> bf16 ----------------
// E2M1 magnitude index i = code & 7 has value {0, .5, 1, 1.5, 2, 3, 4, 6}[i].
// Times 2^d its bf16 has exponent field f_i + d with f = {-, 126, 127, 127,
// 128, 128, 129, 129} and mantissa {0, 0, 0, 0x40, 0, 0x40, 0, 0x40}; the
// decode is exact while every field stays in [1, 254] (|d| <= 125).
QB_DEV float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7u;
    const float v = m < 4u ? 0.5f * (float)m : (m < 6u ? (float)m - 2.0f : 2.0f * (float)m - 8.0f);
    return (code & 8u) ? -v : v;
}

// E8M0 byte -> scale (0xFF: NaN).
QB_DEV float e8m0_value(uint32_t b) {
    return b == 0xffu ? __int_as_float(0x7fffffff) : __int_as_float(b ? (int)(b << 23) : 0x00400000);
}

// High and low bytes of the eight magnitudes' bf16 at scale 2^d, packed four
// per register for byte-permute lookups (h[0]/l[0]: indices 0-3, h[1]/l[1]: 4-7).
__device__ __forceinline__ void mx_tables(int d, uint32_t (&h)[2], uint32_t (&l)[2]) {
    const uint32_t a = 126 + d, b = a + 1, c = a + 2, e = a + 3;   // exponent fields
    h[0] = ((a >> 1) << 8) | ((b >> 1) << 16) | ((b >> 1) << 24);
    h[1] = (c >> 1) | ((c >> 1) << 8) | ((e >> 1) << 16) | ((e >> 1) << 24);
    l[0] = ((a & 1u) << 15) | ((b & 1u) << 23) | (((b & 1u) << 31) | (0x40u << 24));
    l[1] = ((c & 1u) << 7) | ((((c & 1u) << 7) | 0x40u) << 8) | ((e & 1u) << 23) | ((((e & 1u) << 7) | 0x40u) << 24);
}

// Eight E2M1 codes of one 32-bit word (code j in bits 4j..4j+3) -> four bf16
// pairs (elements 2q and 2q+1 in o[q]).
__device__ __forceinline__ void mx_decode_word(uint32_t w, const uint32_t (&h)[2], const uint32_t (&l)[2],
                                               uint32_t (&o)[4]) {
    const uint32_t sel0 = w & 0x7777u, sel1 = (w >> 16) & 0x7777u;     // magnitudes of codes 0-3, 4-7
    const uint32_t h0 = __byte_perm(h[0], h[1], sel0), l0 = __byte_perm(l[0], l[1], sel0);
    const uint32_t h1 = __byte_perm(h[0], h[1], sel1), l1 = __byte_perm(l[0], l[1], sel1);
    o[0] = __byte_perm(l0, h0, 0x5140);
    o[1] = __byte_perm(l0, h0, 0x7362);
    o[2] = __byte_perm(l1, h1, 0x5140);
    o[3] = __byte_perm(l1, h1, 0x7362);
    // sign of code 2q is bit 3 of byte q (-> bit 15), of code 2q+1 bit 7 (-> bit 31)
    const uint32_t w4 = w << 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] |= __byte_perm(w, w4, (q << 12) | ((4 + q) << 4)) & 0x80008000u;
}

// An E2M1 code's magnitude in bits 6..8 of a bf16 (two exponent bits and one of the
// mantissa) and its sign in bit 15 are the code's value times 2^-126, subnormals
// included: one exact product with 2^126 times the scale decodes it.  The factor as
// a pair of bf16; scales from 2^2 on, whose factor has no bf16, take 2^126 first
// (mx_rescale).
constexpr uint32_t kMxLargeScale = 129;   // 2^2
QB_DEV __nv_bfloat162 mx_factor(uint32_t sc) {
    const uint32_t b = (sc < kMxLargeScale ? sc + 126u : 253u) << 7;
    const uint32_t bb = b * 0x10001u;
    return *reinterpret_cast<const __nv_bfloat162*>(&bb);
}
QB_DEV uint32_t mx_mul2(uint32_t v, __nv_bfloat162 f) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), f);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight E2M1 codes of one word -> four bf16 pairs times the factor: elements q and
// q + 4 in o[q], the two that lie 16 bits apart in the word (memory order would
// take another four permutations).
QB_DEV void mx_decode_pairs(uint32_t w, __nv_bfloat162 factor, uint32_t (&o)[4]) {
    constexpr uint32_t S = 0x80008000u, M = 0x01c001c0u;
    o[0] = mx_mul2(((w << 12) & S) | ((w << 6) & M), factor);
    o[1] = mx_mul2(((w << 8) & S) | ((w << 2) & M), factor);
    o[2] = mx_mul2(((w << 4) & S) | ((w >> 2) & M), factor);
    o[3] = mx_mul2((w & S) | ((w >> 6) & M), factor);
}

// The rest of a scale from 2^2 on (an overflow gives infinity, as rounding the
// value would; 0xFF gives NaN).
QB_DEV void mx_rescale(uint32_t sc, uint32_t (&o)[4]) {
    const uint32_t b = (sc == 255u ? 0x7fffu : sc << 7) * 0x10001u;
    const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = mx_mul2(o[q], scale);
}

}  // namespace qb
