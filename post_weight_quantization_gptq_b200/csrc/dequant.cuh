// Dequantization on the fp32 / integer pipes: packed codes -> bf16 weights
//   W_hat = bf16( fp32(s) * (q - z) )   (fp32 product, rounded to nearest-even bf16)
// shared by the tensor-core products with a packed layer.
#pragma once

#include "common.cuh"

namespace gptq {

// Pairs of fp32 values in one 64-bit register, operated on by the packed
// f32x2 instructions of sm_100 (one instruction, two IEEE round-to-nearest
// results: the same values as two scalar operations).
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// x rounded to the nearest bf16 (ties to even), as an fp32 whose low 16 bits
// are zero, on the fp32 pipe: Veltkamp's split with the factor 2^16 + 1,
// c = x (2^16 + 1), hi = c - (c - x), keeps the 8 leading significant bits of
// x rounded to nearest-even (|x| < 2^111); checked against the integer
// rounding rule on random values and exact ties.  It needs each step rounded
// on its own: the scalar intrinsics below are never fused into an fma,
// whereas the packed f32x2 form of the same steps was (its product merged
// into the subtraction after it, which turned the rounding into truncation:
// a one-ulp bf16 error that the parity test caught).  The conversion
// instruction runs on the narrow conversion pipe, which the dequantization
// saturated (ncu: 102 % of its peak); this form does not use it.
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    const float c = __fmul_rn(x, 65537.f);
    return __float_as_uint(__fsub_rn(c, __fsub_rn(c, x)));
}
// both values of a pair as one bf16x2 word (the low value in the low half)
__device__ __forceinline__ uint32_t bf16x2_rne(uint64_t v) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return __byte_perm(bf16_bits(lo), bf16_bits(hi), 0x7632);
}

// The eight codes of chunk c (codes 8c .. 8c+7 of the stage's row) as the
// floats 2^23 + q: each code's bits land in the mantissa of 2^23 (a byte
// permute against the exponent byte 0x4B where a code fills its own byte;
// no int-to-float conversion).
template <int BITS>
__device__ __forceinline__ void chunk_codes(const uint32_t* w, int c, float (&f)[8]) {
    constexpr uint32_t kMagic = 0x4B000000u;
    if constexpr (BITS == 4) {
        const uint32_t x = w[c];
        const uint32_t ev = x & 0x0F0F0F0Fu;          // codes 0, 2, 4, 6 in bytes 0..3
        const uint32_t od = (x >> 4) & 0x0F0F0F0Fu;   // codes 1, 3, 5, 7
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            f[2 * b] = __uint_as_float(__byte_perm(ev, kMagic, 0x7440 + b));
            f[2 * b + 1] = __uint_as_float(__byte_perm(od, kMagic, 0x7440 + b));
        }
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float(__byte_perm(w[2 * c + (i >> 2)], kMagic, 0x7440 + (i & 3)));
    } else {
        const uint32_t h = w[c >> 1] >> (16 * (c & 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(((h >> (2 * i)) & 3u) | kMagic);
    }
}

// prmt.b32 in its default mode: each selector nibble picks one of the 8
// bytes of (a, b); with the nibble's top bit set the picked byte's sign bit
// fills the result byte (0x00 or 0xFF).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// The 16 dequantized weights a 4-bit row group can take, bf16(s (q - z)) for
// q = 0..15 with the same arithmetic as the direct path, as byte tables: lo[j]
// holds the low bytes of entries 4j .. 4j+3, hi[j] their high bytes.
__device__ __forceinline__ void build_table4(float s, float z, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
    const uint64_t s2 = pk2(s, s), z2 = pk2(z, z);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r[4];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float q0 = static_cast<float>(4 * j + 2 * p);
            const uint64_t v = mul2(sub2(pk2(q0, q0 + 1.f), z2), s2);  // q - z exact, one rounding
            float a, b;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
            r[2 * p] = bf16_bits(a);        // bf16 in the high half
            r[2 * p + 1] = bf16_bits(b);
        }
        const uint32_t u01 = __byte_perm(r[0], r[1], 0x7362);  // lo0 lo1 hi0 hi1
        const uint32_t u23 = __byte_perm(r[2], r[3], 0x7362);
        lo[j] = __byte_perm(u01, u23, 0x5410);
        hi[j] = __byte_perm(u01, u23, 0x7632);
    }
}

// The bf16 weights of the eight 4-bit codes of x (code i in bits 4i..4i+3) as
// four bf16x2 words, by table look-up: a byte permute selects each code's
// entry among 8 by its low three bits, in the tables' first and second
// halves, and its fourth bit picks the half.
__device__ __forceinline__ void lookup8(uint32_t x, const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                        uint32_t (&o)[4]) {
    const uint32_t xs = x << 4;  // a code's fourth bit at the top of a byte, even codes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = (x >> (16 * h)) & 0x7777u;
        // 0xFF in byte i where code 4h + i is 8 or more (odd codes' fourth bit
        // is already the top of a byte of x)
        const uint32_t m = prmt(xs, x, h == 0 ? 0xD9C8u : 0xFBEAu);
        const uint32_t la = prmt(lo[0], lo[1], sel), lb = prmt(lo[2], lo[3], sel);
        const uint32_t ha = prmt(hi[0], hi[1], sel), hb = prmt(hi[2], hi[3], sel);
        const uint32_t L = (la & ~m) | (lb & m), H = (ha & ~m) | (hb & m);
        o[2 * h] = __byte_perm(L, H, 0x5140);      // codes 4h, 4h + 1
        o[2 * h + 1] = __byte_perm(L, H, 0x7362);  // codes 4h + 2, 4h + 3
    }
}

}  // namespace gptq
