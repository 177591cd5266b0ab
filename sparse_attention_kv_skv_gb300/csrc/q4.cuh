// The 4-bit form of a 576-value KV row, and the arithmetic between it and
// bf16.  A packed row is 336 bytes:
//   [0, 288)    e2m1 codes, value 2j in the low half of byte j, 2j + 1 in the high half;
//   [288, 324)  e4m3 scales, one for 16 consecutive values (36 groups);
//   324         the row's exponent e as e + 127;
//   [325, 336)  zeros (16-byte rows for the assembly's loads).
// Value i is code_i * scale_(i/16) * 2^e.  A code has 2 significant bits and a
// scale 4, so the product has at most 6 and is exact in bf16: whatever reads a
// packed row as bf16 reads exactly what it stands for.
#pragma once

#include <cstdint>

namespace skv {
namespace q4 {

constexpr int kDim = 576;
constexpr int kGroups = 36;     // of 16 values
constexpr int kRowBytes = 336;
constexpr int kScalesAt = 288, kExpAt = 324;

// Four bytes of codes (eight values) to four f16 pairs, the lower value in the low half.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// An f16 pair of e2m1 values (0, or exponent -1..2 and one fraction bit) as a
// bf16 pair: the sign stays, exponent and fraction move down by 3 bits, which
// reads as the value times 2^-112 (the difference of the two exponent
// biases); the product with 2^112 is exact and leaves 0 alone.
__device__ __forceinline__ uint32_t f16_codes_to_bf16(uint32_t h)
{
    const uint32_t t = (h & 0x80008000u) | ((h >> 3) & 0x0FFF0FFFu);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0x77807780u));  // 0x7780 = bf16 2^112
    return r;
}

// scale * 2^e as a bf16 pair (both halves): the factor of a group's codes.
// scale: an e4m3 byte; eb: the row's exponent byte.
__device__ __forceinline__ float scale_value(uint32_t scale)
{
    uint32_t h;
    asm("{\n .reg .b16 s;\n cvt.u16.u32 s, %1;\n cvt.rn.f16x2.e4m3x2 %0, s;\n}\n" : "=r"(h) : "r"(scale & 0xFFu));
    float f;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h));
    return f;
}
__device__ __forceinline__ uint32_t group_factor(uint32_t scale, uint32_t eb)
{
    const float f = scale_value(scale) * __uint_as_float(eb << 23);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(f));
    return r;
}

// Eight values of one group as four bf16 pairs.  Exact for rows whose values
// lie in bf16's normal range (every row that pack writes).
__device__ __forceinline__ uint4 decode8(uint32_t codes, uint32_t factor)
{
    uint32_t h[4], v[4];
    codes_to_f16(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(f16_codes_to_bf16(h[i])), "r"(factor));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

}  // namespace q4
}  // namespace skv
