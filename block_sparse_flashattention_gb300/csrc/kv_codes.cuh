// 8-bit K/V codes: four at a time to and from fp32 (value 0 in the low byte).
#pragma once

#include <cstdint>

namespace bsattn {

// Two e4m3 codes (16 bits) as two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(const float (&y)[4]) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return r;
}

__device__ __forceinline__ void unpack_e4m3(uint32_t x, float (&y)[4]) {
    const uint32_t h[2] = {e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(x >> 16)};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(y[2 * i]), "=f"(y[2 * i + 1])
            : "r"(h[i]));
}

// y, |y| < 2^22, to the nearest integers (ties to even): adding 1.5 * 2^23 leaves the
// integer in the low bits of the sum, in two's complement.
__device__ __forceinline__ uint32_t pack_int8(const float (&y)[4]) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

__device__ __forceinline__ void unpack_int8(uint32_t x, float (&y)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)(int8_t)(x >> (8 * i));
}

// Four codes as two fp16 pairs (codes 0, 1 and codes 2, 3); exact.  An int8 code c is
// 1152 below the fp16 number whose bits are 0x6400 + (c + 128).
template <bool kInt8>
__device__ __forceinline__ void codes_to_f16x2(uint32_t x, uint32_t &lo, uint32_t &hi) {
    if constexpr (kInt8) {
        const uint32_t u = x ^ 0x80808080u;
        lo = __byte_perm(u, 0x64646464u, 0x4140);
        hi = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
    } else {
        lo = e4m3x2_to_f16x2(x & 0xffffu);
        hi = e4m3x2_to_f16x2(x >> 16);
    }
}

}  // namespace bsattn
