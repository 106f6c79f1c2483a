// q8.cuh -- device arithmetic on the 8-bit cache's codes.
#pragma once

#include "ptx.cuh"
#include "q8.h"

namespace pkv {

// Two codes (the low and the high half of a word: bytes 0, 1 and 2, 3) as fp16, exact.
__device__ __forceinline__ void q8_halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// The same codes times 2^-120 as bf16, exact: a code's exponent and mantissa are where
// bf16 has its lowest exponent bits and its highest mantissa bits once it is moved up
// by 4 in its half, and a code below 2^-6 is below 2^-126 then, bf16's own small end.
// (Not for NaN codes, which come out as 480 * 2^-120.)
__device__ __forceinline__ void q8_bf16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    // a byte to the low half of 16 bits, its top bit to all of the high half
    asm("prmt.b32 %0, %2, 0, 0x9180;\n\tprmt.b32 %1, %2, 0, 0xb3a2;" : "=r"(lo), "=r"(hi) : "r"(w));
    lo = (lo << 4) & 0x87f087f0u;
    hi = (hi << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint32_t bmul2_u(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four floats, at most 448 in size or NaN, to codes, x0 in byte 0: ties to even.
__device__ __forceinline__ uint32_t q8_codes(float x0, float x1, float x2, float x3) {
    uint32_t w;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
        : "=r"(w) : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return w;
}

// A float of fp16's range twice, and packed products.
__device__ __forceinline__ uint32_t pack_half2(float x) { return Elem<__half>::pack2(x, x); }
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^e for e of [-126, 127], and the exponent of a scale.
__device__ __forceinline__ float q8_power(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
__device__ __forceinline__ int q8_exponent(float scale) { return int((__float_as_uint(scale) >> 23) & 255u) - 127; }

// The smallest e of a scale with top <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int q8_exponent_for(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kQ8LeastExp);
}

}  // namespace pkv
