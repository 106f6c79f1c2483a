// q4.cuh -- device arithmetic on the 4-bit cache's codes.
#pragma once

#include "ptx.cuh"
#include "q4.h"

namespace pkv {

// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

// Packed adds and multiply-adds of a 16-bit type, one rounding.
template <typename T>
__device__ __forceinline__ uint32_t q4_add(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (Elem<T>::kBf16) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <typename T>
__device__ __forceinline__ uint32_t q4_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (Elem<T>::kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Untiled bulk copy of `bytes` (a multiple of 16, both addresses too).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// The same with an L2 priority for the lines it reads (an l2_policy_* value).
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                               uint64_t policy) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1], %2, [%3], %4;"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// A word of eight codes -> the eight channels they stand for, in order, two to a
// register: s * (c - 8) + m in one rounding. A code at mantissa bits 0-3 under
// 2^10 (2^7 in bf16) reads 1024 + c (128 + c); s2 and m2 hold s and m twice.
template <typename T>
__device__ __forceinline__ void q4_values(uint32_t w, uint32_t s2, uint32_t m2, uint32_t (&out)[4]) {
    constexpr uint32_t kOne = Elem<T>::kBf16 ? 0x43004300u : 0x64006400u;
    constexpr uint32_t kBack = Elem<T>::kBf16 ? 0xc308c308u : 0xe408e408u;   // minus that and 8
    const uint32_t up = w >> 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // byte e: its low half to the low 16 bits, its high half to the high 16
        const uint32_t two = __byte_perm(w, up, uint32_t(e | ((4 + e) << 8)));
        out[e] = q4_fma<T>(q4_add<T>(and_or(two, 0x000f000fu, kOne), kBack), s2, m2);
    }
}

// The four codes in each 16-bit half of w, as fp16 values c - 8 (exact): out[i]
// holds nibble i of the low half in its low half and nibble i of the high
// half in its high half. Two exponents cover four nibbles with one shift: a
// nibble at mantissa bits 0-3 under 2^10 reads 1024 + c, one at bits 4-7
// reads 1024 + 16 c, which one fused multiply-add takes to c - 8. (Integers
// under a float's exponent are a published method of products with 4-bit
// weights; the constants follow from the format.)
__device__ __forceinline__ void q4_codes(uint32_t w, uint32_t (&out)[4]) {
    const uint32_t up = w >> 8;
    const uint32_t a = and_or(w, 0x000f000fu, 0x64006400u);
    const uint32_t b = and_or(w, 0x00f000f0u, 0x64006400u);
    const uint32_t c = and_or(up, 0x000f000fu, 0x64006400u);
    const uint32_t d = and_or(up, 0x00f000f0u, 0x64006400u);
    out[0] = hadd2_u(a, 0xe408e408u);                  // - 1032
    out[1] = hfma2_u(b, 0x2c002c00u, 0xd480d480u);     // / 16 - 72
    out[2] = hadd2_u(c, 0xe408e408u);
    out[3] = hfma2_u(d, 0x2c002c00u, 0xd480d480u);
}

// The same codes as fp16 values 64 + c: a nibble at mantissa bits 4-7 under 2^6.
// Three shifts and four and-or's, for a product whose offset is taken off its sum.
__device__ __forceinline__ void q4_codes_64(uint32_t w, uint32_t (&out)[4]) {
    out[0] = and_or(w << 4, 0x00f000f0u, 0x54005400u);
    out[1] = and_or(w, 0x00f000f0u, 0x54005400u);
    out[2] = and_or(w >> 4, 0x00f000f0u, 0x54005400u);
    out[3] = and_or(w >> 8, 0x00f000f0u, 0x54005400u);
}

// D = A (16x16) * B (16x8), fp32 sums from zero.
template <bool kBf16>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    }
}

// One (s, m) word as two floats.
template <typename T>
__device__ __forceinline__ float2 q4_pair(uint32_t w) {
    return Elem<T>::unpack2(w);
}

}  // namespace pkv
