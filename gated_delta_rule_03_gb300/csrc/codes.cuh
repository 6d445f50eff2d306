// codes.cuh -- 8-bit codes of a paged cache: to fp16 (exact) and from fp32 (nearest even).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {
namespace codes {

// Two e4m3 codes (low byte first) as two fp16 numbers. Every e4m3 number is an fp16 one.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// Four codes of a word as fp16 pairs: lo holds bytes 0 and 1, hi bytes 2 and 3.
template <int kCode> __device__ __forceinline__ void to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (kCode == GDR_CODE_E4M3) {
        lo = e4m3x2_to_f16x2((uint16_t)(w & 0xffffu));
        hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
    } else {
        // 0x6400 + u is the fp16 number 1024 + u; with u = code + 128 the rest is a subtraction
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 x = __hsub2(reinterpret_cast<const __half2 &>(a), off);
        const __half2 y = __hsub2(reinterpret_cast<const __half2 &>(b), off);
        lo = reinterpret_cast<const uint32_t &>(x);
        hi = reinterpret_cast<const uint32_t &>(y);
    }
}

// Two numbers within the codes' range to the nearest codes, a in the low byte.
template <int kCode> __device__ __forceinline__ uint32_t from_f32x2(float a, float b) {
    if constexpr (kCode == GDR_CODE_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    } else {
        const int x = __float2int_rn(fminf(fmaxf(a, -127.f), 127.f)), y = __float2int_rn(fminf(fmaxf(b, -127.f), 127.f));
        return ((uint32_t)x & 0xffu) | (((uint32_t)y & 0xffu) << 8);
    }
}

// Exponent of the least power of two that, times the largest code, reaches a positive finite fp32
// number with these bits: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6. Held to [-60, 60].
template <int kCode> __device__ __forceinline__ int scale_exponent(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127;
    const uint32_t m = bits & 0x7fffffu;
    const int k = kCode == GDR_CODE_E4M3 ? e - 8 + (m > 0x600000u) : e - 6 + (m > 0x7e0000u);
    return min(max(k, -60), 60);
}
__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((k + 127) << 23); }

}  // namespace codes
}  // namespace gdr
