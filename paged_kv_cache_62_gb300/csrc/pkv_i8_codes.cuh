// int8 codes as f16 operands.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace pkv {

// V scales that count as they are (their log2 rides on the softmax weights, and the row sums divide it out).
constexpr float kMinVScale = 0x1p-104f, kMaxVScale = 0x1p+104f;

// Four int8 codes (byte e is element e) as f16 pairs picked by the two permute selectors (K operands take
// elements (0, 1) and (2, 3), V operands (0, 2) and (1, 3)), 1152 too large: the byte code + 128 under the high
// byte of 1024.
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ void i8x4_biased(uint32_t codes, uint32_t &a, uint32_t &b)
{
    const uint32_t u = codes ^ 0x80808080u;
    a = __byte_perm(u, 0x64646464u, SEL0);
    b = __byte_perm(u, 0x64646464u, SEL1);
}

// The same, exact.
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ void i8x4_to_f16x2x2(uint32_t codes, uint32_t &a, uint32_t &b)
{
    uint32_t x, y;
    i8x4_biased<SEL0, SEL1>(codes, x, y);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 hx = __hsub2(*reinterpret_cast<const __half2 *>(&x), off);
    const __half2 hy = __hsub2(*reinterpret_cast<const __half2 *>(&y), off);
    a = *reinterpret_cast<const uint32_t *>(&hx);
    b = *reinterpret_cast<const uint32_t *>(&hy);
}

}  // namespace pkv
