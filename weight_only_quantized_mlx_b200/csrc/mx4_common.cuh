// The MX4 number format on the device: E2M1 codes (1 sign, 2 exponent, 1
// mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), eight per little-endian 32-bit
// word (the low nibble is the first column), and one E8M0 scale byte per 32
// columns: 2^(byte - 127), 255 = NaN.
#pragma once

#include "device_common.cuh"

namespace mlxq {

constexpr int kMxBlock = 32;  // columns per scale

// 2^(e - 127) as BF16 bits; byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ uint32_t e8m0_to_bf16(uint32_t e) {
    return e == 0u ? 0x0040u : (e == 255u ? 0x7FFFu : e << 7);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes J and J + 4 of a word (J = 0..3) as BF16 in the two halves of a
// register, times 2^-126: an E2M1 code's three magnitude bits, put at the
// bottom of the exponent field and the top of the mantissa, are the same
// number with the exponent bias of BF16 (code 1, the subnormal 0.5, becomes
// the BF16 subnormal 2^-127).  Multiplying by 2^126 is exact.
template <int J>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w) {
    const uint32_t em = J == 3 ? w >> 6 : (J == 2 ? w >> 2 : (J == 1 ? w << 2 : w << 6));
    const uint32_t sg = J == 3 ? w : (J == 2 ? w << 4 : (J == 1 ? w << 8 : w << 12));
    return (em & 0x01C001C0u) | (sg & 0x80008000u);
}

constexpr uint32_t kTwo126 = 0x7E807E80u;  // 2^126 twice, BF16

}  // namespace mlxq
