// sv_quant.cuh -- the 4-bit form of a K or V row.
//
// Codes c_d (0 .. 15) and two bf16 numbers: x_d ~ minimum + step * c_d.  One
// step and minimum a row and head: K's are applied to the f32 scores (step * (q .
// (c - 8)) + (minimum + 8 step) * sum(q)), so that the products have to do with codes
// alone, which are exact in bf16 and f16.
//
// Eight codes are a word, dims 0, 2, 4, 6, 1, 3, 5, 7 from its lowest four bits
// up: the word shifted right by 4 i and masked has dims 2i and 2i + 1 in its two
// halves, a pair of bf16 in order.
#pragma once

#include <stdint.h>

namespace sv {
namespace quant {

constexpr float kFifteenth = 0.06666667014360428f;  // 1 / 15 in f32
constexpr float kSmallestStep = 1.1754943508222875e-38f;  // 2^-126: below it 1 / step may not be finite
constexpr uint32_t kNotFinite = 0x7fc00000u;        // step 0, minimum NaN: a row that has no encoding

// A pair of codes in the last four bits of each half, less 8, as a pair of bf16: in the last bits of
// 128 a code is 128 + code, and what is taken off is exact.
__device__ __forceinline__ uint32_t centred(uint32_t pair) {
    const uint32_t x = (pair & 0x000f000fu) | 0x43004300u;
    uint32_t c;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(0x43084308u));
    return c;
}
// The same as a pair of f16 (in the last bits of 1024).
__device__ __forceinline__ uint32_t centred_f16(uint32_t pair) {
    const uint32_t x = (pair & 0x000f000fu) | 0x64006400u;
    uint32_t c;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(0x64086408u));
    return c;
}
// A word's eight codes less 8 in bf16, dims 0 .. 7 in order.
__device__ __forceinline__ uint4 expand(uint32_t w) {
    return make_uint4(centred(w), centred(w >> 4), centred(w >> 8), centred(w >> 12));
}

// The same in f16: of a byte's two codes the second is 1024 + 16 code where it lies, so that the pairs
// of a word's bytes need no shifts but one.
__device__ __forceinline__ uint32_t centred_f16_high(uint32_t pair) {
    const uint32_t x = (pair & 0x00f000f0u) | 0x64006400u;
    uint32_t c;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(c) : "r"(x), "r"(0x2c002c00u), "r"(0xd480d480u));  // x / 16 - 72
    return c;
}
// A word's eight values in f16, each step * (code - 8) + middle rounded once (step and middle twice each).
__device__ __forceinline__ uint4 scaled_f16(uint32_t w, uint32_t step, uint32_t mid) {
    const uint32_t v = w >> 8;
    uint32_t x[4] = {centred_f16(w), centred_f16_high(w), centred_f16(v), centred_f16_high(v)};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x[i]) : "r"(x[i]), "r"(step), "r"(mid));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

}  // namespace quant
}  // namespace sv
