// sv_pairs.cuh -- three-way maxima and fp32 arithmetic two at a time, as instructions.
#pragma once

#include <stdint.h>

namespace sv {

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two floats in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ uint64_t bits2(uint32_t a, uint32_t b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    return bits2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void unpair2(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

}  // namespace sv
