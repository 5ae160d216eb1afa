// gdn_f32x2.cuh -- pairs of fp32 values in one 64-bit register and the packed
// arithmetic of sm_100 on them (one instruction for two operations, each
// rounded as the scalar one).
#pragma once

#include <stdint.h>

namespace gdn {

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float lo_of(f32x2 x) { return __uint_as_float(uint32_t(x)); }
__device__ __forceinline__ float hi_of(f32x2 x) { return __uint_as_float(uint32_t(x >> 32)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// The two bf16 values of a 32-bit word.
__device__ __forceinline__ f32x2 from_bf16x2(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Two values rounded to bf16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t to_bf16x2(f32x2 x) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi_of(x)), "f"(lo_of(x)));
    return r;
}

}  // namespace gdn
