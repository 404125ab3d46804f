// Two fp32 values at a time: the paired instructions do the work of two in one issue slot (measured on this chip:
// 1.92 paired FMAs a clock and SM against 3.83 single ones, so the lanes are the same and the issue slots half).
#pragma once

#include "common.cuh"

namespace gdr {

typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Exponentials and reciprocals are the hardware's approximations (relative error 2^-22 and 2^-23 at most, results below
// 2^-126 flushed): one instruction each, where expf and a division take several.  What that costs was measured against 64 bits: the scan's states after 8,192 and 16,384 tokens at a memory of 2,000 and 20,000
// are off by 9e-7 and 2e-6, its dA by 1.4e-6 and 3.2e-6 (a plain fp32 recurrence with expf: 2e-5 and 9e-5, 4e-5 and 1e-4).

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 ex2x2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ f2 rcpx2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(rcp(a), rcp(b));
}
// 1 / (1 + e^-x): where e^-x overflows the reciprocal of infinity is the 0 wanted.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-x * LOG2E)); }
__device__ __forceinline__ f2 sigmoid2(f2 x) { return rcpx2(add2(ex2x2(mul2(x, both(-LOG2E))), both(1.f))); }

// Two 16-bit elements in one word.
template <typename T>
__device__ __forceinline__ f2 widen2(uint32_t u) {
    const float2 f = Elt<T>::unpack(u);
    return pack2(f.x, f.y);
}
template <>
__device__ __forceinline__ f2 widen2<__nv_bfloat16>(uint32_t u) {  // a bf16 is the upper half of its fp32
    return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return Elt<T>::pack(a, b);
}

}  // namespace gdr
