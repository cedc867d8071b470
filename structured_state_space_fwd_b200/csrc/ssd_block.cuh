// Device helpers of the operators around the layer: bf16 pairs, SiLU and softplus in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 2^x and 1/x on the special-function unit (2 and 1 ulp).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// v / (1 + exp(-v)): 0 below about -87.3, where the reciprocal of a divisor above 2^126 is flushed (exact:
// above -1.1e-36), NaN for -inf as the formula.
__device__ __forceinline__ float silu(float v) { return v * rcp(1.f + ex2(-kLog2e * v)); }

// Packed pairs of fp32 values, and the same names for one.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float2 mul_(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add_(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 ex2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
__device__ __forceinline__ float2 rcp(float2 v) { return make_float2(rcp(v.x), rcp(v.y)); }
__device__ __forceinline__ float2 silu(float2 v) {
    return mul_(v, rcp(add_(ex2(mul_(v, both(-kLog2e))), both(1.f))));
}
template <typename T>
__device__ __forceinline__ T all(float v) {
    if constexpr (sizeof(T) == 8) return both(v);
    else return v;
}

// 2^(x y), a decay, for exponents mostly in (-1, 0]. The unit's results there lie low, by 2e-8 on
// average where the exponent is between -0.25 and -0.003 (measured), which a state collects at every
// token of its memory; 1.5e-8 more on the exponent halves that, and leaves 2^0 exactly 1.
constexpr float kCentre = 1.5e-8f;
template <typename T>
__device__ __forceinline__ T decay_of(T x, T y) { return ex2(fma_(x, y, all<T>(kCentre))); }
// A decay's rate A in powers of 2, finite below (NaN stays NaN): A = -inf, or one whose product with log2(e)
// is, forgets at every step above 0, and the steps of 0 behind a sequence's end leave the state as it is.
__device__ __forceinline__ float rate_of(float a) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a * kLog2e), "f"(-3.402823466e38f));
    return r;
}
__device__ __forceinline__ float2 rate_of(float2 a) { return make_float2(rate_of(a.x), rate_of(a.y)); }
// -|v|, not below -126: exp is 0 there; keeps infinities finite, and NaN NaN
__device__ __forceinline__ float neg_abs(float v) {
    const float m = -fabsf(v);
    return m < -126.f ? -126.f : m;
}
__device__ __forceinline__ float2 neg_abs(float2 v) { return make_float2(neg_abs(v.x), neg_abs(v.y)); }
__device__ __forceinline__ float positive(float v) { return fmaxf(v, 0.f); }
__device__ __forceinline__ float2 positive(float2 v) { return make_float2(positive(v.x), positive(v.y)); }
// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], of one value or two. With
// s = e / (2 + e) in (0, 1/3], log1p(e) = 2 atanh(s) = 2 s (1 + q P(q)), q = s^2 in (0, 1/9]; P
// interpolates (atanh(sqrt q) / sqrt q - 1) / q in four Chebyshev nodes, which leaves a relative
// error of 1.6e-8. So small steps keep their precision, which log(1 + e) would lose; the rounding
// of the exponent v log2(e), of its product and of the constant, moves e by at most 1.22 2^-24 |v|.
template <typename T>
__device__ __forceinline__ T softplus(T v) {
    const T e = ex2(mul_(neg_abs(v), all<T>(kLog2e)));
    const T s = mul_(e, rcp(add_(e, all<T>(2.f))));
    const T q = mul_(s, s);
    T p = fma_(q, all<T>(0.1342574954f), all<T>(0.1411830932f));
    p = fma_(p, q, all<T>(0.2000378072f));
    p = fma_(p, q, all<T>(0.3333331943f));
    p = fma_(p, q, all<T>(1.f));
    return fma_(mul_(s, all<T>(2.f)), p, positive(v));
}

}  // namespace ssd
