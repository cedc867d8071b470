// Device helpers of the operators around the layer: typed 1-, 4- and 8-element
// loads and stores, SiLU and softplus in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

// VW consecutive elements as they lie in memory: 16 bytes, or one element.
template <typename E, int VW>
struct Pack {
    using T = uint4;
};
template <typename E>
struct Pack<E, 1> {
    using T = E;
};

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

__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) {
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(float q, float (&v)[1]) { v[0] = q; }
__device__ __forceinline__ void unpack(__nv_bfloat16 q, float (&v)[1]) { v[0] = __bfloat162float(q); }

__device__ __forceinline__ void pack(const float (&v)[8], uint4& q) {
    q = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void pack(const float (&v)[4], uint4& q) {
    q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void pack(const float (&v)[1], float& q) { q = v[0]; }
__device__ __forceinline__ void pack(const float (&v)[1], __nv_bfloat16& q) { q = __float2bfloat16_rn(v[0]); }

template <typename P>
__device__ __forceinline__ P zero_pack() {
    if constexpr (sizeof(P) == 16) {
        return make_uint4(0, 0, 0, 0);
    } else {
        return P(0.f);
    }
}

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

// v / (1 + exp(-v)): 0 for very negative v (the divisor is inf), NaN for -inf as the formula.
__device__ __forceinline__ float silu(float v) { return v * rcp(1.f + ex2(-kLog2e * v)); }

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], of two values. With
// s = e / (2 + e) in (0, 1/3], log1p(e) = 2 atanh(s) = 2 s (1 + q P(q)), q = s^2 in (0, 1/9]; P
// interpolates (atanh(sqrt q) / sqrt q - 1) / q in four Chebyshev nodes, which leaves a relative
// error of 1.6e-8. So small steps keep their precision, which log(1 + e) would lose; the rounding
// of the exponent v log2(e) moves e by at most 2^-24 |v|.
__device__ __forceinline__ float2 softplus2(float2 v) {
    float2 m = make_float2(-fabsf(v.x), -fabsf(v.y));
    m.x = m.x < -126.f ? -126.f : m.x;      // e is 0 there; keeps infinities finite, and NaN NaN
    m.y = m.y < -126.f ? -126.f : m.y;
    const float2 one = make_float2(1.f, 1.f), two = make_float2(2.f, 2.f);
    float2 e = __fmul2_rn(m, make_float2(kLog2e, kLog2e));
    e = make_float2(ex2(e.x), ex2(e.y));
    const float2 d = __fadd2_rn(e, two);
    const float2 s = __fmul2_rn(e, make_float2(rcp(d.x), rcp(d.y)));
    const float2 q = __fmul2_rn(s, s);
    float2 p = __ffma2_rn(q, make_float2(0.1342574954f, 0.1342574954f), make_float2(0.1411830932f, 0.1411830932f));
    p = __ffma2_rn(p, q, make_float2(0.2000378072f, 0.2000378072f));
    p = __ffma2_rn(p, q, make_float2(0.3333331943f, 0.3333331943f));
    p = __ffma2_rn(p, q, one);
    return __ffma2_rn(__fmul2_rn(s, two), p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v) { return softplus2(make_float2(v, v)).x; }

}  // namespace ssd
