// E4M3 conversion and the dynamic scales of include/ep.h's quantisation modes,
// for the kernels that quantise fp32 values held in registers.
#pragma once

#include <cuda_fp8.h>

#include "ep_common.cuh"

namespace ep {

__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
    // __nv_cvt_float2_to_fp8x2: round to nearest even, saturate to +-448;
    // the first element of the pair lands in the low byte.
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
}

// The fp32 scale of a 1x128 group: s = max(amax, 1e-4) / 448, an IEEE
// round-to-nearest division.
__device__ __forceinline__ float group_scale(float amax) {
    return __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f);
}
// x / s to the nearest fp32, ep_dispatch's rule, without a division for each x:
// inv is 1 / s to the nearest, q the quotient's estimate, q * s - x its error, which
// one fused product-and-sum gives exactly, and q - error * inv rounds to the quotient
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000",
// IBM J. Res. Dev. 34, 1990); compared with the division for every significand of s
// at every tie of E4M3.  The error is inexact only where the quotient is far below
// E4M3's smallest value.  Zeros keep their sign.  An infinite scale (of an infinite
// amax) leaves 0 of finite x and NaN of the others, as a division does.
__device__ __forceinline__ float group_quotient(float x, float s, float inv) {
    const float q = x * inv, err = fmaf(q, fminf(s, 3.402823466e38f), -x);
    return fmaf(-err, inv, q);
}
// s rounded up to a power of two 2^(e-127): the biased exponent e.
__device__ __forceinline__ int ue8m0_exponent(float s) {
    const uint32_t bits = __float_as_uint(s);
    return (int)((bits >> 23) & 0xffu) + ((bits & 0x7fffffu) != 0u);
}
// The E8M0 byte of a 1x32 MX block: log2(X) + 127, X = 2^(floor(log2 amax) - 8)
// clamped at 2^-127.
__device__ __forceinline__ int mx_exponent(float amax) {
    const int be = (int)((__float_as_uint(amax) >> 23) & 0xffu);  // 0: zero or subnormal
    return be > 8 ? be - 8 : 0;
}
// 2^(127-e), the reciprocal of the scale 2^(e-127), for e in [0, 253].
__device__ __forceinline__ float exp_reciprocal(int e) {
    return __uint_as_float((uint32_t)(254 - e) << 23);
}
// 2^(e-127) as fp32 (e = 0: the subnormal 2^-127).
__device__ __forceinline__ float ue8m0_value(uint32_t e) {
    return e ? __uint_as_float(e << 23) : __uint_as_float(0x00400000u);
}

}  // namespace ep
