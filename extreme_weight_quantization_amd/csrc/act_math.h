// Activations of the fused products and their slopes, in fp32 (device helpers).
//
//   relu       max(z, 0)                             slope 1 for z > 0, else 0
//   silu       z p,           p = 1 / (1 + e^-z)     slope p (1 + z (1 - p))
//   gelu       z erfc(-z / sqrt 2) / 2               slope erfc(-z / sqrt 2) / 2 + z e^(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z (1 + tanh v) / 2 = z p(2v),         slope p + z p (1 - p) 2 v',
//              v = sqrt(2 / pi) (z + 0.044715 z^3)   v' = sqrt(2 / pi) (1 + 0.134145 z^2)
//
// gelu is written with erfc and gelu_tanh with the logistic function of 2v, so that neither
// takes a difference of two numbers near one where z is far below zero.  NaN stays NaN.
#pragma once
#include "aqlm_device.h"

namespace aqlm {

// Values of aqlm_act (include/aqlm.h).
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// __expf is exact to about |z| 2^-24 relative (the rounding of z log2 e): far inside the one
// fp16 rounding that every result here takes next.
__device__ __forceinline__ float logistic(float z) { return 1.f / (1.f + __expf(-z)); }

constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;
    if constexpr (ACT == kActSilu) return z / (1.f + __expf(-z));
    if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(z * -0.70710678118654752f);
    if constexpr (ACT == kActGeluTanh) return z / (1.f + __expf(-kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z)));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.f ? 0.f : 1.f;
    if constexpr (ACT == kActSilu) {
        const float p = logistic(z);
        return p * (1.f + z * (1.f - p));
    }
    if constexpr (ACT == kActGelu)
        return 0.5f * erfcf(z * -0.70710678118654752f) + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    if constexpr (ACT == kActGeluTanh) {
        const float p = logistic(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
        return p + z * p * (1.f - p) * kTwoSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
    }
    return 1.f;
}

// v[i] = act(v[i]).  One branch for all N: with a branch per value the five bodies, unrolled
// through an epilogue, outgrew the instruction cache (19 us for the gradients of 8 tokens).
template <int ACT, int N>
__device__ __forceinline__ void act_values_of(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value<ACT>(v[i]);
}

template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        case kActRelu: act_values_of<kActRelu>(v); break;
        case kActSilu: act_values_of<kActSilu>(v); break;
        case kActGelu: act_values_of<kActGelu>(v); break;
        case kActGeluTanh: act_values_of<kActGeluTanh>(v); break;
        default: break;
    }
}

// v[i] = slope of act at v[i], one branch for all N.
template <int ACT, int N>
__device__ __forceinline__ void act_slopes_of(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_slope<ACT>(v[i]);
}

template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&v)[N]) {
    switch (act) {
        case kActRelu: act_slopes_of<kActRelu>(v); break;
        case kActSilu: act_slopes_of<kActSilu>(v); break;
        case kActGelu: act_slopes_of<kActGelu>(v); break;
        case kActGeluTanh: act_slopes_of<kActGeluTanh>(v); break;
        default: act_slopes_of<kActNone>(v); break;
    }
}

// A row scale s = m 2^e as an fp16 power of two, which goes into the fp16 weights exactly
// (but for subnormals), and the rest, which goes into the other factor, so that only
// one of the two is rounded: 1 <= |m| < 2 for normal s, m
// below 1 for subnormal s (e = -14), m = s for zero, infinity and NaN (e = 0).
__device__ __forceinline__ f16 scale_power(f16 s) {
    const uint16_t b = __builtin_bit_cast(uint16_t, s), x = b & 0x7c00u;
    const uint16_t p = (x == 0x7c00u || (b & 0x7fffu) == 0) ? 0x3c00u : x == 0 ? 0x0400u : x;
    return __builtin_bit_cast(f16, p);
}
// (The quotient by a power of two is the product with its reciprocal, exactly.)
__device__ __forceinline__ float scale_rest(f16 s) {
    const uint32_t e = (uint32_t)__builtin_bit_cast(uint16_t, scale_power(s)) >> 10;   // 1 .. 30
    return (float)s * __builtin_bit_cast(float, (142u - e) << 23);
}

}  // namespace aqlm
