// Activations of the fused products and their slopes, in fp32 (device helpers).
//
//   relu       max(z, 0)                             slope 1 for z > 0, 0 for z <= 0
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
    if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;   // NaN: neither
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

// The matrix cores' operand d of dx = d W is fp16, while its values (dy zu act'(zg), times a row scale) span far
// more than fp16's range.  So d is stored in units of 2^(20 L), the level L chosen per token and
// block of rows from the block's largest finite magnitude m:  2^(20 L - 5) <= m < 2^(20 L + 15).  Nothing
// overflows, elements from 2^-9 m on keep all their bits, and one that becomes subnormal is off by 2^-25 units, at
// most 2^-20 m, far below the rounding of the large ones.  Levels this coarse are mostly the same along a row,
// which the products that join blocks make use of: in steps of 12 bits, gradients of about 2^3 put two levels into
// nearly every row (dz of gated 4096x11008 at 2048 tokens rewritten in 23 us).
// Bounds: m < 65504^3 1.13 < 2^49, and m = 0 takes the lowest level (2^-60 keeps every product of three fp16
// numbers that could move a sum).
constexpr int kLevelBits = 20, kLevelMin = -3, kLevelMax = 2;
constexpr int kLevelCols = 512;   // rows of W that share a level

__device__ __forceinline__ int grad_level(float m) {
    const int e = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 127;   // floor(log2 m); m >= 0
    const int l = (e + 5 + 8 * kLevelBits) / kLevelBits - 8;            // floor((e + 5) / 20): e >= -127
    return min(max(l, kLevelMin), kLevelMax);
}
// 2^(20 l), for levels and their differences.
__device__ __forceinline__ float level_unit(int l) { return __builtin_bit_cast(float, (uint32_t)(127 + kLevelBits * l) << 23); }
// The largest finite magnitude of a lane's 8 values (infinities and NaN stay what they are at any level).
// All lanes of a wave call it: where one of them has an infinity, the wave looks again.
__device__ __forceinline__ float largest_finite(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(v[q]));   // fmaxf passes over NaN
    if (__any(m == __builtin_inff())) {
        m = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(v[q]) < __builtin_inff() ? fabsf(v[q]) : 0.f);
    }
    return m;
}
// Eight fp16 values from units of one level to those of one `by` >= 0 levels higher, rounded once more where
// they become subnormal.  In factors of 2^-20, an fp16 number: finite values vanish from two levels on, infinities
// stay.
__device__ __forceinline__ u32x4 raise_level(u32x4 v, int by) {
    const f16 p = (f16)level_unit(by > 0 ? -1 : 0), q = (f16)level_unit(by > 1 ? -1 : 0);
    return as_u32x4(as_f16x8(v) * f16x8{p, p, p, p, p, p, p, p} * f16x8{q, q, q, q, q, q, q, q});
}

}  // namespace aqlm
