// The hidden vector of a mixture-of-experts layer between its products (device helpers).
//
// A value h = act(zg) zu is kept as two fp16 numbers, rows 2 pair and 2 pair + 1 of an array [..][rows]:
//     h = kPairUnit (hi + lo / kPairFine),   hi = nearest(h / kPairUnit),   lo = nearest(kPairFine (h / kPairUnit - hi)).
// One rounding to fp16 would add its error to that of the layer's own result; the second number costs a column that the matrix cores
// multiply anyway.  hi is off by 2^-11 of itself or 2^-25, lo again: together 2^-22 |h| or 2^-36 kPairUnit = 2^-28.  The unit of 2^8
// moves the range up, to |h| = 2^8 * 65504; kPairFine keeps lo out of fp16's subnormals and is the most that |lo| <= 2^-11 2^16 allows.
#pragma once
#include "aqlm_device.h"

namespace aqlm {

constexpr float kPairUnit = 256.f, kPairFine = 2048.f;

__device__ __forceinline__ void store_pair(float h, f16* y, int pair, int row, int rows) {
    h *= 1.f / kPairUnit;
    const f16 hi = (f16)h;
    y[(size_t)(2 * pair) * rows + row] = hi;
    y[(size_t)(2 * pair + 1) * rows + row] = fabsf((float)hi) < __builtin_inff() ? (f16)((h - (float)hi) * kPairFine) : (f16)0.f;
}

}  // namespace aqlm
