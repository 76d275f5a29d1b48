// MX4, microscaled 4-bit floating point, and how it reaches the matrix cores (device helpers).
//
// A row of n values is n / 32 blocks.  Value i of a block is q_i 2^(s - 127): q_i one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
// (one sign, two exponent, one mantissa bit), value 2i in the low half of byte i, and s the block's scale byte (255: NaN).
//
// Next to MX4 activations: the scaled matrix instruction D = C + sum_k (a_k 2^sa) (b_k 2^sb) over 128 values reads MX4 as it lies in
// memory: lane l of a wave supplies the 32 values (16 bytes) of block l / 16 and its scale byte, for row l % 16 of A or column
// l % 16 of B.  (Measured layout: 4-bit operands hold 32 consecutive values a lane.)
//
// Next to fp16 activations: q 2^(s - 127) is an fp16 number for 104 <= s <= 140 (0.5 2^-23 to 6 2^13), so a conversion of two
// values an instruction (as fast as an addition) gives the fp16 matrix instruction its operand without rounding, activations enter as they
// are, and only the sums are rounded, to fp32.  The four instructions that 128 values take cost what the scaled one would with
// activations split into four 4- or 6-bit floats, which lost what lies 2^-19 below a block's largest value.
// Blocks of other scales count as zero there and are added behind (odd blocks): q alone goes through the matrix instruction, block
// by block, and its sums are scaled in fp32.  Quantized fp16 blocks whose largest value is
// 2^-21 or more have none of those.  s = 0 (blocks of zeros) is left out: 2^-127 moves no result.
#pragma once
#include "aqlm_device.h"

namespace aqlm {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;          // values that share a scale
constexpr int kMxBlockBytes = 16;     // codes of a block
constexpr uint32_t kScaleNaN = 255;

// Activations of a product: fp16, or MX4 (the instruction's format number).
constexpr int kFmt16 = 0, kFmt4 = 4;

__device__ __forceinline__ i32x8 operand4(u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; }

// acc + A B for 16 rows and 16 columns of MX4; the scales are the low bytes of sa and sb.
__device__ __forceinline__ f32x4 mfma_mx(i32x8 a, i32x8 b, f32x4 acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFmt4, kFmt4, 0, (int)sa, 0, (int)sb);
}
// The same over 64 values for 32 rows and columns, scales in bytes SEL: lane l supplies the 32 values of block l / 32 for row (column) l % 32
// and holds D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32] for r = 0 .. 15.
template <int SEL>
__device__ __forceinline__ f32x16 mfma_mx32(i32x8 a, i32x8 b, f32x16 acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFmt4, kFmt4, SEL, (int)sa, SEL, (int)sb);
}
// fp16, over 16 values: lane l supplies 8 of them, 8 (l / 32) and on.
__device__ __forceinline__ f32x16 mfma32x32x16(f16x8 a, f16x8 b, f32x16 acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc, 0, 0, 0);
}

// Whether 4-bit floats times 2^(s - 127) are fp16 numbers; whether a block is an odd one; the factor of the others.
__device__ __forceinline__ bool plain_scale(uint32_t s) { return s - 104u <= 36u; }
__device__ __forceinline__ bool odd_scale(uint32_t s) { return s - 104u > 36u && s != 0u; }
__device__ __forceinline__ float scale_value(uint32_t s) { return __builtin_bit_cast(float, s << 23); }   // 0 < s < 255

// Eight codes times `scale`.
__device__ __forceinline__ f16x8 decode8(uint32_t codes, float scale) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A sum that is infinite because an activation was: NaN, as for MX4 activations, whose block is NaN then.  (Plain blocks alone
// stay below 2^52.)
__device__ __forceinline__ float no_infinity(float v) { return __builtin_fabsf(v) == __builtin_inff() ? __builtin_nanf("") : v; }

// The sum of an odd block's products, times its scale.
__device__ __forceinline__ float odd_sum(float d, uint32_t s) {
    return s == kScaleNaN ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(no_infinity(d), (int)s - 127);
}

// Keeps a finished accumulator in registers before control flow diverges: the compiler may otherwise move the last
// matrix instruction into the branch that uses its result, and the moves that feed it then skip the lanes that do not
// take the branch.
template <class V>
__device__ __forceinline__ void pin(V& v) { asm volatile("" : "+v"(v)); }

__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }   // -126 <= e <= 127

// floor(log2 |h|) of fp16 bits 0 < h < 0x7c00.
__device__ __forceinline__ int exponent16(uint32_t h) {
    return h >= 0x400u ? (int)(h >> 10) - 15 : 31 - __builtin_clz(h) - 24;
}

// Bytes d, d + 1, ... of r (0 <= d <= 16), then zeros.
__device__ __forceinline__ u32x4 move_bytes(u32x4 r, int d) {
    if (d & 1) r = u32x4{(uint32_t)__builtin_amdgcn_alignbyte(r[1], r[0], 1), (uint32_t)__builtin_amdgcn_alignbyte(r[2], r[1], 1),
                         (uint32_t)__builtin_amdgcn_alignbyte(r[3], r[2], 1), r[3] >> 8};
    if (d & 2) r = u32x4{(uint32_t)__builtin_amdgcn_alignbyte(r[1], r[0], 2), (uint32_t)__builtin_amdgcn_alignbyte(r[2], r[1], 2),
                         (uint32_t)__builtin_amdgcn_alignbyte(r[3], r[2], 2), r[3] >> 16};
    if (d & 4) r = u32x4{r[1], r[2], r[3], 0u};
    if (d & 8) r = u32x4{r[2], r[3], 0u, 0u};
    if (d & 16) r = u32x4{0u, 0u, 0u, 0u};
    return r;
}

}  // namespace aqlm
