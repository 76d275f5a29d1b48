// MX4, microscaled 4-bit floating point, and how fp16 activations reach the matrix cores next to it (device helpers).
//
// A row of n values is n / 32 blocks.  Value i of a block is q_i 2^(s - 127): q_i one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
// (one sign, two exponent, one mantissa bit), value 2i in the low half of byte i, and s the block's scale byte (255: NaN).
//
// The scaled matrix instruction D = C + sum_k (a_k 2^sa) (b_k 2^sb) over 128 values reads MX4 as it lies in memory: lane
// l of a wave supplies the 32 values (16 bytes) of block l / 16 and its scale byte, for row l % 16 of A or column l % 16
// of B.  So weights are never decoded by vector instructions.  (Measured layout: 4- and 6-bit operands hold 32
// consecutive values a lane; 8-bit ones would hold 16 and 16, 64 apart.)
//
// fp16 activations become such an operand without losing what fp16 holds: a block x of 32 values, 2^e <= max |x| <
// 2^(e + 1), is written as a sum of four 6-bit floats a value (two exponent, three mantissa bits: steps of 1/8 below 2,
// 1/4 to 4),
//     x = sum_p c_p 2^(e - 1 - 5 p) + r,   c_p = nearest((x - sum_{j < p} ...) / 2^(e - 1 - 5 p)),   p = 0 .. 3.
// |x| / 2^(e - 1) < 4 leaves at most half of a step of 1/4, 2^-3, which is again at most 4 in units 2^5 finer, and so on:
// |r| <= 2^-3 2^(e - 16) <= 2^-18 max |x| / 2.  Values down to 2^-8 of the block's largest keep all their 11 bits, smaller ones
// are off by at most 2^-19 of it, far below the rounding of an fp16 result.  Why four products of 6 bits: they run at the
// rate of 4-bit ones (8.3 PFLOP/s measured, against 4.4 for 8-bit floats, of which it would take three), and their
// products with MX4 weights span 10 bits, which the instruction adds up exactly within a block; 8-bit floats span more than the
// 13 bits that it keeps below a block's largest product.
#pragma once
#include "aqlm_device.h"

namespace aqlm {

typedef _Float16 f16x32 __attribute__((ext_vector_type(32)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;          // values that share a scale
constexpr int kMxBlockBytes = 16;     // codes of a block
constexpr int kMxStep = 128;          // values a scaled matrix instruction multiplies per row
constexpr int kPieces = 4;            // 6-bit floats a value of fp16 activations
constexpr int kPieceDwords = 6;       // 32 of them
constexpr int kSplitDwords = kPieces * kPieceDwords;   // a block in four pieces: 96 bytes
constexpr uint32_t kScaleNaN = 255;

// Split activations lie in records, one for every tile of w tokens (w = 32 in a workspace) and block of 32 inputs: for each
// piece the first 16 bytes of the tokens' 24, then for each piece the other 8, then the tokens' scale words.  So an
// operand is one 16-byte and one 8-byte access, and neighbouring tokens are neighbours in memory.
constexpr int kSplitTokens = 32;
constexpr int kSplitTokenBytes = kPieces * kPieceDwords * 4 + 4;          // 100
constexpr int kSplitRecord = kSplitTokens * kSplitTokenBytes;             // 3200
struct SplitRows {
    char* base;
    int w, nb;   // tokens of a tile, blocks of a row
    // 16-byte aligned whatever w is: reads of 16 bytes from LDS at 100-byte steps took 6 us of a single token's 12.
    __host__ __device__ static constexpr int record_bytes(int w) { return (w * kSplitTokenBytes + 15) / 16 * 16; }
    __device__ __forceinline__ char* record(int token, int block) const {
        return base + ((size_t)(token / w) * nb + block) * (size_t)record_bytes(w);
    }
    __device__ __forceinline__ u32x4* first(char* rec, int token, int p) const {
        return reinterpret_cast<u32x4*>(rec + 16 * (p * w + token % w));
    }
    __device__ __forceinline__ u32x2* rest(char* rec, int token, int p) const {
        return reinterpret_cast<u32x2*>(rec + 64 * w + 8 * (p * w + token % w));
    }
    __device__ __forceinline__ uint32_t* scales(char* rec, int token) const {
        return reinterpret_cast<uint32_t*>(rec + 96 * w) + token % w;
    }
};


__device__ __forceinline__ i32x8 operand4(u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; }
__device__ __forceinline__ i32x8 operand6(u32x6 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)v[4], (int)v[5], 0, 0};
}

// acc + A B for MX4 A (16 rows) and B (16 columns) of 4- or 6-bit floats; the scale of B is byte SEL of sb.
constexpr int kFmt6 = 2, kFmt4 = 4;   // the instruction's format numbers (6 bits: two exponent, three mantissa)
// The same over 64 values for 32 rows and columns, A in MX4: lane l supplies the 32 values of block l / 32 for row (column) l % 32
// and holds D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32] for r = 0 .. 15.
template <int FMT_B, int SEL_A, int SEL_B>
__device__ __forceinline__ f32x16 mfma_mx32(i32x8 a, i32x8 b, f32x16 acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, kFmt4, FMT_B, SEL_A, (int)sa, SEL_B, (int)sb);
}
template <int FMT_B, int SEL>
__device__ __forceinline__ f32x4 mfma_mx(i32x8 a, i32x8 b, f32x4 acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFmt4, FMT_B, 0, (int)sa, SEL, (int)sb);
}

// Keeps a finished accumulator in registers before control flow diverges: the compiler may otherwise move the last
// matrix instruction into the branch that uses its result, and the moves that feed it then skip the lanes that do not
// take the branch.
template <class V>
__device__ __forceinline__ void pin(V& v) { asm volatile("" : "+v"(v)); }

__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }   // -126 <= e <= 127

// Largest magnitude of 32 fp16 values as fp16 bits (sign cleared); infinities and NaN compare above all others.
__device__ __forceinline__ uint32_t top_bits(const f16x32& v) {
    uint32_t m = 0;
    const auto* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t a = w[i] & 0x7fff7fffu;
        m = max(m, max(a & 0xffffu, a >> 16));
    }
    return m;
}

// floor(log2 |h|) of fp16 bits 0 < h < 0x7c00.
__device__ __forceinline__ int exponent16(uint32_t h) {
    return h >= 0x400u ? (int)(h >> 10) - 15 : 31 - __builtin_clz(h) - 24;
}

__device__ __forceinline__ f16x32 load_block16(const f16* __restrict__ x) {   // 16-byte aligned
    f16x32 v;
    auto* w = reinterpret_cast<u32x4*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = load16(x + 8 * i);
    return v;
}

// a - b, both fp16 and the result exact, two at a time (as one expression the compiler takes the vectors apart).
__device__ __forceinline__ f16x32 subtract(const f16x32& a, const f16x32& b) {
    f16x32 r;
    const auto *pa = reinterpret_cast<const f16x2*>(&a), *pb = reinterpret_cast<const f16x2*>(&b);
    auto* pr = reinterpret_cast<f16x2*>(&r);
#pragma unroll
    for (int i = 0; i < 16; ++i) pr[i] = pa[i] - pb[i];
    return r;
}

// Four pieces of a block and, in byte p of `scales`, the scale of piece p.  A block of zeros has pieces 0; one with an
// infinity or NaN scales of NaN, which every product with it is.
__device__ __forceinline__ void split_block(f16x32 v, uint32_t (&out)[kSplitDwords], uint32_t& scales) {
    const uint32_t top = top_bits(v);
    const bool none = top == 0, bad = top >= 0x7c00u;
    int e = none || bad ? 0 : exponent16(top);
    // above 2^15 a piece could round up to 2^16, which fp16 lacks: such a block is halved (exact but for values 2^-38 of
    // its largest)
    const f16 half = (f16)(e >= 15 ? 0.5f : 1.f);
    const int down = e >= 15;
    e -= down;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = v[i] * half;
    scales = 0;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const float unit = pow2(e - 1 - 5 * p);
        const u32x6 c = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(v, unit);
        if (p + 1 < kPieces) v = subtract(v, __builtin_amdgcn_cvt_scalef32_pk32_f16_fp6(c, unit));
#pragma unroll
        for (int i = 0; i < kPieceDwords; ++i) out[p * kPieceDwords + i] = none || bad ? 0u : c[i];
        scales |= (bad ? kScaleNaN : (uint32_t)(127 + e + down - 1 - 5 * p)) << (8 * p);
    }
}

// The same for the fp32 values 2i (even[i]) and 2i + 1 (odd[i]) of a block, for results that go on into another product.  Below 2^-110 a block counts as zero, from 2^126 on
// as infinite.
__device__ __forceinline__ void split_block32(f32x16 even, f32x16 odd, uint32_t (&out)[kSplitDwords], uint32_t& scales) {
    uint32_t top = 0;   // magnitudes order as their bits do
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = even[i], b = odd[i];
        top = max(top, max(__builtin_bit_cast(uint32_t, a) & 0x7fffffffu, __builtin_bit_cast(uint32_t, b) & 0x7fffffffu));
    }
    int e = (int)(top >> 23) - 127;
    const bool none = e < -110, bad = e >= 126;
    if (none || bad) e = 0;
    scales = 0;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const float unit = pow2(e - 1 - 5 * p);
        const u32x6 c = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(even, odd, unit);
        if (p + 1 < kPieces) {
            const auto back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(c, unit);
#pragma unroll
            for (int i = 0; i < 16; ++i) {   // exact
                even[i] -= back[2 * i];
                odd[i] -= back[2 * i + 1];
            }
        }
#pragma unroll
        for (int i = 0; i < kPieceDwords; ++i) out[p * kPieceDwords + i] = none || bad ? 0u : c[i];
        scales |= (bad ? kScaleNaN : (uint32_t)(127 + e - 1 - 5 * p)) << (8 * p);
    }
}

__device__ __forceinline__ void store_split(const SplitRows& to, int token, int block, const uint32_t (&o)[kSplitDwords],
                                            uint32_t scales) {
    char* rec = to.record(token, block);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const uint32_t* q = o + p * kPieceDwords;
        *to.first(rec, token, p) = u32x4{q[0], q[1], q[2], q[3]};
        *to.rest(rec, token, p) = u32x2{q[4], q[5]};
    }
    *to.scales(rec, token) = scales;
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
