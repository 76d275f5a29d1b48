// Conversions between fp16 and MX4 (mx4.h).
//
// quantize: the scale of a block is 2^(floor(log2 max |v|) - 2), so that the largest value lies in [4, 8) of the 4-bit
// floats' range; values are rounded to nearest even and at most 6.  A block of zeros takes scale byte 0, one with an
// infinity or a NaN scale byte 255 (NaN) and codes 0.  The scale is taken from the exponent bits, and the division by a power of
// two and the rounding are the conversion instruction's (exact rounding checked on every fp16 value).
//
// Both directions move 2 + 17/32 bytes a value and are bound by memory: a lane takes 8 values (16 bytes of fp16), four
// neighbouring lanes a block, so every access of a wave is contiguous.  28672 x 8192: 103 and 108 us, 5.5 TB/s.
#include <algorithm>

#include "mx4.h"
#include "mx4_launch.h"

namespace aqlm {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(const f16* __restrict__ w, uint32_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales, int64_t lanes) {
    for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < lanes; at += (int64_t)gridDim.x * kThreads) {
        const u32x4 v = load_nt16(w + at * 8);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = v[i] & 0x7fff7fffu;
            m = max(m, max(a & 0xffffu, a >> 16));
        }
        // a block's four lanes are neighbours (lanes is a multiple of 4, so all four are here)
        m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
        const bool bad = m >= 0x7c00u, none = m == 0;
        const int e = bad || none ? 0 : exponent16(m) - 2;
        const float unit = pow2(e);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)v[0]), unit, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)v[1]), unit, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)v[2]), unit, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)v[3]), unit, 3);
        codes[at] = bad ? 0u : c;
        if ((at & 3) == 0) scales[at >> 2] = (uint8_t)(bad ? kScaleNaN : none ? 0 : (uint32_t)(127 + e));
    }
}

// fp16 nearest to q 2^(s - 127): the product in fp32 is exact down to 2^-127 / 2, far below fp16.
__global__ __launch_bounds__(kThreads) void mx4_decode_kernel(const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, f16* __restrict__ w,
                                                              int64_t lanes) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < lanes; at += (int64_t)gridDim.x * kThreads) {
        const uint32_t c = __builtin_nontemporal_load(codes + at);
        const int s = scales[at >> 2];
        f16x8 o;
        f32x2 p[4];
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __builtin_amdgcn_ldexpf(p[i / 2][i % 2], s - 127);
            o[i] = s == (int)kScaleNaN ? (f16)__builtin_nanf("") : (f16)f;
        }
        __builtin_nontemporal_store(as_u32x4(o), reinterpret_cast<u32x4*>(w + at * 8));
    }
}

dim3 flat_grid(int64_t threads, int per_cu) {
    return dim3((unsigned)std::min<int64_t>((threads + kThreads - 1) / kThreads, (int64_t)device_cu_count() * per_cu));
}

}  // namespace

hipError_t launch_mx4_quantize(const void* w, void* codes, void* scales, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL(mx4_quantize_kernel, flat_grid(blocks * 4, 32), dim3(kThreads), 0, stream, static_cast<const f16*>(w),
                       static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales), blocks * 4);
    return hipGetLastError();
}

hipError_t launch_mx4_decode(const void* codes, const void* scales, void* w, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL(mx4_decode_kernel, flat_grid(blocks * 4, 32), dim3(kThreads), 0, stream,
                       static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales), static_cast<f16*>(w),
                       blocks * 4);
    return hipGetLastError();
}

}  // namespace aqlm
