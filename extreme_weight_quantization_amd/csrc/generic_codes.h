// Codes and codewords of any scheme: M codebooks (1..8) of 2^B codewords (B = 1..16)
// of g entries, codes in whole bytes or bit-packed (device helpers).
#pragma once
#include "aqlm_device.h"

namespace aqlm {

#pragma clang fp contract(off)

// The codeword index of code i: the low B bits of its CB-byte stored pattern, or,
// for bit-packed codes (CB = 0), the B bits at bit i * B of the little-endian
// 32-bit word stream (least significant bit first; a code may straddle two words,
// and the second word is read only then).
template <int CB>
__device__ __forceinline__ uint32_t code_at(const uint8_t* __restrict__ codes, size_t i, uint32_t mask, int B) {
    if constexpr (CB == 1) {
        return (uint32_t)codes[i] & mask;
    } else if constexpr (CB == 2) {
        return (uint32_t)reinterpret_cast<const uint16_t*>(codes)[i] & mask;
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(codes);
        const uint64_t bit = (uint64_t)i * (uint64_t)B;
        const size_t wi = (size_t)(bit >> 5);
        const int off = (int)(bit & 31);
        uint32_t v = w[wi] >> off;
        if (off + B > 32) v |= w[wi + 1] << (32 - off);
        return v & mask;
    }
}

// N consecutive fp16 values starting at p (p aligned to 2N bytes, N <= 8).
template <int N>
__device__ __forceinline__ void load_f16(const f16* p, float (&v)[N]) {
    if constexpr (N == 8) {
        const f16x8 c = *reinterpret_cast<const f16x8*>(p);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = (float)c[t];
    } else if constexpr (N == 4) {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        const f16x4 c = *reinterpret_cast<const f16x4*>(p);
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = (float)c[t];
    } else if constexpr (N == 2) {
        const f16x2 c = *reinterpret_cast<const f16x2*>(p);
        v[0] = (float)c[0];
        v[1] = (float)c[1];
    } else {
        v[0] = (float)p[0];
    }
}

// Entries t0 .. t0+N-1 of the sum over m of the codewords selected by the M codes
// starting at codes[c0]: codebook 0's entry, then + codebook m, m ascending,
// each sum rounded to fp32.  cb points at codebook 0 ([M][2^B][G]).
template <int G, int N, int CB>
__device__ __forceinline__ void sum_codewords(const uint8_t* __restrict__ codes, size_t c0, const f16* cb,
                                              int M, int B, uint32_t mask, int t0, float (&v)[N]) {
    load_f16<N>(cb + (size_t)code_at<CB>(codes, c0, mask, B) * G + t0, v);
    for (int m = 1; m < M; ++m) {
        float c[N];
        load_f16<N>(cb + (((size_t)m << B) + code_at<CB>(codes, c0 + m, mask, B)) * G + t0, c);
#pragma unroll
        for (int t = 0; t < N; ++t) v[t] = __fadd_rn(v[t], c[t]);
    }
}

// The whole group (G entries) as fp32, in pieces of at most 8 entries.
template <int G, int CB>
__device__ __forceinline__ void group_weights(const uint8_t* __restrict__ codes, size_t c0, const f16* cb,
                                              int M, int B, uint32_t mask, float (&v)[G]) {
    constexpr int N = G < 8 ? G : 8;
#pragma unroll
    for (int p = 0; p < G / N; ++p) {
        float part[N];
        sum_codewords<G, N, CB>(codes, c0, cb, M, B, mask, p * N, part);
#pragma unroll
        for (int t = 0; t < N; ++t) v[p * N + t] = part[t];
    }
}

// Copies n_elems fp16 codebook entries into LDS: 16 bytes at a time when the
// size allows, else one entry at a time.
__device__ __forceinline__ void stage_codebook(f16* dst, const f16* __restrict__ src, size_t n_elems) {
    if ((n_elems & 7) == 0) {
        u32x4* d = reinterpret_cast<u32x4*>(dst);
        for (size_t i = threadIdx.x; i < n_elems / 8; i += blockDim.x) d[i] = load16(src + i * 8);
    } else {
        for (size_t i = threadIdx.x; i < n_elems; i += blockDim.x) dst[i] = src[i];
    }
    __syncthreads();
}

}  // namespace aqlm
