// Decoded weights as the work matrices of the dense products: row by row with padded
// rows, and transposed.
//
// "The AQLM Quantization Algorithm, Explained", Figure 2 of the MCQ section: a group's
// weights are the sum of one codeword per codebook, times the row's scale.  A thread
// builds pieces of 8 weights (fp32 sum, codebook 0 first; one rounding to fp16).
//
//   decode_rows        w[row][0 .. kp), inputs past `in` zero: the dense product steps
//                      over 64 inputs at a time, so a row is padded to kp % 64 == 0.
//   decode_transposed  wt[k][row], rows past `out` zero: dx = dz W sums over the rows of
//                      W, and the dense product wants the summed index innermost.  A
//                      thread decodes the pieces of 8 consecutive rows at one place,
//                      transposes the 8 x 8 block in registers, and stores 8 pieces of 8
//                      rows; 8 consecutive lanes fill a 128-byte line.
//
// Both are bound by the write of 2 bytes per weight.
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"
#include "generic_codes.h"

namespace aqlm {

namespace {

struct DecodeArgs {
    const uint8_t* codes[2];
    const f16* codebooks[2];
    const f16* scales[2];
    f16* w[2];
};

// The fp32 weights of inputs 8p .. 8p+7 of a row before the scale, zero past `in`.
// kScheme2x8 reads the codebooks' LDS copy (slot 256 m + k), 1x16 gathers its codeword, any
// other scheme (g = G, code storage CB as in code_at) reads the codebooks through L2.
template <int SCHEME, int G, int CB>
__device__ __forceinline__ void piece_weights(const uint8_t* __restrict__ codes, const f16* __restrict__ codebooks,
                                              const u32x4* cb_lds, uint32_t row, uint32_t p, int in, int M, int B,
                                              float (&v)[8]) {
    if constexpr (SCHEME == kScheme2x8 || SCHEME == kScheme1x16) {
        const uint32_t n_grp = (uint32_t)in / kGroup;
        if (p >= n_grp) {
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = 0.f;
            return;
        }
        const uint32_t c = reinterpret_cast<const uint16_t*>(codes)[(size_t)row * n_grp + p];
        if constexpr (SCHEME == kScheme2x8) {
            const f16x8 a = as_f16x8(cb_lds[c & 0xff]), b = as_f16x8(cb_lds[kCodewords2x8 + (c >> 8)]);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = __fadd_rn((float)a[t], (float)b[t]);
        } else {
            const f16x8 a = as_f16x8(load16(codebooks + (size_t)c * kGroup));
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = (float)a[t];
        }
    } else {
        const uint32_t mask = (1u << B) - 1u;
        const int n_grp = in / G, k = (int)p * 8;
        const size_t rbase = (size_t)row * n_grp;
        if constexpr (G >= 8) {
            if (k < in) {
                sum_codewords<G, 8, CB>(codes, (rbase + k / G) * M, codebooks, M, B, mask, k % G, v);
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = 0.f;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8 / G; ++q) {
                float part[G];
#pragma unroll
                for (int t = 0; t < G; ++t) part[t] = 0.f;
                const int kq = k + q * G;
                if (kq < in) sum_codewords<G, G, CB>(codes, (rbase + kq / G) * M, codebooks, M, B, mask, 0, part);
#pragma unroll
                for (int t = 0; t < G; ++t) v[q * G + t] = part[t];
            }
        }
    }
}

// The row's factor under the weight-scale mode.
template <WeightScale WS>
__device__ __forceinline__ float row_factor(const f16* __restrict__ scales, uint32_t row) {
    if constexpr (WS == WeightScale::kNone) return 1.f;
    const float s = (float)scales[row];
    if constexpr (WS == WeightScale::kFull) return s;
    int e;
    scale_mantissa(s, &e);
    return ldexpf(1.f, e);
}

// Layer 2x8: its codebooks into LDS (512 slots of 16 bytes).
template <int SCHEME>
__device__ __forceinline__ void stage_2x8(u32x4* cb_lds, const f16* __restrict__ codebooks) {
    if constexpr (SCHEME == kScheme2x8) {
        for (int i = threadIdx.x; i < 2 * kCodewords2x8; i += blockDim.x) cb_lds[i] = load16(codebooks + (size_t)i * kGroup);
        __syncthreads();
    }
}

template <int SCHEME, int G, int CB, WeightScale WS>
__global__ __launch_bounds__(256) void decode_rows_kernel(DecodeArgs a, uint32_t n_pieces, uint32_t per_row, int in,
                                                          int M, int B) {
    __shared__ u32x4 cb_lds[SCHEME == kScheme2x8 ? 2 * kCodewords2x8 : 1];
    const int l = blockIdx.y;
    const uint8_t* codes = l ? a.codes[1] : a.codes[0];
    const f16* codebooks = l ? a.codebooks[1] : a.codebooks[0];
    const f16* scales = l ? a.scales[1] : a.scales[0];
    f16* w = l ? a.w[1] : a.w[0];
    stage_2x8<SCHEME>(cb_lds, codebooks);
    // 64-bit loop index: n_pieces may come within a stride of 2^32
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i64 = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i64 < n_pieces; i64 += stride) {
        const uint32_t i = (uint32_t)i64, row = i / per_row, p = i - row * per_row;
        float v[8];
        piece_weights<SCHEME, G, CB>(codes, codebooks, cb_lds, row, p, in, M, B, v);
        const float s = row_factor<WS>(scales, row);
        f16x8 o;
#pragma unroll
        for (int t = 0; t < 8; ++t) o[t] = (f16)__fmul_rn(v[t], s);
        // non-temporal: the write stream must not evict the codebook or the codes from L2
        __builtin_nontemporal_store(as_u32x4(o), reinterpret_cast<u32x4*>(w + (size_t)i * 8));
    }
}

// Tile of 64 rows x 32 pieces: thread (piece tid / 8, rows 8 (tid % 8) ..).
template <int SCHEME, int G, int CB, WeightScale WS>
__global__ __launch_bounds__(256) void decode_transposed_kernel(DecodeArgs a, int out, int in, int op, int ldt,
                                                                int n_row_tiles, int M, int B) {
    __shared__ u32x4 cb_lds[SCHEME == kScheme2x8 ? 2 * kCodewords2x8 : 1];
    const int l = blockIdx.y;
    const uint8_t* codes = l ? a.codes[1] : a.codes[0];
    const f16* codebooks = l ? a.codebooks[1] : a.codebooks[0];
    const f16* scales = l ? a.scales[1] : a.scales[0];
    stage_2x8<SCHEME>(cb_lds, codebooks);
    const int rt = (int)(blockIdx.x % n_row_tiles), pt = (int)(blockIdx.x / n_row_tiles);
    const int row0 = rt * 64 + 8 * (threadIdx.x & 7), p = pt * 32 + (threadIdx.x >> 3);
    const int k0 = 8 * p;
    if (k0 >= in) return;
    f16 o[8][8];   // [row][input]
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int row = min(row0 + r, out - 1);
        float v[8];
        piece_weights<SCHEME, G, CB>(codes, codebooks, cb_lds, row, p, in, M, B, v);
        const float s = row_factor<WS>(scales, row);
#pragma unroll
        for (int t = 0; t < 8; ++t) o[r][t] = row0 + r < out ? (f16)__fmul_rn(v[t], s) : (f16)0.f;
    }
    f16* w = a.w[0] + (size_t)l * op + row0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (k0 + t < in) {
            f16x8 c;
#pragma unroll
            for (int r = 0; r < 8; ++r) c[r] = o[r][t];
            *reinterpret_cast<u32x4*>(w + (size_t)(k0 + t) * ldt) = as_u32x4(c);
        }
    }
}

__global__ __launch_bounds__(256) void pad_rows_kernel(const f16* __restrict__ x, f16* __restrict__ xp,
                                                       uint64_t n_pieces, uint32_t per_row, int in) {
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_pieces; i += stride) {
        const uint64_t t = i / per_row;
        const int k = (int)(i - t * per_row) * 8;
        const f16* src = x + t * (uint64_t)in + k;
        f16x8 o;
        if (in % 8 == 0) {
            o = k < in ? *reinterpret_cast<const f16x8*>(src) : f16x8{};
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = k + q < in ? src[q] : (f16)0.f;
        }
        *reinterpret_cast<u32x4*>(xp + i * 8) = as_u32x4(o);
    }
}

DecodeArgs decode_args(const ActLayers& L) {
    DecodeArgs a = {};
    for (int l = 0; l < L.n; ++l) {
        a.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        a.codebooks[l] = static_cast<const f16*>(L.codebooks[l]);
        a.scales[l] = static_cast<const f16*>(L.scales[l]);
    }
    return a;
}

// One launch of decode_rows (T = false) or decode_transposed (T = true).
template <bool T, int SCHEME, int G, int CB, WeightScale WS>
hipError_t launch_ws(const DecodeArgs& a, int n, int64_t out, int64_t in, int64_t ld, int64_t op, int M, int B,
                     hipStream_t stream) {
    if constexpr (T) {
        const int64_t n_rt = op / 64, n_pt = (in + 255) / 256;
        if (n_rt * n_pt > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL((decode_transposed_kernel<SCHEME, G, CB, WS>), dim3((unsigned)(n_rt * n_pt), n), dim3(256), 0,
                           stream, a, (int)out, (int)in, (int)op, (int)ld, (int)n_rt, M, B);
    } else {
        const uint64_t per_row = (uint64_t)ld / 8, n_pieces = (uint64_t)out * per_row;
        if (n_pieces > UINT32_MAX) return hipErrorInvalidValue;
        uint64_t blocks = (n_pieces + 255) / 256;
        const uint64_t cap = (uint64_t)device_cu_count() * 16;
        if (blocks > cap) blocks = cap;
        hipLaunchKernelGGL((decode_rows_kernel<SCHEME, G, CB, WS>), dim3((unsigned)blocks, n), dim3(256), 0, stream, a,
                           (uint32_t)n_pieces, (uint32_t)per_row, (int)in, M, B);
    }
    return hipGetLastError();
}

template <bool T, int SCHEME, int G, int CB>
hipError_t launch_scheme(WeightScale ws, const DecodeArgs& a, int n, int64_t out, int64_t in, int64_t ld, int64_t op,
                         int M, int B, hipStream_t stream) {
    if (ws == WeightScale::kFull)
        return launch_ws<T, SCHEME, G, CB, WeightScale::kFull>(a, n, out, in, ld, op, M, B, stream);
    if constexpr (T) return launch_ws<T, SCHEME, G, CB, WeightScale::kPow2>(a, n, out, in, ld, op, M, B, stream);
    else return launch_ws<T, SCHEME, G, CB, WeightScale::kNone>(a, n, out, in, ld, op, M, B, stream);
}

template <bool T>
hipError_t launch_any(const GenericScheme& sc, WeightScale ws, const DecodeArgs& a, int n, int64_t out, int64_t in,
                      int64_t ld, int64_t op, hipStream_t stream) {
    const int M = sc.M, B = sc.B;
    if (M == 2 && B == 8 && sc.g == 8)
        return launch_scheme<T, kScheme2x8, 8, 1>(ws, a, n, out, in, ld, op, M, B, stream);
    if (M == 1 && B == 16 && sc.g == 8)
        return launch_scheme<T, kScheme1x16, 8, 2>(ws, a, n, out, in, ld, op, M, B, stream);
#define AQLM_ROWS(G)                                                                                              \
    case G:                                                                                                       \
        return B <= 8 ? launch_scheme<T, kSchemeGeneric, G, 1>(ws, a, n, out, in, ld, op, M, B, stream)            \
                      : launch_scheme<T, kSchemeGeneric, G, 2>(ws, a, n, out, in, ld, op, M, B, stream);
    switch (sc.g) {
        AQLM_ROWS(1)
        AQLM_ROWS(2)
        AQLM_ROWS(4)
        AQLM_ROWS(8)
        AQLM_ROWS(16)
        AQLM_ROWS(32)
        default: return hipErrorInvalidValue;
    }
#undef AQLM_ROWS
}

}  // namespace

hipError_t launch_decode_rows(const GenericScheme& sc, const ActLayers& L, WeightScale ws, void* const* w,
                              int64_t out, int64_t in, int64_t kp, hipStream_t stream) {
    DecodeArgs a = decode_args(L);
    for (int l = 0; l < L.n; ++l) a.w[l] = static_cast<f16*>(w[l]);
    return launch_any<false>(sc, ws, a, L.n, out, in, kp, 0, stream);
}

hipError_t launch_decode_transposed(const GenericScheme& sc, const ActLayers& L, WeightScale ws, void* wt,
                                    int64_t out, int64_t in, int64_t op, hipStream_t stream) {
    DecodeArgs a = decode_args(L);
    a.w[0] = static_cast<f16*>(wt);
    return launch_any<true>(sc, ws, a, L.n, out, in, L.n * op, op, stream);
}

hipError_t launch_pad_rows(const void* x, void* xp, int64_t batch, int64_t in, int64_t kp, hipStream_t stream) {
    const uint64_t per_row = (uint64_t)kp / 8, n_pieces = (uint64_t)batch * per_row;
    uint64_t blocks = (n_pieces + 255) / 256;
    const uint64_t cap = (uint64_t)device_cu_count() * 16;
    if (blocks > cap) blocks = cap;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, static_cast<const f16*>(x),
                       static_cast<f16*>(xp), n_pieces, (uint32_t)per_row, (int)in);
    return hipGetLastError();
}

}  // namespace aqlm
