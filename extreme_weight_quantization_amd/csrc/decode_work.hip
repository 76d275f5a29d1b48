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

// 16-byte LDS slots of a scheme's codebooks: 2x8 codeword k of codebook m at 256 m + k; 4x8 g16
// half h of it at 1024 h + 256 m + k; 1x8 g4 codeword k in 8-byte slot k.  1x16 codewords
// are gathered from L2, those of any other scheme (kSchemeGeneric) read through it.
template <int SCHEME>
constexpr int work_cb_slots() {
    return SCHEME == kScheme2x8 ? 2 * kCodewords2x8 : SCHEME == kSchemeB8M4 ? 8 * kCodewords2x8
         : SCHEME == kSchemeB8M1 ? kCodewords2x8 / 2 : 1;
}

template <int SCHEME>
__device__ __forceinline__ void stage_codebooks(u32x4* lds, const f16* __restrict__ codebooks) {
    if constexpr (SCHEME == kScheme2x8 || SCHEME == kSchemeB8M1) {
        for (int i = threadIdx.x; i < work_cb_slots<SCHEME>(); i += blockDim.x) lds[i] = load16(codebooks + (size_t)i * 8);
    } else if constexpr (SCHEME == kSchemeB8M4) {
        for (int i = threadIdx.x; i < work_cb_slots<SCHEME>(); i += blockDim.x)
            lds[i] = load16(codebooks + (size_t)(i & 1023) * 16 + (i >> 10) * 8);
    }
    __syncthreads();
}

// The codes of piece p (inputs 8p .. 8p+7) of a row of P whole pieces, p clamped into it; 4x8
// g16: those of its group.  Nothing for kSchemeGeneric.
template <int SCHEME>
__device__ __forceinline__ uint32_t piece_codes(const uint8_t* __restrict__ codes, uint32_t row, uint32_t p, uint32_t P) {
    if constexpr (SCHEME == kSchemeGeneric) return 0u;
    p = min(p, P - 1);
    if constexpr (SCHEME == kSchemeB8M4)
        return reinterpret_cast<const uint32_t*>(codes)[(size_t)row * (P / 2) + (p >> 1)];
    return reinterpret_cast<const uint16_t*>(codes)[(size_t)row * P + p];
}

// a + b in fp32 as fma(a, 1, b): one instruction on the fp16 values (v_fma_mix_f32) instead of
// two conversions and an addition.  The 1 is hidden from the compiler, which would fold it.
__device__ __forceinline__ float hidden_one() {
    float one = 1.f;
    asm("" : "+v"(one));
    return one;
}

// The fp32 weights of piece p of a row before the scale, zero past `in`, from its codes c
// (kSchemeGeneric, g = G, code storage CB: read here).
template <int SCHEME, int G, int CB>
__device__ __forceinline__ void piece_weights(uint32_t c, const uint8_t* __restrict__ codes,
                                              const f16* __restrict__ codebooks, const u32x4* lds, uint32_t row,
                                              uint32_t p, int in, int M, int B, float (&v)[8]) {
    [[maybe_unused]] const float one = hidden_one();
    if constexpr (SCHEME == kScheme2x8) {
        const f16x8 a = as_f16x8(lds[c & 0xff]), b = as_f16x8(lds[kCodewords2x8 + (c >> 8)]);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = __builtin_fmaf((float)a[t], one, (float)b[t]);
    } else if constexpr (SCHEME == kScheme1x16) {
        const f16x8 a = as_f16x8(load16(codebooks + (size_t)c * kGroup));
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = (float)a[t];
    } else if constexpr (SCHEME == kSchemeB8M1) {
        const u32x2* lds8 = reinterpret_cast<const u32x2*>(lds);
        const u32x2 lo = lds8[c & 0xff], hi = lds8[c >> 8];
        const f16x8 a = as_f16x8(u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = (float)a[t];
    } else if constexpr (SCHEME == kSchemeB8M4) {
        const u32x4* half = lds + 1024 * (p & 1);
        f16x8 a[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) a[m] = as_f16x8(half[256 * m + ((c >> (8 * m)) & 0xff)]);
#pragma unroll
        for (int t = 0; t < 8; ++t)
            v[t] = __builtin_fmaf((float)a[3][t], one,
                                  __builtin_fmaf((float)a[2][t], one, __builtin_fmaf((float)a[0][t], one, (float)a[1][t])));
    } else {
        const uint32_t mask = (1u << B) - 1u;
        const int n_grp = in / G, k = (int)p * 8;
        const size_t rbase = (size_t)row * n_grp;
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = 0.f;
        if constexpr (G >= 8) {
            if (k < in) sum_codewords<G, 8, CB>(codes, (rbase + k / G) * M, codebooks, M, B, mask, k % G, v);
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
    if constexpr (SCHEME != kSchemeGeneric) {
        const bool inside = (int)p * 8 < in;
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = inside ? v[t] : 0.f;
    }
}

// The row's factor under the weight-scale mode.
template <WeightScale WS>
__device__ __forceinline__ float row_factor(const f16* __restrict__ scales, uint32_t row) {
    if constexpr (WS == WeightScale::kNone) return 1.f;
    return (float)scales[row];
}

// A workgroup's 256 threads take 256 >> shift rows of 1 << shift pieces each, so a piece's row
// and place come from shifts and scalars.  The layers are decoded one after the other: one 1x16
// codebook at a time in L2.  Two, four or eight pieces a thread in hand change the time by less than 10 %:
// the write bounds it.  Between products that read the weights it takes 1.4-1.7 times what the same launch
// takes when it only follows itself (28672x8192 2x8 125 against 88 us, 1x16 250 against 146): a
// product keeps the clock near 1.5 GHz and leaves its weights in the last-level cache.
constexpr int kRowThreads = 256;

template <int SCHEME, int G, int CB, WeightScale WS>
__global__ __launch_bounds__(kRowThreads) void decode_rows_kernel(DecodeArgs a, int n, int out, int per_row, int shift,
                                                                  int chunks, int n_items, int in, int M, int B) {
    __shared__ u32x4 cb_lds[work_cb_slots<SCHEME>()];
    const uint32_t P = (uint32_t)in / 8;   // whole pieces of a row (the schemes but kSchemeGeneric: in % 8 == 0)
    const int trow = threadIdx.x >> shift, tp = threadIdx.x & ((1 << shift) - 1);
    for (int l = 0; l < n; ++l) {
        const uint8_t* codes = l ? a.codes[1] : a.codes[0];
        const f16* codebooks = l ? a.codebooks[1] : a.codebooks[0];
        const f16* scales = l ? a.scales[1] : a.scales[0];
        f16* w = l ? a.w[1] : a.w[0];
        if (l > 0) __syncthreads();   // the first layer's lookups are done
        stage_codebooks<SCHEME>(cb_lds, codebooks);
        for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
            const int rb = item / chunks, ch = item - rb * chunks;   // scalars: row block, chunk of the row
            const int row = (rb << (8 - shift)) + trow, p = (ch << shift) + tp;
            if (row >= out || p >= per_row) continue;
            const uint32_t c = piece_codes<SCHEME>(codes, row, p, P);
            float v[8];
            piece_weights<SCHEME, G, CB>(c, codes, codebooks, cb_lds, row, p, in, M, B, v);
            const float s = row_factor<WS>(scales, row);
            f16x8 o;
#pragma unroll
            for (int t = 0; t < 8; ++t) o[t] = (f16)__fmul_rn(v[t], s);
            // non-temporal: the write stream must not evict the codebook or the codes from L2
            __builtin_nontemporal_store(as_u32x4(o), reinterpret_cast<u32x4*>(w + ((size_t)row * per_row + p) * 8));
        }
    }
}

// The levels of dz's blocks and the one unit that each of its rows gets.
struct GradAlign {
    f16* dz;
    const int8_t* levels;
    float* units;
    int T, cols;   // tokens (0: nothing to do), level columns of a layer
};

// Lanes that share a row of dz: a power of two, one a block or 64.
__host__ __device__ inline int align_lanes(int n_blk) {
    int lanes = 1;
    while (lanes < 64 && lanes < n_blk) lanes *= 2;
    return lanes;
}

// Brings every row of dz to the unit of its largest level, since the dense product sums over whole rows, and
// writes the units; blocks at a lower level are rewritten.  Done here because this launch lies between
// the one that writes dz and the product anyway; levels are 20 bits apart, so few rows have two.
__device__ __forceinline__ void align_gradients(const GradAlign& g, int n, int op) {
    const int lane = threadIdx.x & 63, n_blk = n * g.cols, lanes = align_lanes(n_blk), rows = 64 / lanes;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    for (int64_t t0 = wave * rows; t0 < g.T; t0 += (int64_t)gridDim.x * 4 * rows) {
        const int64_t t = t0 + lane / lanes;
        int top = kLevelMin, low = kLevelMax;
        if (t < g.T) {
            for (int b = lane % lanes; b < n_blk; b += lanes) {
                const int v = g.levels[t * n_blk + b];
                top = max(top, v);
                low = min(low, v);
            }
        }
        for (int o = lanes / 2; o >= 1; o /= 2) {
            top = max(top, __shfl_xor(top, o, 64));
            low = min(low, __shfl_xor(low, o, 64));
        }
        const bool first = lane % lanes == 0 && t < g.T;
        if (first) g.units[t] = level_unit(top);
        for (uint64_t mixed = __ballot(first && low != top); mixed != 0; mixed &= mixed - 1) {   // the wave a row
            const int src = __ffsll((unsigned long long)mixed) - 1, highest = __shfl(top, src, 64);
            const int64_t row = t0 + src / lanes;
            for (int b = 0; b < n_blk; ++b) {
                const int d = highest - g.levels[row * n_blk + b];
                const int l = b / g.cols, c = (b - l * g.cols) * kLevelCols + 8 * lane;   // its 512 rows of W, 8 a lane
                if (d == 0 || c >= op) continue;
                u32x4* p = reinterpret_cast<u32x4*>(g.dz + row * n * op + (int64_t)l * op + c);
                *p = raise_level(*p, d);
            }
        }
    }
}

// Tiles of 64 rows x 32 pieces: thread (piece tid / 8, rows 8 (tid % 8) ..).  A workgroup stages
// the codebooks once and walks tiles; a tile's codes are loaded while the one before is decoded.
template <int SCHEME, int G, int CB, WeightScale WS>
__global__ __launch_bounds__(256) void decode_transposed_kernel(DecodeArgs a, int n, int out, int in, int op, int ldt,
                                                                int n_row_tiles, int n_tiles, int M, int B, GradAlign grads) {
    __shared__ u32x4 cb_lds[work_cb_slots<SCHEME>()];
    align_gradients(grads, n, op);
    if ((int)blockIdx.x >= n_tiles) return;   // the whole workgroup: few tiles, many rows of dz
    const uint32_t P = (uint32_t)in / 8;
    const int oct = threadIdx.x & 7, piece = threadIdx.x >> 3;
    auto row_of = [&](int tile) { return (tile % n_row_tiles) * 64 + 8 * oct; };
    auto piece_of = [&](int tile) { return (tile / n_row_tiles) * 32 + piece; };
    for (int l = 0; l < n; ++l) {
        const uint8_t* codes = l ? a.codes[1] : a.codes[0];
        const f16* codebooks = l ? a.codebooks[1] : a.codebooks[0];
        const f16* scales = l ? a.scales[1] : a.scales[0];
        auto load = [&](int tile, uint32_t (&c)[8], f16 (&s)[8]) {
            const int t = min(tile, n_tiles - 1);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int row = min(row_of(t) + r, out - 1);
                c[r] = piece_codes<SCHEME>(codes, row, piece_of(t), P);
                s[r] = scales[row];
            }
        };
        uint32_t c[8];
        f16 s[8];
        load(blockIdx.x, c, s);
        if (l > 0) __syncthreads();   // the first layer's lookups are done
        stage_codebooks<SCHEME>(cb_lds, codebooks);
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
            uint32_t cn[8];
            f16 sn[8];
            load(tile + gridDim.x, cn, sn);
            const int row0 = row_of(tile), p = piece_of(tile), k0 = 8 * p;
            if (k0 < in) {
                f16 o[8][8];   // [row][input]
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float v[8];
                    piece_weights<SCHEME, G, CB>(c[r], codes, codebooks, cb_lds, min(row0 + r, out - 1), p, in, M, B, v);
                    const float f = WS == WeightScale::kNone ? 1.f : (float)s[r];
#pragma unroll
                    for (int t = 0; t < 8; ++t) o[r][t] = (f16)__fmul_rn(v[t], f);
                }
                if ((tile % n_row_tiles) * 64 + 64 > out) {   // rows past the layer: zeros
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int t = 0; t < 8; ++t) o[r][t] = row0 + r < out ? o[r][t] : (f16)0.f;
                }
                f16* w = a.w[0] + (size_t)l * op + row0;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if (k0 + t < in) {
                        f16x8 x;
#pragma unroll
                        for (int r = 0; r < 8; ++r) x[r] = o[r][t];
                        *reinterpret_cast<u32x4*>(w + (size_t)(k0 + t) * ldt) = as_u32x4(x);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                c[r] = cn[r];
                s[r] = sn[r];
            }
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
                     const GradAlign& grads, hipStream_t stream) {
    if constexpr (T) {
        const int64_t n_rt = op / 64, n_pt = (in + 255) / 256;
        const int64_t tiles = n_rt * n_pt, cap = (int64_t)device_cu_count() * 8;
        if (tiles > INT32_MAX / 2) return hipErrorInvalidValue;
        const int64_t per = 4 * 64 / align_lanes(n * grads.cols);   // rows of dz a workgroup aligns at a time
        const int64_t rows = (grads.T + per - 1) / per, work = rows > tiles ? rows : tiles;
        hipLaunchKernelGGL((decode_transposed_kernel<SCHEME, G, CB, WS>), dim3((unsigned)(work < cap ? work : cap)),
                           dim3(256), 0, stream, a, n, (int)out, (int)in, (int)op, (int)ld, (int)n_rt, (int)tiles, M, B, grads);
    } else {
        const int64_t per_row = ld / 8;
        int shift = 0;
        while (shift < 8 && (1 << shift) < per_row) ++shift;
        const int64_t rows = kRowThreads >> shift, chunks = (per_row + (1 << shift) - 1) >> shift;
        const int64_t items = (out + rows - 1) / rows * chunks, cap = (int64_t)device_cu_count() * 16;
        if (items > INT32_MAX / 2) return hipErrorInvalidValue;
        hipLaunchKernelGGL((decode_rows_kernel<SCHEME, G, CB, WS>), dim3((unsigned)(items < cap ? items : cap)),
                           dim3(kRowThreads), 0, stream, a, n, (int)out, (int)per_row, shift, (int)chunks, (int)items,
                           (int)in, M, B);
    }
    return hipGetLastError();
}

template <bool T, int SCHEME, int G, int CB>
hipError_t launch_scheme(WeightScale ws, const DecodeArgs& a, int n, int64_t out, int64_t in, int64_t ld, int64_t op,
                         int M, int B, const GradAlign& grads, hipStream_t stream) {
    if (ws == WeightScale::kFull)
        return launch_ws<T, SCHEME, G, CB, WeightScale::kFull>(a, n, out, in, ld, op, M, B, grads, stream);
    return launch_ws<T, SCHEME, G, CB, WeightScale::kNone>(a, n, out, in, ld, op, M, B, grads, stream);
}

template <bool T>
hipError_t launch_any(const GenericScheme& sc, WeightScale ws, const DecodeArgs& a, int n, int64_t out, int64_t in,
                      int64_t ld, int64_t op, const GradAlign& grads, hipStream_t stream) {
    const int M = sc.M, B = sc.B;
    if (M == 2 && B == 8 && sc.g == 8)
        return launch_scheme<T, kScheme2x8, 8, 1>(ws, a, n, out, in, ld, op, M, B, grads, stream);
    if (M == 1 && B == 16 && sc.g == 8)
        return launch_scheme<T, kScheme1x16, 8, 2>(ws, a, n, out, in, ld, op, M, B, grads, stream);
    if (M == 4 && B == 8 && sc.g == 16)
        return launch_scheme<T, kSchemeB8M4, 16, 1>(ws, a, n, out, in, ld, op, M, B, grads, stream);
    if (M == 1 && B == 8 && sc.g == 4 && in % 8 == 0)
        return launch_scheme<T, kSchemeB8M1, 4, 1>(ws, a, n, out, in, ld, op, M, B, grads, stream);
#define AQLM_ROWS(G)                                                                                              \
    case G:                                                                                                       \
        return B <= 8 ? launch_scheme<T, kSchemeGeneric, G, 1>(ws, a, n, out, in, ld, op, M, B, grads, stream)            \
                      : launch_scheme<T, kSchemeGeneric, G, 2>(ws, a, n, out, in, ld, op, M, B, grads, stream);
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
    return launch_any<false>(sc, ws, a, L.n, out, in, kp, 0, GradAlign{}, stream);
}

hipError_t launch_decode_transposed(const GenericScheme& sc, const ActLayers& L, WeightScale ws, void* wt,
                                    int64_t out, int64_t in, int64_t op, hipStream_t stream) {
    DecodeArgs a = decode_args(L);
    a.w[0] = static_cast<f16*>(wt);
    GradAlign g = {};
    if (L.grads.dz != nullptr)
        g = GradAlign{static_cast<f16*>(L.grads.dz), grad_levels(L.grads.dz, L.n, op, L.grads.batch),
                      grad_units(L.grads.dz, L.n, op, L.grads.batch), (int)L.grads.batch, (int)grad_level_cols(op)};
    return launch_any<true>(sc, ws, a, L.n, out, in, L.n * op, op, g, stream);
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
