// Decode-phase products (batch 1..16) with an epilogue, and the gated product of two layers:
// the bodies of gemv_body.h and gemv_stream.hip with their epilogue kinds, one launch, no
// workspace.
//
// Bounds and layout are those of the plain products (gemv.hip): the codes are read once, and
// the lookups, the fixed latencies and the launch bound the time.  The gated product reads x
// and stages the codebooks once for both layers and writes one output per pair of rows.
//
// Schemes without a tuned body (gemv_generic_kernel's): a wave per output row adds the row's
// products over its lanes, layer after layer, weights in fp32.
#include <algorithm>

#include "act_launch.h"
#include "aqlm_device.h"
#include "generic_codes.h"
#include "gemv_body.h"

namespace aqlm {

namespace {

constexpr int kRtp = 2;   // row tiles a pass, as the plain launches

template <int SCHEME, int REPL, bool VEC, int XM, int KIND>
__global__ __launch_bounds__(kGemvThreads) void gemv_act_kernel(const uint8_t* __restrict__ codes,
                                                                const f16* __restrict__ codebooks,
                                                                const f16* __restrict__ scales, f16* y, int out,
                                                                const f16* __restrict__ x, int in, int T, GemvEpi epi) {
    gemv_body<SCHEME, REPL, VEC, kRtp, XM, KIND>(codes, codebooks, scales, y, out, (int)blockIdx.x, (int)gridDim.x, x, in,
                                                 T, epi);
}

// One call's operands.
struct ActCall {
    const ActLayers& L;
    const GemvEpi& epi;
    const void* x;
    void* y;
    int out, in, T;
    hipStream_t stream;
};

template <int SCHEME, int REPL, int XM, int KIND>
hipError_t launch_v(const ActCall& c) {
    auto kern = c.in % 64 == 0 ? gemv_act_kernel<SCHEME, REPL, true, XM, KIND>   // 16-byte aligned code rows
                               : gemv_act_kernel<SCHEME, REPL, false, XM, KIND>;
    const size_t lds = (size_t)cb_slots<SCHEME, REPL>() * 16 +
                       std::max((size_t)kGemvWaves * kRedStride * sizeof(float),
                                (size_t)kGemvWaves * kXStageSlots(XM) * 16);
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    constexpr int tile = KIND == kGemvGated ? kRowTile / 2 : kRowTile;
    const int grid = std::min((c.out + tile - 1) / tile, device_cu_count());
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kGemvThreads), lds, c.stream, static_cast<const uint8_t*>(c.L.codes[0]),
                       static_cast<const f16*>(c.L.codebooks[0]), static_cast<const f16*>(c.L.scales[0]),
                       static_cast<f16*>(c.y), c.out, static_cast<const f16*>(c.x), c.in, c.T, c.epi);
    return hipGetLastError();
}

// How x reaches the registers and how many codebook replicas fit next to it: as the plain
// launches choose (gemv.hip), but for 4x8 g16: four replicas, read without conflicts, and direct
// x loads at batch 1 and 2 (gated: to 8), else two replicas, read with 2-way conflicts, and staged x:
// 4096^2 at batch 8 7.1 us (direct 7.9), at 16 7.6 (12.2); gated 4096x11008 at 4 21.7 (direct
// 19.8), at 16 22.7 (25.1).
template <int KIND>
hipError_t launch_tuned(int scheme, const ActCall& c) {
    const bool one = c.T <= 2, eight = c.T <= 8;
    switch (scheme) {
        case kScheme2x8:
            if (one) return launch_v<kScheme2x8, 8, kXDirect, KIND>(c);
            return eight ? launch_v<kScheme2x8, 8, kXStaged8, KIND>(c) : launch_v<kScheme2x8, 8, kXStaged16in8, KIND>(c);
        case kScheme1x16:
            return eight ? launch_v<kScheme1x16, 1, kXStaged8, KIND>(c) : launch_v<kScheme1x16, 1, kXStaged16, KIND>(c);
        case kSchemeB8M1:
            if (one) return launch_v<kSchemeB8M1, 8, kXDirect, KIND>(c);
            return eight ? launch_v<kSchemeB8M1, 8, kXStaged8, KIND>(c) : launch_v<kSchemeB8M1, 8, kXStaged16, KIND>(c);
        default:
            if (!eight) return launch_v<kSchemeB8M4, 2, kXStaged16in8, KIND>(c);
            if constexpr (KIND == kGemvAct) {
                if (!one) return launch_v<kSchemeB8M4, 2, kXStaged8, KIND>(c);
            }
            return launch_v<kSchemeB8M4, 4, kXDirect, KIND>(c);
    }
}

// Any scheme: wave w of a workgroup takes rows 16 blockIdx + w, stepping by 16 gridDim, and
// both layers of a row; lane l takes the row's groups l, l + 64, ...
template <int G, int CB, int KIND>
__global__ __launch_bounds__(kGemvThreads) void gemv_act_generic_kernel(const uint8_t* __restrict__ codes,
                                                                        const f16* __restrict__ codebooks,
                                                                        const f16* __restrict__ scales, f16* y, int out,
                                                                        const f16* __restrict__ x, int in, int T, int M,
                                                                        int B, GemvEpi epi) {
    constexpr int kN = KIND == kGemvGated ? 2 : 1, kMaxT = 16;
    const uint32_t mask = (1u << B) - 1u;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n_grp = in / G;
    for (int row = (int)blockIdx.x * 16 + wave; row < out; row += (int)gridDim.x * 16) {
        float acc[kN][kMaxT];
#pragma unroll
        for (int l = 0; l < kN; ++l) {
            const uint8_t* cl = l ? epi.codes1 : codes;
            const f16* cb = l ? epi.codebooks1 : codebooks;
#pragma unroll
            for (int b = 0; b < kMaxT; ++b) acc[l][b] = 0.f;
            for (int j = lane; j < n_grp; j += 64) {
                float v[G];
                group_weights<G, CB>(cl, ((size_t)row * n_grp + j) * M, cb, M, B, mask, v);
#pragma unroll
                for (int b = 0; b < kMaxT; ++b) {
                    if (b < T) {
                        constexpr int N = G < 8 ? G : 8;
                        float d = 0.f;
#pragma unroll
                        for (int p = 0; p < G / N; ++p) {
                            float xv[N];
                            load_f16<N>(x + (size_t)b * in + (size_t)j * G + p * N, xv);
#pragma unroll
                            for (int t = 0; t < N; ++t) d += v[p * N + t] * xv[t];
                        }
                        acc[l][b] += d;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kMaxT; ++b) {
                if (b < T) {
                    float a = acc[l][b];
#pragma unroll
                    for (int o = 32; o >= 1; o >>= 1) a += __shfl_xor(a, o, 64);
                    acc[l][b] = a;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kMaxT; ++b)   // lane b finishes batch row b
            if (b < T && lane == b) gemv_finish<KIND>(acc[0][b], acc[kN - 1][b], scales, y, b, row, out, epi);
    }
}

template <int KIND>
hipError_t launch_generic(const GenericScheme& sc, const ActCall& c) {
    const int grid = std::min((c.out + 15) / 16, 2 * device_cu_count());
#define AQLM_GEN(G, CB)                                                                                             \
    hipLaunchKernelGGL((gemv_act_generic_kernel<G, CB, KIND>), dim3(grid), dim3(kGemvThreads), 0, c.stream,            \
                       static_cast<const uint8_t*>(c.L.codes[0]), static_cast<const f16*>(c.L.codebooks[0]),          \
                       static_cast<const f16*>(c.L.scales[0]), static_cast<f16*>(c.y), c.out,                         \
                       static_cast<const f16*>(c.x), c.in, c.T, sc.M, sc.B, c.epi)
#define AQLM_GEN_G(G)                                                                                               \
    case G:                                                                                                         \
        if (sc.B <= 8) AQLM_GEN(G, 1);                                                                               \
        else AQLM_GEN(G, 2);                                                                                         \
        break;
    switch (sc.g) {
        AQLM_GEN_G(1)
        AQLM_GEN_G(2)
        AQLM_GEN_G(4)
        AQLM_GEN_G(8)
        AQLM_GEN_G(16)
        AQLM_GEN_G(32)
        default: return hipErrorInvalidValue;
    }
#undef AQLM_GEN_G
#undef AQLM_GEN
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv_act(const GenericScheme& sc, const ActLayers& L, const void* x, const Epilogue& e, int64_t out,
                           int64_t in, int64_t batch, hipStream_t stream) {
    GemvEpi epi = {};
    if (L.n == 2) {
        epi.codes1 = static_cast<const uint8_t*>(L.codes[1]);
        epi.codebooks1 = static_cast<const f16*>(L.codebooks[1]);
        epi.scales1 = static_cast<const f16*>(L.scales[1]);
    }
    for (int l = 0; l < L.n; ++l) {
        epi.bias[l] = static_cast<const f16*>(e.bias[l]);
        epi.z[l] = static_cast<f16*>(e.z[l]);
    }
    epi.residual = static_cast<const f16*>(e.residual);
    epi.act = e.act;
    const ActCall c = {L, epi, x, e.y, (int)out, (int)in, (int)batch, stream};
    int scheme = kSchemeGeneric;
    if (sc.M == 2 && sc.B == 8 && sc.g == 8) {
        hipError_t r = hipSuccess;
        if (launch_gemv_stream_act(L, epi, x, e.y, out, in, batch, stream, &r)) return r;
        scheme = kScheme2x8;
    } else if (sc.M == 1 && sc.B == 16 && sc.g == 8) {
        scheme = kScheme1x16;
    } else if (sc.B == 8 && sc.g == 4 * sc.M && in % 8 == 0 && (sc.M == 1 || sc.M == 4)) {
        scheme = sc.M == 1 ? kSchemeB8M1 : kSchemeB8M4;
    }
    if (scheme == kSchemeGeneric) return L.n == 2 ? launch_generic<kGemvGated>(sc, c) : launch_generic<kGemvAct>(sc, c);
    return L.n == 2 ? launch_tuned<kGemvGated>(scheme, c) : launch_tuned<kGemvAct>(scheme, c);
}

}  // namespace aqlm
