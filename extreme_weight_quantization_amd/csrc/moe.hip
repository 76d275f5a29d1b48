// A mixture-of-experts layer for few tokens, experts in an AQLM scheme: gate and up products with their activation, down
// product, weighted sum, in three launches.
//
// Bounds: the codes of the experts that are asked for, read once per 16 tokens (down: 8) of an expert; then the lookups, and for a
// single token the fixed latencies of the launches.  2x8, 64 experts of 2048 x 1408, 1 token of 8: 24 us in a graph (gate and up 11.6,
// down 9.0, combining 2); 1x16, 8 experts of 4096 x 11008, 16 tokens of 2: 560 to 620 us (by card), 217 to 241 G gathers a
// second of the 264 that a kernel of nothing else reaches.
//
// The products are those of gemv_act.hip: workgroups of 16 waves that hold the expert's codebooks in LDS (2x8, 1x8 g4,
// 4x8 g16) or gather codewords from L2 (1x16), on the columns that moe_plan.h finds.  An expert's workgroups are neighbours on
// one XCD, whose L2 then holds its codebook.  The hidden vector h of a pair (token, choice) is kept as two fp16 numbers (hidden_pair.h); the down
// product takes both as columns.  Its results stay apart per pair, in fp32, and the last launch weights and adds a
// token's pairs in the order of its choices: no atomics, the same result every time.
#include <algorithm>

#include "gemv_body.h"
#include "generic_codes.h"
#include "moe_plan.h"

namespace aqlm {

namespace {

// Rows of up to 8 slabs of 256 inputs would leave half of a workgroup's 16 waves without work: there two teams of 8 waves take a
// tile each, and a pass is one tile; else 16 waves a tile and two tiles a pass, as the plain launches.  In teams | not, us:
//   2x8, 64 experts 2048x1408: 1 token 24 | 28, 16 tokens 79 | 119; 8 experts 4096x11008: 1 token 52 | 47
constexpr int kTeam = 8;
constexpr int rtp(int team) { return team == kGemvWaves ? 2 : 1; }

// One launch's layers: rows x in of each expert, the second layer for the gated kind only.
struct MoeProduct {
    const uint8_t* codes[2];
    const f16* codebooks[2];
    const f16* scales[2];
    size_t codes_stride, codebooks_stride;   // bytes, entries
    const f16* x;
    f16* h;          // GatedAt: [pairs][2][rows]
    float* part;     // PartAt: [pairs][rows], before the weights
    const int32_t* ids;
    int experts, pairs, k, rows, in, act;
    float fixed;     // cost of starting on an item, in items
};

// Pairs of an item: as many as a way for x to reach the registers has columns for (two a pair in the down product).
constexpr int moe_chunk(int kind, int xm = kXDirect) { return (xm == kXStaged8 ? 8 : 16) / (kind == kGemvPartAt ? 2 : 1); }

template <int KIND>
__device__ __forceinline__ GemvEpi expert_epi(const MoeProduct& p, int e) {
    GemvEpi epi = {};
    if constexpr (KIND == kGemvGatedAt) {
        epi.codes1 = p.codes[1] + p.codes_stride * e;
        epi.codebooks1 = p.codebooks[1] + p.codebooks_stride * e;
        epi.scales1 = p.scales[1] + (size_t)p.rows * e;
    }
    epi.act = p.act;
    return epi;
}

template <int SCHEME, int REPL, bool VEC, int XM, int KIND, int TEAM>
__global__ __launch_bounds__(kGemvThreads) void moe_gemv_kernel(MoeProduct p) {
    __shared__ MoeLds m;
    constexpr int kChunk = moe_chunk(KIND, XM);
    constexpr int kTile = gemv_gated(KIND) ? kRowTile / 2 : kRowTile;
    const MoeItems items = moe_items<moe_chunk(KIND)>(p.ids, p.pairs, p.experts, kChunk, m);
    const int n = items.n;
    const int tiles = (p.rows + kTile - 1) / kTile;
    const int parts = moe_parts(n, (int)gridDim.x, tiles, p.fixed);
    for (int u = xcd_run((int)blockIdx.x, (int)gridDim.x); u < n * parts; u += (int)gridDim.x) {
        int e;
        const int cols = moe_item<KIND == kGemvPartAt>(items, u / parts, p.pairs, p.k, kChunk, m, e);
        gemv_body<SCHEME, REPL, VEC, rtp(TEAM), XM, KIND, TEAM>(
            p.codes[0] + p.codes_stride * e, p.codebooks[0] + p.codebooks_stride * e, p.scales[0] + (size_t)p.rows * e, p.h, p.rows,
            u % parts, parts, p.x, p.in, KIND == kGemvPartAt ? 2 * cols : cols, expert_epi<KIND>(p, e),
            GemvRows{m.x, m.y, p.part});
    }
}

template <int SCHEME, int REPL, int XM, int KIND, int TEAM>
hipError_t launch_team(const MoeProduct& p, hipStream_t stream) {
    auto kern = p.in % 64 == 0 ? moe_gemv_kernel<SCHEME, REPL, true, XM, KIND, TEAM>
                               : moe_gemv_kernel<SCHEME, REPL, false, XM, KIND, TEAM>;
    const size_t lds = (size_t)cb_slots<SCHEME, REPL>() * 16 +
                       std::max((size_t)kGemvWaves * kRedStride * sizeof(float),
                                (size_t)kGemvWaves * kXStageSlots(XM) * 16);
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(device_cu_count()), dim3(kGemvThreads), lds, stream, p);
    return hipGetLastError();
}

template <int SCHEME, int REPL, int XM, int KIND>
hipError_t launch_v(const MoeProduct& p, hipStream_t stream) {
    return p.in <= kTeam * kSlabGroups * kGroup ? launch_team<SCHEME, REPL, XM, KIND, kTeam>(p, stream)
                                                : launch_team<SCHEME, REPL, XM, KIND, kGemvWaves>(p, stream);
}

// How x reaches the registers, by the most columns of an expert whose pairs belong to different tokens: as gemv_act.hip chooses.
// Where tokens name an expert twice it may have more; they are an item of their own then (moe_chunk).
template <int KIND>
hipError_t launch_tuned(int scheme, const MoeProduct& p, int cols, hipStream_t stream) {
    const bool one = cols <= 2, eight = cols <= 8;
    switch (scheme) {
        case kScheme2x8:
            if (one) return launch_v<kScheme2x8, 8, kXDirect, KIND>(p, stream);
            return eight ? launch_v<kScheme2x8, 8, kXStaged8, KIND>(p, stream)
                         : launch_v<kScheme2x8, 8, kXStaged16in8, KIND>(p, stream);
        case kScheme1x16:
            return eight ? launch_v<kScheme1x16, 1, kXStaged8, KIND>(p, stream)
                         : launch_v<kScheme1x16, 1, kXStaged16, KIND>(p, stream);
        case kSchemeB8M1:
            if (one) return launch_v<kSchemeB8M1, 8, kXDirect, KIND>(p, stream);
            return eight ? launch_v<kSchemeB8M1, 8, kXStaged8, KIND>(p, stream)
                         : launch_v<kSchemeB8M1, 8, kXStaged16, KIND>(p, stream);
        default:
            if (!eight) return launch_v<kSchemeB8M4, 2, kXStaged16in8, KIND>(p, stream);
            if constexpr (KIND == kGemvPartAt) {
                if (!one) return launch_v<kSchemeB8M4, 2, kXStaged8, KIND>(p, stream);
            }
            return launch_v<kSchemeB8M4, 4, kXDirect, KIND>(p, stream);
    }
}

// Any scheme: wave w of a workgroup takes rows 16 part + w, stepping by 16 parts, and both layers of a row; lane l takes the
// row's groups l, l + 64, ...; weights in fp32.
template <int G, int CB, int KIND>
__global__ __launch_bounds__(kGemvThreads) void moe_generic_kernel(MoeProduct p, int M, int B) {
    __shared__ MoeLds m;
    constexpr int kChunk = moe_chunk(KIND), kN = KIND == kGemvGatedAt ? 2 : 1;
    const uint32_t mask = (1u << B) - 1u;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n_grp = p.in / G;
    const MoeItems items = moe_items<moe_chunk(KIND)>(p.ids, p.pairs, p.experts, kChunk, m);
    const int n = items.n;
    const int parts = moe_parts(n, (int)gridDim.x, (p.rows + 15) / 16, p.fixed);
    for (int u = xcd_run((int)blockIdx.x, (int)gridDim.x); u < n * parts; u += (int)gridDim.x) {
        int e;
        const int cols = moe_item<KIND == kGemvPartAt>(items, u / parts, p.pairs, p.k, kChunk, m, e);
        const GemvEpi epi = expert_epi<KIND>(p, e);
        const f16* scales = p.scales[0] + (size_t)p.rows * e;
        for (int row = u % parts * 16 + wave; row < p.rows; row += parts * 16) {
            float acc[kN][kChunk];
#pragma unroll
            for (int l = 0; l < kN; ++l) {
                const uint8_t* cl = l ? epi.codes1 : p.codes[0] + p.codes_stride * e;
                const f16* cb = l ? epi.codebooks1 : p.codebooks[0] + p.codebooks_stride * e;
#pragma unroll
                for (int b = 0; b < kChunk; ++b) acc[l][b] = 0.f;
                for (int j = lane; j < n_grp; j += 64) {
                    float v[G];
                    group_weights<G, CB>(cl, ((size_t)row * n_grp + j) * M, cb, M, B, mask, v);
#pragma unroll
                    for (int b = 0; b < kChunk; ++b) {
                        if (b < cols) {
                            constexpr int N = G < 8 ? G : 8;
                            float d = 0.f;
#pragma unroll
                            for (int q = 0; q < G / N; ++q) {
                                float xv[N];
                                load_f16<N>(p.x + (size_t)m.x[KIND == kGemvPartAt ? 2 * b : b] * p.in + (size_t)j * G + q * N, xv);
                                if constexpr (KIND == kGemvPartAt) {
                                    float lo[N];
                                    load_f16<N>(p.x + (size_t)m.x[2 * b + 1] * p.in + (size_t)j * G + q * N, lo);
#pragma unroll
                                    for (int t = 0; t < N; ++t) xv[t] += lo[t] * (1.f / kPairFine);
                                }
#pragma unroll
                                for (int t = 0; t < N; ++t) d += v[q * N + t] * xv[t];
                            }
                            acc[l][b] += d;
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < kChunk; ++b) {
                    if (b < cols) {
                        float a = acc[l][b];
#pragma unroll
                        for (int o = 32; o >= 1; o >>= 1) a += __shfl_xor(a, o, 64);
                        acc[l][b] = a;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kChunk; ++b) {   // lane b finishes column b
                if (b < cols && lane == b) {
                    if constexpr (KIND == kGemvPartAt)
                        p.part[(size_t)m.y[b] * p.rows + row] = acc[0][b] * kPairUnit * (float)scales[row];
                    else
                        gemv_finish_pair(acc[0][b], acc[kN - 1][b], scales, p.h, m.y[b], row, p.rows, epi);
                }
            }
        }
    }
}

template <int KIND>
hipError_t launch_generic(const GenericScheme& sc, const MoeProduct& p, hipStream_t stream) {
    const dim3 grid(2 * device_cu_count());
#define AQLM_GEN(G, CB) \
    hipLaunchKernelGGL((moe_generic_kernel<G, CB, KIND>), grid, dim3(kGemvThreads), 0, stream, p, sc.M, sc.B)
#define AQLM_GEN_G(G)                      \
    case G:                                \
        if (sc.B <= 8) AQLM_GEN(G, 1);      \
        else AQLM_GEN(G, 2);                \
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

template <int KIND>
hipError_t launch_product(const GenericScheme& sc, const MoeProduct& p, int cols, hipStream_t stream) {
    if (sc.M == 2 && sc.B == 8 && sc.g == 8) return launch_tuned<KIND>(kScheme2x8, p, cols, stream);
    if (sc.M == 1 && sc.B == 16 && sc.g == 8) return launch_tuned<KIND>(kScheme1x16, p, cols, stream);
    if (sc.B == 8 && sc.g == 4 * sc.M && p.in % 8 == 0 && (sc.M == 1 || sc.M == 4))
        return launch_tuned<KIND>(sc.M == 1 ? kSchemeB8M1 : kSchemeB8M4, p, cols, stream);
    return launch_generic<KIND>(sc, p, stream);
}

__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, const f16* residual, f16* y, int n, int in, int k, int experts) {
    const int at = (int)blockIdx.x * 256 + (int)threadIdx.x;
    if (at >= n) return;
    constexpr int kStep = 8;
    const int t = at / in, i = at % in;
    float s = 0.f;
    for (int j0 = 0; j0 < k; j0 += kStep) {   // kStep loads in flight
        int e[kStep];
        float v[kStep], w[kStep];
#pragma unroll
        for (int q = 0; q < kStep; ++q) {
            const size_t pair = (size_t)t * k + min(j0 + q, k - 1);
            e[q] = ids[pair];
            w[q] = weights[pair];
            v[q] = part[pair * in + i];
        }
#pragma unroll
        for (int q = 0; q < kStep; ++q)   // a pair without an expert has no part: whatever is there is left out
            if (j0 + q < k && e[q] >= 0 && e[q] < experts) s += w[q] * v[q];
    }
    if (residual != nullptr) s += (float)residual[at];
    y[at] = (f16)s;
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// The cost of starting on an item next to the item's whole work, for the deal of parts: about 2 us for codebooks and the
// first codes, against 2-bit codes at a workgroup's share of the memory rate (20 GB/s).
float start_cost(int layers, int64_t rows, int64_t in) { return 2.f / ((float)layers * (float)rows * (float)in / 4.f / 20e3f); }

}  // namespace

int64_t moe_workspace(int64_t in, int64_t inner, int64_t tokens, int64_t k) {
    return round256(tokens * k * 2 * inner * 2) + round256(tokens * k * in * 4);
}

hipError_t launch_moe_combine(const float* part, const MoeCall& c, hipStream_t stream) {
    const int n = (int)(c.tokens * c.in);
    hipLaunchKernelGGL(moe_combine_kernel, dim3((n + 255) / 256), dim3(256), 0, stream, part, c.ids, c.weights,
                       static_cast<const f16*>(c.residual), static_cast<f16*>(c.y), n, (int)c.in, c.k, c.experts);
    return hipGetLastError();
}

hipError_t launch_moe(const GenericScheme& sc, const MoeLayers& L, const MoeCall& c, void* workspace, hipStream_t stream) {
    f16* h = static_cast<f16*>(workspace);
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256((int64_t)c.pairs() * 2 * c.inner * 2));
    const size_t codebook = ((size_t)sc.M << sc.B) * sc.g, code = sc.B <= 8 ? 1 : 2;
    MoeProduct p = {};
    for (int l = 0; l < 2; ++l) {
        p.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        p.codebooks[l] = static_cast<const f16*>(L.codebooks[l]);
        p.scales[l] = static_cast<const f16*>(L.scales[l]);
    }
    p.codebooks_stride = codebook;
    p.codes_stride = (size_t)c.inner * (c.in / sc.g) * sc.M * code;
    p.x = static_cast<const f16*>(c.x);
    p.h = h;
    p.part = part;
    p.ids = c.ids;
    p.experts = c.experts;
    p.pairs = c.pairs();
    p.k = c.k;
    p.rows = (int)c.inner;
    p.in = (int)c.in;
    p.act = c.act;
    p.fixed = start_cost(2, c.inner, c.in);
    hipError_t r = launch_product<kGemvGatedAt>(sc, p, std::min(c.tokens, 16), stream);
    if (r != hipSuccess) return r;
    p.codes[0] = static_cast<const uint8_t*>(L.codes[2]);
    p.codebooks[0] = static_cast<const f16*>(L.codebooks[2]);
    p.scales[0] = static_cast<const f16*>(L.scales[2]);
    p.codes_stride = (size_t)c.in * (c.inner / sc.g) * sc.M * code;
    p.x = h;
    p.rows = (int)c.in;
    p.in = (int)c.inner;
    p.fixed = start_cost(1, c.inner, c.in);
    r = launch_product<kGemvPartAt>(sc, p, 2 * std::min(c.tokens, 8), stream);
    if (r != hipSuccess) return r;
    return launch_moe_combine(part, c, stream);
}

}  // namespace aqlm
