// Decode-phase product y[b][i] = s[i] * sum_k Wc[i][k] x[b][k], batch 1..16.
//
// "The AQLM Quantization Algorithm, Explained": weights are dequantized at
// run time after being fetched from memory (section "Why and what do we
// quantize?"); Figure 2 of the MCQ section gives the dequantization (sum of
// one codeword per codebook, then the row scale).  Decoding is memory-bound
// (same section), so this kernel streams every code byte exactly once and
// keeps everything else on chip.
//
// Work decomposition (one workgroup of 16 waves per CU):
//  * rows are cut into tiles of 16 (the M side of a 16x16x32 fp16 matrix-core
//    product); workgroup w of the W workgroups of a layer owns its row tiles
//    w, w + W, w + 2W, ...
//  * the input dimension is cut into slabs of 32 groups (256 inputs); the
//    waves of a workgroup take slabs round-robin, and for each slab keep the
//    activation operand (x, batch padded to 16 columns) in registers while
//    they run through the workgroup's row tiles;
//  * one 16-byte load gives lane l the codes of groups 8*(l/16) .. 8*(l/16)+7
//    of its slab in row l%16; lane l decodes group 8*(l/16) + q for the q-th
//    product;
//  * the x operand gives lane l batch row l%16, so the 16 lanes of a quarter
//    read 16 different rows.  At batch 1-2 (2x8) few lanes are active and x
//    is loaded straight into registers; otherwise each wave first copies its
//    slab's x rows into an LDS stage of its own with direct-to-LDS loads in
//    which four consecutive lanes read 64 contiguous bytes of one row, then
//    reads the operand layout from the stage (a direct load at batch 16
//    looks up one cache line per lane, which made x the largest cost);
//  * the 2x8 codebooks live in LDS, replicated REPL times with entry k of
//    replica r at 16-byte slot (2k + m) * REPL + r; lane l reads replica
//    l % REPL.  The LDS serves a 16-byte read to 16 lanes per clock from 16
//    bank groups (measured: about 4.8 clocks a conflict-free wave read,
//    8.5 when pairs of lanes share a group), so with REPL = 8 (64 KB, up to
//    batch 8) lane l reads codebook (l / 8) % 2 first: the 16 lanes served
//    together then touch 16 distinct groups.  With the 16-row x stage (128 KB)
//    above batch 8 only 4 replicas fit.  1x16 codewords are gathered from the
//    L2-resident 1 MiB codebook;
//  * at batch 1-2 on layers with at least two slab steps per wave, and at
//    batch 3-4 with at least four, the streaming kernel of gemv_stream.hip
//    runs instead (gemv_stream_lds);
//  * the other 2-bit schemes with B = 8 ("Key AQLM quantization parameters":
//    1x8 g4, 4x8 g16, 8x8 g32 cost the same bits as 2x8) store in/4 code bytes
//    per row too, so the same decomposition serves them; only the decode of a
//    piece of 8 inputs and the codebook copy differ (chunk_mfma, cb_slots);
//  * per-wave partial tiles are summed in LDS; the row scale is applied once
//    in fp32 and y is rounded to fp16.
//
// One launch can serve several layers that share x (the q, k and v
// projections of an attention block, the gate and up projections of its
// MLP): each workgroup belongs to one layer, whose codebooks it stages, and
// walks that layer's row tiles exactly as a launch for that layer alone
// would, so the results are bit-identical to separate launches.  The launch
// and the first-load, codebook-staging and reduction latencies are then paid
// once per group of layers instead of once per layer.
#include <algorithm>

#include "aqlm_device.h"
#include "aqlm_launch.h"
#include "gemv_body.h"

namespace aqlm {

// One layer: its arguments directly (a small argument block, read in one round trip).
template <int SCHEME, int REPL, bool VEC, int RTP, int XM>
__global__ __launch_bounds__(kGemvThreads) void gemv_kernel(const uint8_t* __restrict__ codes,
                                                            const f16* __restrict__ codebooks,
                                                            const f16* __restrict__ scales, f16* __restrict__ y,
                                                            int out, const f16* __restrict__ x, int in, int T) {
    gemv_body<SCHEME, REPL, VEC, RTP, XM>(codes, codebooks, scales, y, out, (int)blockIdx.x, (int)gridDim.x, x, in, T);
}

// Several layers that share x: the workgroup's layer is the number of layer ends at
// or below blockIdx.x; its first and last workgroups are picked from the ends
// already in scalar registers.
template <int SCHEME, int REPL, bool VEC, int RTP, int XM>
__global__ __launch_bounds__(kGemvThreads) void gemv_fused_kernel(const GemvLayers L, const f16* __restrict__ x,
                                                                  int in, int T) {
    int li = 0, wg0 = 0, wg1 = L.wg_end[0];
#pragma unroll
    for (int i = 0; i + 1 < kGemvMaxLayers; ++i) {
        const bool past = i + 1 < L.n && (int)blockIdx.x >= L.wg_end[i];
        li += past ? 1 : 0;
        wg0 = past ? L.wg_end[i] : wg0;
        wg1 = past ? L.wg_end[i + 1] : wg1;
    }
    gemv_body<SCHEME, REPL, VEC, RTP, XM>(static_cast<const uint8_t*>(L.codes[li]),
                                      static_cast<const f16*>(L.codebooks[li]),
                                      static_cast<const f16*>(L.scales[li]), static_cast<f16*>(L.y[li]), L.out[li],
                                      (int)blockIdx.x - wg0, wg1 - wg0, x, in, T);
}

template <int SCHEME, int REPL, bool VEC, int RTP, int XM>
static hipError_t launch_gemv_t(const GemvLayers& layers, const void* x, int in, int T, hipStream_t stream) {
    const bool fused = layers.n > 1;
    const void* kern = fused ? (const void*)gemv_fused_kernel<SCHEME, REPL, VEC, RTP, XM>
                             : (const void*)gemv_kernel<SCHEME, REPL, VEC, RTP, XM>;
    const size_t lds = (size_t)cb_slots<SCHEME, REPL>() * 16 +
                       std::max((size_t)kGemvWaves * kRedStride * sizeof(float),
                                (size_t)kGemvWaves * kXStageSlots(XM) * 16);
    if (lds > 65536) {
        hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    if (fused)
        hipLaunchKernelGGL((gemv_fused_kernel<SCHEME, REPL, VEC, RTP, XM>), dim3(layers.wg_end[layers.n - 1]),
                           dim3(kGemvThreads), lds, stream, layers, (const f16*)x, in, T);
    else
        hipLaunchKernelGGL((gemv_kernel<SCHEME, REPL, VEC, RTP, XM>), dim3(layers.wg_end[0]), dim3(kGemvThreads), lds,
                           stream, static_cast<const uint8_t*>(layers.codes[0]),
                           static_cast<const f16*>(layers.codebooks[0]), static_cast<const f16*>(layers.scales[0]),
                           static_cast<f16*>(layers.y[0]), layers.out[0], (const f16*)x, in, T);
    return hipGetLastError();
}

// Deals at most one workgroup per compute unit to the layers: a layer with
// n_rt row tiles and w workgroups costs ceil(n_rt / w) tile passes, and each
// further workgroup goes to the layer that costs most (a single layer gets
// min(n_rt, CUs) workgroups).
static void deal_workgroups(GemvLayers& layers, int cus) {
    int w[kGemvMaxLayers], n_rt[kGemvMaxLayers];
    int total = 0;
    for (int l = 0; l < layers.n; ++l) {
        n_rt[l] = (layers.out[l] + kRowTile - 1) / kRowTile;
        w[l] = 1;
        ++total;
    }
    while (total < cus) {
        int best = -1, best_cost = 1;
        for (int l = 0; l < layers.n; ++l) {
            const int cost = (n_rt[l] + w[l] - 1) / w[l];
            if (cost > best_cost || (cost == best_cost && best >= 0 && n_rt[l] > n_rt[best])) {
                best = l;
                best_cost = cost;
            }
        }
        if (best < 0) break;   // every layer already has one workgroup per row tile
        ++w[best];
        ++total;
    }
    int end = 0;
    for (int l = 0; l < layers.n; ++l) {
        end += w[l];
        layers.wg_end[l] = end;
    }
}

template <int SCHEME, int REPL, int RTP, int XM>
static hipError_t launch_gemv_v(const GemvLayers& layers, const void* x, int n, int T, hipStream_t stream) {
    return (n % 64) == 0   // 16-byte aligned code rows
               ? launch_gemv_t<SCHEME, REPL, true, RTP, XM>(layers, x, n, T, stream)
               : launch_gemv_t<SCHEME, REPL, false, RTP, XM>(layers, x, n, T, stream);
}

// Up to this batch the 2x8 product loads x directly (a few active lanes per
// load); above it x is staged.
constexpr int kGemvDirectBatch2x8 = 2;
// Above this batch 16 rows are staged: for 2x8 in two halves through an 8-row
// stage, so that the codebooks keep 8 replicas (LDS: 64 + 64 KB; with a 16-row
// stage only 4 fit, and their lookups met 2-way bank conflicts).
constexpr int kGemvStage8Batch = 8;

template <int RTP>
static hipError_t launch_gemv_2x8(const GemvLayers& layers, const void* x, int n, int T, hipStream_t stream) {
    if (T <= kGemvDirectBatch2x8) return launch_gemv_v<kScheme2x8, 8, RTP, kXDirect>(layers, x, n, T, stream);
    if (T <= kGemvStage8Batch) return launch_gemv_v<kScheme2x8, 8, RTP, kXStaged8>(layers, x, n, T, stream);
    return launch_gemv_v<kScheme2x8, 8, RTP, kXStaged16in8>(layers, x, n, T, stream);
}

// The other 2-bit B = 8 schemes: as 2x8, with the replicas that fit next to the x stage.
// 1x8 g4 (2 KB a copy): 8 replicas.  4x8 g16 (32 KB a copy, four lookups a piece, bound
// by LDS bank conflicts): direct x with 4 replicas at batches 1-2 and above 8, the 8-row
// stage with 3 replicas at 3-8 (measured faster than the 16-row stage, which leaves room
// for one copy, on the 11008-row and 11008-input layers).  8x8 g32 (128 KB): one copy
// and direct x loads (no room for a stage); its launcher takes it only above batch 8.
template <int RTP>
static hipError_t launch_gemv_b8(int scheme, const GemvLayers& layers, const void* x, int n, int T,
                                 hipStream_t stream) {
    if (scheme == kSchemeB8M1) {
        if (T <= kGemvDirectBatch2x8) return launch_gemv_v<kSchemeB8M1, 8, RTP, kXDirect>(layers, x, n, T, stream);
        if (T <= kGemvStage8Batch) return launch_gemv_v<kSchemeB8M1, 8, RTP, kXStaged8>(layers, x, n, T, stream);
        return launch_gemv_v<kSchemeB8M1, 8, RTP, kXStaged16>(layers, x, n, T, stream);
    }
    if (scheme == kSchemeB8M4) {
        if (T > kGemvDirectBatch2x8 && T <= kGemvStage8Batch)
            return launch_gemv_v<kSchemeB8M4, 3, RTP, kXStaged8>(layers, x, n, T, stream);
        return launch_gemv_v<kSchemeB8M4, 4, RTP, kXDirect>(layers, x, n, T, stream);
    }
    return launch_gemv_v<kSchemeB8M8, 1, RTP, kXDirect>(layers, x, n, T, stream);
}

template <int RTP>
static hipError_t launch_gemv_1x16(const GemvLayers& layers, const void* x, int n, int T, hipStream_t stream) {
    if (T <= kGemvStage8Batch) return launch_gemv_v<kScheme1x16, 1, RTP, kXStaged8>(layers, x, n, T, stream);
    return launch_gemv_v<kScheme1x16, 1, RTP, kXStaged16>(layers, x, n, T, stream);
}

// Layer l of a group as a group of its own.
static GemvLayers one_layer(const GemvLayers& g, int l) {
    GemvLayers one = {};
    one.codes[0] = g.codes[l];
    one.codebooks[0] = g.codebooks[l];
    one.scales[0] = g.scales[l];
    one.y[0] = g.y[l];
    one.out[0] = g.out[l];
    one.n = 1;
    return one;
}

static void add_layer(GemvLayers& g, const GemvLayers& from, int l) {
    g.codes[g.n] = from.codes[l];
    g.codebooks[g.n] = from.codebooks[l];
    g.scales[g.n] = from.scales[l];
    g.y[g.n] = from.y[l];
    g.out[g.n] = from.out[l];
    ++g.n;
}

// 2x8: the streaming kernel serves a layer of a group only where it would serve
// that layer alone (the two kernels add in different orders), so that a fused
// call gives bit for bit what separate calls give.  The layers it serves share
// one launch when their LDS fits, the others one launch of gemv_fused_kernel.
template <int RTP>
static hipError_t launch_gemv_2x8_group(const GemvLayers& layers, const void* x, int64_t in, int64_t batch,
                                        int cus, hipStream_t stream) {
    GemvLayers streamed = {}, rest = {};
    for (int l = 0; l < layers.n; ++l) {
        GemvLayers one = one_layer(layers, l);
        deal_workgroups(one, cus);
        if (gemv_stream_lds(one, in, batch) > 0) add_layer(streamed, layers, l);
        else add_layer(rest, layers, l);
    }
    if (streamed.n > 0) {
        deal_workgroups(streamed, cus);
        const size_t lds = gemv_stream_lds(streamed, in, batch);
        if (lds > 0) {
            const hipError_t e = launch_gemv_stream(streamed, x, in, batch, lds, stream);
            if (e != hipSuccess) return e;
        } else {   // together they need more LDS: one launch each
            for (int l = 0; l < streamed.n; ++l) {
                GemvLayers one = one_layer(streamed, l);
                deal_workgroups(one, cus);
                const hipError_t e = launch_gemv_stream(one, x, in, batch, gemv_stream_lds(one, in, batch), stream);
                if (e != hipSuccess) return e;
            }
        }
    }
    if (rest.n > 0) {
        deal_workgroups(rest, cus);
        return launch_gemv_2x8<RTP>(rest, x, (int)in, (int)batch, stream);
    }
    return hipSuccess;
}

hipError_t launch_gemv_fused(int scheme, GemvLayers layers, const void* x, int64_t in,
                             int64_t batch, hipStream_t stream) {
    constexpr int RTP = 2;
    if (layers.n < 1) return hipSuccess;
    const int cus = device_cu_count();
    if (scheme == kScheme2x8) return launch_gemv_2x8_group<RTP>(layers, x, in, batch, cus, stream);
    deal_workgroups(layers, cus);
    const int n = (int)in, T = (int)batch;
    if (scheme == kScheme1x16) return launch_gemv_1x16<RTP>(layers, x, n, T, stream);
    return launch_gemv_b8<RTP>(scheme, layers, x, n, T, stream);
}

hipError_t launch_gemv(int scheme, const void* codes, const void* codebooks, const void* scales,
                       const void* x, void* y, int64_t out, int64_t in, int64_t batch,
                       hipStream_t stream) {
    GemvLayers layers = {};
    layers.codes[0] = codes;
    layers.codebooks[0] = codebooks;
    layers.scales[0] = scales;
    layers.y[0] = y;
    layers.out[0] = (int)out;
    layers.n = 1;
    return launch_gemv_fused(scheme, layers, x, in, batch, stream);
}

}  // namespace aqlm
